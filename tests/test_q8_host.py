"""Refusals of the calls over 8-bit pages: each is found on the host before
anything is launched, so they are tested without a GPU, on a zeroed handle."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from split_kv_flash_attn_gb300 import build as b
    b.build()
    from split_kv_flash_attn_gb300 import _lib
    return _lib.load()


@pytest.fixture()
def hnd():
    return ctypes.create_string_buffer(1 << 16)        # stands for a handle: refusals read nothing of it


A = 1 << 20                                            # an address that is never followed, 16-byte aligned


def _pool(**kw):
    from split_kv_flash_attn_gb300 import _lib
    d = dict(n_pages=10, D=128, k=A, v=A, k_scale=A, v_scale=A, k_min=A, k_max=A)
    d.update(kw)
    return _lib.SkvQ8Pool(*d.values())


def _shape(**kw):
    from split_kv_flash_attn_gb300 import _lib
    d = dict(S=2, nq=1, H=8, Hk=2, D=128, scale=0.1, k_type=0, v_type=0, k_row_bytes=0, v_row_bytes=0)
    d.update(kw)
    return _lib.SkvShape(*d.values())


BAD_POOL = [(dict(n_pages=0), 1), (dict(n_pages=2 ** 31), 1), (dict(D=96), 2), (dict(D=256), 2), (dict(k=None), 1),
            (dict(v_scale=None), 1), (dict(k_max=None), 1), (dict(k=A + 8), 2), (dict(k_min=A + 4), 2), (dict(k_scale=A + 2), 2)]


@pytest.mark.parametrize("kw,rc", BAD_POOL)
def test_bad_pools(lib, hnd, kw, rc):
    p, sh = _pool(**kw), _shape()
    assert lib.skv_q8_append(hnd, p, 2, 2, 1, 3, A, A, A, 4, A, None, None) == rc
    assert lib.skv_q8_attn(hnd, p, sh, A, A, 4, A, None, None, 0, None, 3, A, A, None) == rc
    assert lib.skv_q8_select(hnd, p, sh, A, A, 4, A, None, 4, 1, 1, A, None) == rc
    assert lib.skv_last_error(hnd)


def test_null_handle_and_pool(lib, hnd):
    p, sh = _pool(), _shape()
    assert lib.skv_q8_append(None, p, 2, 2, 1, 3, A, A, A, 4, A, None, None) == 1
    assert lib.skv_q8_attn(None, p, sh, A, A, 4, A, None, None, 0, None, 3, A, A, None) == 1
    assert lib.skv_q8_select(None, p, sh, A, A, 4, A, None, 4, 1, 1, A, None) == 1
    assert lib.skv_q8_evict(None, 1, 1, 4, A, A, A, 2, 1, 1, A, A, A, A, None) == 1
    assert lib.skv_q8_append(hnd, None, 2, 2, 1, 3, A, A, A, 4, A, None, None) == 1
    assert lib.skv_q8_attn(hnd, None, sh, A, A, 4, A, None, None, 0, None, 3, A, A, None) == 1
    assert lib.skv_q8_attn(hnd, p, None, A, A, 4, A, None, None, 0, None, 3, A, A, None) == 1


@pytest.mark.parametrize("i,val,rc", [(2, 0, 1), (3, 0, 1), (2, 65536, 2), (3, 70000, 2), (4, -1, 1), (5, 1, 1), (6, None, 1),
                                      (7, A + 8, 2), (8, None, 1), (9, 0, 1), (9, 1 << 26, 1), (10, None, 1)])
def test_append_arguments(lib, hnd, i, val, rc):
    args = [hnd, _pool(), 2, 2, 1, 3, A, A, A, 4, A, None, None]
    args[i] = val
    assert lib.skv_q8_append(*args) == rc


def test_append_of_nothing_is_fine(lib, hnd):
    assert lib.skv_q8_append(hnd, _pool(), 2, 2, 0, 3, None, None, A, 4, A, None, None) == 0


@pytest.mark.parametrize("kw,rc", [(dict(S=0), 1), (dict(nq=0), 1), (dict(H=9), 1), (dict(Hk=0), 1), (dict(D=64), 1),
                                   (dict(S=65536), 2), (dict(nq=2 ** 30, S=4), 2),
                                   (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1)])
def test_bad_shapes(lib, hnd, kw, rc):
    sh = _shape(**kw)
    assert lib.skv_q8_attn(hnd, _pool(), sh, A, A, 4, A, None, None, 0, None, 3, A, A, None) == rc
    assert lib.skv_q8_select(hnd, _pool(), sh, A, A, 4, A, None, 4, 1, 1, A, None) == rc


@pytest.mark.parametrize("i,val,rc", [(3, None, 1), (3, A + 2, 2), (4, None, 1), (5, 0, 1), (6, None, 1), (11, 1, 1), (12, None, 1),
                                      (12, A + 4, 2), (13, None, 1)])
def test_attn_arguments(lib, hnd, i, val, rc):
    args = [hnd, _pool(), _shape(), A, A, 4, A, None, None, 0, None, 3, A, A, None]
    args[i] = val
    assert lib.skv_q8_attn(*args) == rc


def test_attn_empty_selection(lib, hnd):
    assert lib.skv_q8_attn(hnd, _pool(), _shape(), A, A, 4, A, None, A, 0, None, 3, A, A, None) == 1


@pytest.mark.parametrize("n,first,last", [(0, 0, 0), (4, -1, 1), (4, 1, -1), (4, 3, 2), (2 ** 31 - 1, 2 ** 31 - 1, 1)])
def test_select_counts(lib, hnd, n, first, last):
    assert lib.skv_q8_select(hnd, _pool(), _shape(), A, A, 4, A, None, n, first, last, A, None) == 1
    assert lib.skv_q8_select(hnd, _pool(), _shape(), A, A, 4, A, None, 4, 1, 1, None, None) == 1


def test_evict_arguments(lib, hnd):
    n = 2 * 2 * 4 * 4
    b = [A + i * 4096 for i in range(7)]
    ok = [hnd, 2, 2, 4, b[0], b[1], b[2], 2, 1, 1, b[3], b[4], b[5], b[6], None]
    for i, val in ((1, 0), (2, 0), (3, 0), (4, None), (5, None), (6, None), (7, 0), (8, -1), (9, 0), (9, 2), (10, None), (11, None),
                   (12, None), (13, None), (10, b[0]), (11, b[1]), (10, b[1] + n - 4), (13, b[0] - n + 4), (11, b[3]), (13, b[3] + 4),
                   (12, b[2]), (12, b[3] + 8), (12, b[0])):
        args = list(ok)
        args[i] = val
        assert lib.skv_q8_evict(*args) == 1, (i, val)


def test_python_checks_tensors():
    import torch
    import split_kv_flash_attn_gb300 as skv
    with pytest.raises(skv.SplitKVError, match="k_min"):
        skv.Q8Pool(torch.zeros(4, 64, 128, dtype=torch.int8), torch.zeros(4, 64, 128, dtype=torch.int8), torch.zeros(4),
                   torch.zeros(4), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 128, dtype=torch.int8))
    with pytest.raises(skv.SplitKVError, match="non-contiguous"):
        skv.Q8Pool(torch.zeros(4, 64, 128, dtype=torch.int8), torch.zeros(64, 4, 128, dtype=torch.int8).transpose(0, 1),
                   torch.zeros(4), torch.zeros(4), torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4, 128, dtype=torch.int8))
    pool = skv.Q8Pool.empty(4, 128, device="cpu")

    class H:
        device = 0
    ids, n = torch.zeros(1, 2, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.float16)
    with pytest.raises(skv.SplitKVError, match="handle on cuda:0"):
        skv.q8_attn(H(), pool, q, ids, n)
    with pytest.raises(skv.SplitKVError, match="page_ids"):
        skv.q8_attn(H(), pool, q, ids.long(), n)
    with pytest.raises(skv.SplitKVError, match="kv_len"):
        skv.q8_attn(H(), pool, q, ids, n.long())
    with pytest.raises(skv.SplitKVError, match="q:"):
        skv.q8_attn(H(), pool, q.float(), ids, n)
    with pytest.raises(skv.SplitKVError, match="q_pos"):
        skv.q8_attn(H(), pool, q, ids, n, q_pos=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(skv.SplitKVError):
        skv.q8_append(H(), pool, q, q, ids, n)


def test_library_header_matches_binding(lib):
    from split_kv_flash_attn_gb300 import _lib
    import os
    txt = open(os.path.join(os.path.dirname(_lib.PKG), "include", "splitkv.h")).read()
    assert f"#define SKV_Q8_PAGE {_lib.Q8_PAGE}" in txt and f"#define SKV_F32 {_lib.F32} " in txt

"""Refusals of the calls for rows around attention and for gradients: each is found on the host before anything is
launched, so they are tested without a GPU, on a zeroed handle."""
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
F32, F16, BF16 = 3, 0, 4


def _spec(**kw):
    from split_kv_flash_attn_gb300 import _lib
    d = dict(D=128, rot_dims=128, interleaved=0, n_axes=1, freq=A, axis=None, factor=1.0, eps=1e-6)
    d.update(kw)
    return _lib.SkvRopeSpec(*d.values())


def _rope(lib, h, spec=None, **kw):
    d = dict(n=4, H=8, Hk=2, xt=F16, q=A, qs=1024, k=A, ks=256, qw=None, kw=None, pos=A, ot=F16, qo=A, ko=A, st=None)
    d.update(kw)
    return lib.skv_rope(h, spec if spec is not None else _spec(), *d.values())


def _dst(**kw):
    from split_kv_flash_attn_gb300 import _lib
    d = dict(type=0, row_bytes=512, dst0=None, n_rows0=0, dst1=None, n_rows1=0)
    d.update(kw)
    return _lib.SkvCacheDst(*d.values())


def _append(lib, h, spec=None, **kw):
    d = dict(n=4, H=8, Hk=2, xt=F16, q=A, qs=1024, k=A, ks=256, v=A, vs=256, qw=None, kw=None, pos=A, at=A, qo=A, kd=_dst(), vd=_dst(), st=None)
    d.update(kw)
    return lib.skv_rope_append(h, spec if spec is not None else _spec(), *d.values())


def _back(lib, h, spec=None, **kw):
    d = dict(n=4, H=8, Hk=2, xt=F16, q=A, qs=1024, k=A, ks=256, qw=None, kw=None, pos=A, gt=F16, gq=A, gk=A, dq=A, dqs=1024, dk=A, dks=256,
             dqw=None, dkw=None, st=None)
    d.update(kw)
    return lib.skv_rope_backward(h, spec if spec is not None else _spec(), *d.values())


SPECS = [(dict(D=96), 2), (dict(D=256), 2), (dict(rot_dims=-2), 1), (dict(rot_dims=130), 1), (dict(rot_dims=7), 1), (dict(rot_dims=36), 2),
         (dict(rot_dims=36, interleaved=1, freq=None), 1), (dict(n_axes=0), 1), (dict(n_axes=9), 1), (dict(freq=None), 1), (dict(freq=A + 2), 2),
         (dict(axis=A + 1), 2)]


@pytest.mark.parametrize("kw,rc", SPECS)
def test_bad_specs(lib, hnd, kw, rc):
    assert _rope(lib, hnd, _spec(**kw)) == rc
    assert _append(lib, hnd, _spec(**kw)) == rc
    assert _back(lib, hnd, _spec(**kw)) == rc
    assert lib.skv_last_error(hnd)


ROWS = [(dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(H=-1), 1), (dict(Hk=70000), 1), (dict(xt=1), 1), (dict(xt=9), 1), (dict(q=None), 1),
        (dict(k=None), 1), (dict(pos=None), 1), (dict(pos=A + 2), 2), (dict(q=A + 8), 2), (dict(qs=1000), 1), (dict(qs=1028), 2), (dict(ks=255), 1)]


@pytest.mark.parametrize("kw,rc", ROWS)
def test_bad_rows(lib, hnd, kw, rc):
    assert _rope(lib, hnd, **kw) == rc
    assert _append(lib, hnd, **kw) == rc
    if set(kw) & {"q", "qs", "k", "ks"}:                  # gradients read rows only where there is a weight
        kw = dict(kw, qw=A, kw=A, dqw=A, dkw=A)
    assert _back(lib, hnd, **kw) == rc


def test_results_weights_and_handles(lib, hnd):
    for kw, rc in [(dict(ot=2), 1), (dict(qo=None), 1), (dict(ko=A + 4), 2), (dict(qw=A + 4), 2), (dict(kw=A + 8), 2)]:
        assert _rope(lib, hnd, **kw) == rc
    for kw, rc in [(dict(gt=1), 1), (dict(gq=None), 1), (dict(gk=A + 8), 2), (dict(dq=None), 1), (dict(dqs=1023), 1), (dict(dks=260), 2),
                   (dict(qw=A), 1), (dict(dkw=A), 1), (dict(qw=A + 4, dqw=A), 2), (dict(kw=A, dkw=A + 2), 2)]:
        assert _back(lib, hnd, **kw) == rc
    assert _rope(lib, None) == _append(lib, None) == _back(lib, None) == 1
    assert _rope(lib, hnd, n=0) == 0 and _rope(lib, hnd, H=0, Hk=0) == 0
    assert lib.skv_rope(hnd, None, *([0] * 15)) == 1


def test_cache_destinations(lib, hnd):
    for kw, rc in [(dict(type=3), 1), (dict(type=-1), 1), (dict(row_bytes=511), 1), (dict(n_rows0=-1), 1), (dict(n_rows0=4), 1), (dict(n_rows1=4), 1),
                   (dict(row_bytes=514), 2), (dict(type=1, row_bytes=273), 2)]:
        assert _append(lib, hnd, kd=_dst(**kw)) == rc, kw
        assert _append(lib, hnd, vd=_dst(**kw)) == rc, kw
    assert _append(lib, hnd, kd=None) == 1 and _append(lib, hnd, vd=None) == 1
    assert _append(lib, hnd, at=None) == 1 and _append(lib, hnd, Hk=0) == 1 and _append(lib, hnd, v=None) == 1 and _append(lib, hnd, vs=100) == 1
    assert _append(lib, hnd, n=0) == 0


def _shape(**kw):
    from split_kv_flash_attn_gb300 import _lib
    d = dict(S=2, nq=16, H=8, Hk=2, D=128, scale=0.1, k_type=0, v_type=0, k_row_bytes=512, v_row_bytes=512)
    d.update(kw)
    return _lib.SkvShape(*d.values())


def _attn(lib, h, shape=None, **kw):
    d = dict(q=A, k=A, v=A, q_pos=None, pos0=0, rows=None, ld=0, per_head=0, lo=0, hi=100, o=A, lse=A, dt=F16, d_o=A, d_lse=None, gt=F16, dq=A, dk=A, dv=A,
             st=None)
    d.update(kw)
    return lib.skv_attn_backward(h, shape if shape is not None else _shape(), *d.values())


@pytest.mark.parametrize("kw,rc", [(dict(S=0), 1), (dict(nq=0), 1), (dict(H=0), 1), (dict(Hk=3), 1), (dict(D=80), 2), (dict(k_type=1), 2), (dict(v_type=2), 2),
                                   (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(k_row_bytes=510), 1), (dict(v_row_bytes=520), 2),
                                   (dict(k_row_bytes=1 << 39), 2), (dict(S=1 << 16, nq=1 << 15), 2)])
def test_bad_shapes(lib, hnd, kw, rc):
    assert _attn(lib, hnd, _shape(**kw)) == rc


@pytest.mark.parametrize("kw,rc", [(dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(d_o=None), 1),
                                   (dict(dk=None), 1), (dict(dv=None), 1), (dict(lo=-1), 1), (dict(lo=101), 1), (dict(rows=A, ld=99), 1), (dict(dt=1), 1),
                                   (dict(dt=BF16), 1), (dict(gt=BF16), 1), (dict(q=A + 8), 2), (dict(k=A + 8), 2), (dict(o=A + 4), 2), (dict(d_o=A + 2), 2),
                                   (dict(dq=A + 8), 2), (dict(dv=A + 4), 2), (dict(lse=A + 2), 2), (dict(d_lse=A + 1), 2), (dict(q_pos=A + 2), 2),
                                   (dict(rows=A + 2, ld=100), 2), (dict(hi=1 << 31), 2)])
def test_bad_gradient_arguments(lib, hnd, kw, rc):
    assert _attn(lib, hnd, **kw) == rc
    assert lib.skv_last_error(hnd)


def test_gradient_limits(lib, hnd):
    assert _attn(lib, None) == 1
    assert lib.skv_attn_backward(hnd, None, A, A, A, None, 0, None, 0, 0, 0, 100, A, A, F16, A, None, F16, A, A, A, None) == 1
    assert _attn(lib, hnd, dq=None, dk=None, dv=None) == 0           # nothing is asked for
    # a KV head's query tiles: 32768
    assert _attn(lib, hnd, _shape(S=1, nq=1 << 23, H=1, Hk=1, k_row_bytes=256, v_row_bytes=256)) == 2
    # a sequence's rows beyond a tensor map's strides
    assert _attn(lib, hnd, _shape(S=2, nq=1 << 20, H=4096, Hk=4096, k_row_bytes=1 << 20, v_row_bytes=1 << 20), rows=A, ld=100) == 2


def test_python_checks():
    """The Python layer's own checks, on CPU tensors (a handle and tensors must share a device)."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    f = torch.zeros(64)
    with pytest.raises(skv.SplitKVError):
        skv.Rope(128, f.double())
    with pytest.raises(skv.SplitKVError):
        skv.Rope(128, f.view(8, 8))
    with pytest.raises(skv.SplitKVError):
        skv.Rope(128, f, axis=torch.zeros(63, dtype=torch.int32))
    spec = skv.Rope(128, f, axis=torch.arange(64, dtype=torch.int32) % 3)
    assert spec.n_axes == 3 and spec.rot_dims == 128

    class Handle:
        device, _h, ptr = -1, None, None

        def check(self, rc):
            assert rc == 0

    h, x = Handle(), torch.zeros((5, 6, 128), dtype=torch.float16)
    pos = torch.zeros((3, 5), dtype=torch.int32)
    bad = [dict(q=x.long()), dict(q=x[:, :, :64]), dict(k=x.float()), dict(k=x[:4]), dict(pos=pos[:2]), dict(pos=pos.long()), dict(q=None, k=None),
           dict(q=x.transpose(0, 1)), dict(q_weight=f), dict(k_weight=torch.zeros(128, dtype=torch.float16)), dict(o_dtype=torch.int8)]
    for kw in bad:
        args = dict(q=x, k=x, pos=pos, stream=0)
        args.update(kw)
        with pytest.raises(skv.SplitKVError) as e:
            skv.rope(h, spec, args.pop("q"), args.pop("k"), args.pop("pos"), **args)
        assert e.value.status == 1, kw
    # a packed projection's parts, [S, n, heads, D]: one stride for all tokens
    y = torch.zeros((2, 5, 9, 128), dtype=torch.float16)
    assert skv._token_rows("q", y[:, :, :4], (2, 5), 128, torch.float16, -1) == (4, 9 * 128)
    assert skv._token_rows("q", y[:1, :, :4], (1, 5), 128, torch.float16, -1) == (4, 9 * 128)
    assert skv._token_rows("q", y[:, :1, 3:], (2, 1), 128, torch.float16, -1) == (6, 5 * 9 * 128)
    with pytest.raises(skv.SplitKVError):
        skv._token_rows("q", y[:, :4, :4], (2, 4), 128, torch.float16, -1)
    with pytest.raises(skv.SplitKVError):
        skv._token_rows("q", y[:, :, ::2], (2, 5), 128, torch.float16, -1)


def test_python_checks_of_gradients(monkeypatch):
    """What k and v must hold for the heads and the range that the call names."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    from split_kv_flash_attn_gb300 import _lib

    class Handle:
        device, _h, ptr = -1, None, None

        def check(self, rc):
            assert rc == 0

    class Lib:
        def skv_attn_backward(self, *a):
            return 0

    monkeypatch.setattr(_lib, "lib", lambda: Lib())
    q = torch.zeros((1, 4, 8, 64), dtype=torch.float16)
    kv = torch.zeros((10, 2, 64), dtype=torch.float16)
    o, lse = torch.zeros((1, 4, 8, 64)), torch.zeros((1, 4, 8))

    def call(k=kv, v=kv, Hk=2, **kw):
        return skv.attn_backward(Handle(), q, k, v, o, lse, q, Hk=Hk, stream=0, need_dq=False, need_dkv=False, **kw)

    wide = torch.zeros((10, 6, 64), dtype=torch.float16)
    rows = torch.zeros((1, 7), dtype=torch.int32)
    call(), call(kv_begin=3, kv_end=9), call(kv_rows=rows), call(wide[:, :2], wide[:, 2:4], k_row_bytes=768, v_row_bytes=768)
    call(wide[:, 4:], wide[:, 2:4], k_row_bytes=768, v_row_bytes=768)            # ends with the storage
    bad = [dict(Hk=8), dict(Hk=1), dict(Hk=4, kv_rows=rows), dict(v=kv[:, :1].contiguous()), dict(k=kv[:8]), dict(kv_end=11),
           dict(k=wide[:, :2]), dict(k_row_bytes=272), dict(v_row_bytes=512), dict(k=wide[:, 4:], k_row_bytes=784)]
    for kw in bad:
        with pytest.raises(skv.SplitKVError) as e:
            call(**kw)
        assert e.value.status == 1, kw

"""Sizes that the calls over 8-bit pages refuse, found on the host before anything is launched:
tested without a GPU, on a zeroed handle."""
import math

import pytest

from test_q8_host import A, _pool, _shape, hnd, lib  # noqa: F401


@pytest.mark.parametrize("n", [2 ** 30, 2 ** 31 - 1])
def test_selections_whose_entries_outgrow_32_bits(lib, hnd, n):  # noqa: F811
    """A loop over n entries in steps of a CTA's threads would pass 2^31 and go on below zero."""
    assert lib.skv_q8_select(hnd, _pool(), _shape(), A, A, 4, A, None, n, 1, 1, A, None) == 2
    assert lib.skv_q8_attn(hnd, _pool(), _shape(), A, A, 4, A, None, A, n, None, 3, A, A, None) == 2
    assert b"n_sel" in lib.skv_last_error(hnd)


def test_more_lists_and_heads_than_a_launch_has(lib, hnd):  # noqa: F811
    """Refused before their page weights' scratch is counted: its size, 2^64 bytes here, was zero in
    64 bits, by which the call divided."""
    sh = _shape(S=2 ** 14, Hk=2 ** 14, H=2 ** 30)
    assert lib.skv_q8_attn(hnd, _pool(), sh, A, A, 2 ** 17, A, None, None, 0, A, 3, A, A, None) == 2
    assert lib.skv_q8_attn(hnd, _pool(), sh, A, A, 4, A, None, A, 2 ** 17, A, 3, A, A, None) == 2
    assert b"too many" in lib.skv_last_error(hnd)


VISITS = 2 ** 32 - 2 ** 16


@pytest.mark.parametrize("S,nq,H,Hk,n", [(1, 8191, 128, 1, 16400), (1, 8191, 128, 1, 2 ** 21), (4, 100, 32, 8, 2 ** 29 + 1),
                                         (1, 9, 1024, 1, 2 ** 25), (1, 1, 4, 1, 5), (3, 70000, 8, 8, 64)])
def test_page_visits_of_a_launch(lib, S, nq, H, Hk, n):  # noqa: F811
    """A launch's line of page visits is counted in 32 bits: a call goes in as many launches as that takes."""
    import split_kv_flash_attn_gb300 as skv
    G = H // Hk
    groups = math.ceil(G / (8 if G <= 8 else 16))
    one = S * Hk * groups
    want = min(nq, 65535 // one, VISITS // (one * n))
    if want == 0:
        with pytest.raises(skv.SplitKVError):
            skv.plan_q8_tokens(S, nq, H, Hk, 2 ** 20, n_sel=n)
        return
    assert skv.plan_q8_tokens(S, nq, H, Hk, 2 ** 20, n_sel=n) == want
    # with page weights: 256 MiB of log sums, or one token's
    most = max(1, 2 ** 28 // (S * H * n * 8))
    assert skv.plan_q8_tokens(S, nq, H, Hk, 2 ** 20, n_sel=n, mass=True) == min(want, most)


def test_page_visits_of_whole_lists(lib):  # noqa: F811
    import split_kv_flash_attn_gb300 as skv
    assert skv.plan_q8_tokens(2, 32, 8, 8, 1000) == 32
    assert skv.plan_q8_tokens(2, 32, 8, 8, 2 ** 25 - 1) == 32           # 2^30 visits twice
    assert skv.plan_q8_tokens(10, 32, 8, 8, 2 ** 25 - 1) == 16          # one row group a launch
    with pytest.raises(skv.SplitKVError):
        skv.plan_q8_tokens(17, 1, 8, 8, 2 ** 25 - 1)
    assert skv.plan_q8_tokens(2, 5000, 8, 8, 2 ** 20) == 5000
    assert skv.plan_q8_tokens(1, 2 ** 20, 1, 1, 2 ** 20) == 2 ** 20     # tensor cores: 2^12 pairs of tiles of 2^19
    assert skv.plan_q8_tokens(1, 2 ** 21, 1, 1, 2 ** 20) == 2 ** 20


def test_a_token_of_too_many_page_visits(lib, hnd):  # noqa: F811
    """64 row groups of 1024 heads for each of four lists: 2^33 visits of one token."""
    sh = _shape(S=2, Hk=2, H=2048)
    assert lib.skv_q8_attn(hnd, _pool(), sh, A, A, 4, A, None, A, 2 ** 25, None, 3, A, A, None) == 2
    assert b"too many" in lib.skv_last_error(hnd)

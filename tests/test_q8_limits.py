"""Sizes that the calls over 8-bit pages refuse, found on the host before anything is launched:
tested without a GPU, on a zeroed handle."""
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

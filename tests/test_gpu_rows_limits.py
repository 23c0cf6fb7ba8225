"""Gradients of attention at the largest number of query rows that a call takes."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,nq,H", [(1, 1 << 22, 1), (2, 1 << 18, 8)])
def test_as_many_query_tiles_as_a_kv_head_may_have(S, nq, H):
    """2^22 rows over 70 keys against the formulas, with the derived bounds (grad_util: sums over rows are emptied every 128
    tiles; 256 such sums are added in fp32, 2^-24 of the magnitudes each, within its 1024 steps)."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import split_kv_flash_attn_gb300 as skv
    from tests.grad_util import attention_backward, attention_forward, check
    n, D, T = 70, 64, S * nq
    h = skv.Handle(0)
    g = torch.Generator(device="cuda")
    g.manual_seed(nq)
    q, d_o = (torch.randn((S, nq, H, D), device="cuda", generator=g).half() for _ in "ab")
    k, v = (torch.randn((n, 1, D), device="cuda", generator=g).half() for _ in "ab")
    see = torch.ones((1, T, n), dtype=torch.bool, device="cuda")
    q1, d1 = q.view(1, T, H, D), d_o.view(1, T, H, D)
    o, lse = (torch.cat(x, 2) for x in zip(*(attention_forward(q1[:, :, i:i + 1], k[None], v[None], see, D ** -0.5) for i in range(H))))
    got = skv.attn_backward(h, q, k, v, o.view(S, nq, H, D), lse.view(S, nq, H), d_o, Hk=1)
    assert h.status() == 0
    dk, dv, bk, bv = (torch.zeros((n, 1, D), dtype=torch.float64, device="cuda") for _ in "abcd")
    for i in range(H):                                       # a head at a time: the formulas' matrices are large
        one = slice(i, i + 1)
        want, bound = attention_backward(q1[:, :, one], k[None], v[None], see, D ** -0.5, o[:, :, one], lse[:, :, one], d1[:, :, one])
        check(got[0].view(1, T, H, D)[:, :, one], want[0], bound[0], "dq")
        for sums, x in ((dk, want[1]), (dv, want[2]), (bk, bound[1]), (bv, bound[2])):
            sums += x[0]
    check(got[1], dk, bk, "dk")
    check(got[2], dv, bv, "dv")
    h.close()

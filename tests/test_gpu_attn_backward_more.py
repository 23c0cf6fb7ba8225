"""Gradients of attention: differences of the forward call itself, and the rounding that dq gives back."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import split_kv_flash_attn_gb300 as m
    return m


@pytest.fixture(scope="module")
def h(skv):
    return skv.Handle(0)


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _forward64(q, k, v, see, scale):
    """p [H, T, n], o [T, H, D], lse [T, H] in 64 bits of q [T, H, D] over k, v [n, Hk, D]."""
    import torch
    G = q.shape[1] // k.shape[1]
    s = torch.einsum("thd,nhd->htn", q.double(), k.double().repeat_interleave(G, 1)) * scale
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.unsqueeze(-1))
    return p, torch.einsum("htn,nhd->thd", p, v.double().repeat_interleave(G, 1)), lse.t()


@pytest.mark.parametrize("nq,n,H,Hk,D,lists", [(64, 160, 4, 2, 128, False), (64, 160, 4, 2, 128, True), (1, 160, 8, 1, 64, False), (33, 90, 6, 2, 64, False)])
def test_against_differences_of_the_forward_call(skv, h, nq, n, H, Hk, D, lists):
    """(f(x + t z) - f(x - t z)) / 2t of f = sum(o w) + sum(lse u), o and lse from attn_partial, beside sum(gradient z), z the
    gradient's signs (so that all values count with their sizes and errors add up against them, at worst).  Values are
    multiples of 2^-6 below 2 and t = 2^-3, so that x +- t z are fp16 numbers.
    Room: the forward call rounds its weights to fp16: 2^-11 sum |w| p |v| for f, an eighth more for its fp32 sums (2^-14),
    2^-16 of |u| for lse (fp32 sums of scores below 2^6, logarithms), both points: over t; the difference's own error as
    64 bits have it; and the bounds of the gradient's values."""
    import torch
    from tests.grad_util import attention_backward
    g = _gen(nq + n)

    def grid(*s):
        return (torch.randint(-96, 97, s, device="cuda", generator=g) / 64.0).half()

    q, k, v = grid(nq, H, D), grid(n, Hk, D), grid(n, Hk, D)
    w = (torch.randint(-64, 65, (nq, H, D), device="cuda", generator=g) / 64.0).float()
    u = torch.randn((nq, H), device="cuda", generator=g)
    pos = (torch.arange(nq, device="cuda") + n - nq).view(1, nq).to(torch.int32)
    see = torch.arange(n, device="cuda").view(1, n) <= pos.view(nq, 1)
    scale, t = D ** -0.5, 2.0 ** -3
    rows = torch.arange(n, device="cuda", dtype=torch.int32).view(1, n) if lists else None

    def call(q, k, v):
        return skv.attn_partial(h, q.view(1, nq, H, D), k, v, Hk=Hk, q_pos=pos, kv_rows=rows)

    def value(o, lse):
        return float((o.double().view(nq, H, D) * w.double()).sum() + (lse.double().view(nq, H) * u.double()).sum())

    o, lse = call(q, k, v)
    got = skv.attn_backward(h, q.view(1, nq, H, D), k, v, o, lse, w.view(1, nq, H, D), Hk=Hk, q_pos=pos, d_lse=u.view(1, nq, H), kv_rows=rows)
    assert h.status() == 0
    p = _forward64(q, k, v, see, scale)[0]
    forward = float((w.double().abs() * torch.einsum("htn,nhd->thd", p, v.double().abs().repeat_interleave(H // Hk, 1))).sum()) * 2.0 ** -11 * 1.125
    forward += float(u.abs().sum()) * 2.0 ** -16
    bounds = attention_backward(q[None], k[None], v[None], see[None], scale, o, lse, w[None], u[None])[1]
    for i, x in enumerate((q, k, v)):
        mine = got[i].double().view(x.shape)
        z = mine.sign()
        ends = []
        for sign in (1, -1):
            a = [q, k, v]
            a[i] = (x.double() + sign * t * z).half()
            assert torch.equal(a[i].double(), x.double() + sign * t * z)
            ends.append((value(*call(*a)), value(*_forward64(*a, see, scale)[1:])))
        slope, exact = ((ends[0][j] - ends[1][j]) / (2 * t) for j in (0, 1))
        j = [q.double().requires_grad_(), k.double().requires_grad_(), v.double().requires_grad_()]
        _, o64, l64 = _forward64(*j, see, scale)
        true = float((torch.autograd.grad((o64 * w.double()).sum() + (l64 * u.double()).sum(), j)[i] * z).sum())
        room = forward / t + abs(exact - true) + float(bounds[i].sum())
        mine = float((mine * z).sum())
        assert room < 0.2 * abs(true), (i, room, true)       # (a factor or a sign would show)
        assert abs(slope - mine) <= room, (i, slope, mine, room)


@pytest.mark.parametrize("D,common,noise,amp", [(64, 8.0, 0.1, 0.05), (128, 16.0, 0.25, 0.02)])
def test_what_rounding_takes_from_common_keys_is_given_back(skv, h, D, common, noise, amp):
    """Keys that differ little from a large vector m that they have in common: dq = scale sum ds_k (K_k - m) is small beside
    what rounding ds takes, sum eps_k m, unless that is given back.  128 keys, so that the mean given back is theirs.
    Bound of a value: |eps_k| |K_k - mean| with |eps_k| at most 2^-11 |ds_k| or 2^-37 of the scale; the fp32 errors of p and
    d_o.v - delta (2^-20 of the sums of magnitudes: 8 truncated steps of 2^-23, and a tree of 8) times |K_k|; sums of n / 16
    steps; what is given back in fp32 (2^-14 of it).  The plain rounding, computed here, lies outside."""
    import torch
    nq, n = 200, 128
    g = _gen(D)
    q = (torch.randn((nq, D), device="cuda", generator=g) * amp).half()
    k = (torch.randn((1, D), device="cuda", generator=g).sign() * common + torch.randn((n, D), device="cuda", generator=g) * noise).half()
    v = torch.randn((n, D), device="cuda", generator=g).half()
    d_o = (torch.randn((nq, D), device="cuda", generator=g) * 0.1).half()
    scale = D ** -0.5
    qd, kd, vd, dd = (x.double() for x in (q, k, v, d_o))
    s = qd @ kd.t() * scale
    lse = torch.logsumexp(s, -1).float()
    p = torch.exp(s - lse.double().unsqueeze(1))
    o = (p @ vd).float()
    dp, delta = dd @ vd.t(), (dd * o.double()).sum(1, keepdim=True)
    ds = p * (dp - delta)
    want, mean = ds @ kd * scale, kd.mean(0)
    shape = (1, nq, 1, D)
    got = skv.attn_backward(h, q.view(shape), k.view(n, 1, D), v.view(n, 1, D), o.view(shape), lse.view(1, nq, 1), d_o.view(shape), Hk=1,
                            need_dkv=False)[0].view(nq, D).double()
    assert h.status() == 0
    size = torch.linalg.vector_norm(dd, dim=1, keepdim=True) * torch.linalg.vector_norm(vd, dim=1).max() + delta.abs()
    eps = ds.abs() * 2.0 ** -11 + size * 2.0 ** -37
    sizes = dd.abs() @ vd.abs().t() + (dd * o.double()).abs().sum(1, keepdim=True)
    ep = (qd.abs() @ kd.abs().t() * scale) * (D / 16) * 2.0 ** -23 + (s.abs() + lse.double().abs().unsqueeze(1)) * 2.0 ** -22 + 2.0 ** -21
    fp32 = ds.abs() * (ep + n / 16 * 2.0 ** -24) + p * sizes * 2.0 ** -20
    bound = (torch.einsum("qk,kd->qd", eps, (kd - mean).abs()) + fp32 @ kd.abs() + eps.sum(1, keepdim=True) * mean.abs() * 2.0 ** -14) * scale
    bound = bound + want.abs() * 2.0 ** -24
    power = torch.exp2(15 - torch.ceil(torch.log2(size)))
    plain = (ds * power).half().double() / power @ kd * scale
    assert float(((plain - want).abs() / bound).max()) > 1.5
    off = ((got - want).abs() / bound).max()
    assert float(off) <= 1, float(off)
    # in the 2-norm: eps_k of random signs, at most 2^-11 |ds_k| each, 2^-11 |ds|_2 (K - mean) for a row; 4 of it leave room
    rms = (kd - mean).square().mean(0).sqrt()
    row = torch.linalg.vector_norm(ds, dim=1, keepdim=True) * rms * scale
    assert float((got - want).norm()) <= 4 * 2.0 ** -11 * float(row.norm())
    assert float((plain - want).norm()) > 4 * 2.0 ** -11 * float(row.norm())


PARTS = [
    # S, nq, n, H, Hk, D, causal, lists; what has two parts
    (1, 64, 256, 4, 1, 64, True, False, "all"),
    (1, 4, 21, 8, 2, 64, False, False, "all"),
    (1, 30, 1126, 8, 8, 128, True, False, "all"),
    (1, 300, 300, 4, 2, 128, True, False, "all"),
    (3, 70, 150, 6, 2, 128, True, True, "all"),
    (2, 500, 60, 5, 1, 64, False, True, "all"),
    (1, 1, 1, 4, 4, 128, False, False, "all"),
    (1, 512, 2048, 8, 2, 128, True, False, "dq"),         # 512 tiles
    (3, 200, 520, 16, 4, 64, False, True, "dq"),          # 420 of lists
    (1, 3, 30000, 8, 8, 128, True, False, "dq"),          # 1880 tiles, one of query rows for each KV head
    (1, 16, 21000, 64, 8, 64, False, False, "dq"),        # 128 rows of it
]


@pytest.mark.parametrize("S,nq,n,H,Hk,D,causal,lists,parts", PARTS)
def test_small_calls_hold_more_bits(skv, h, S, nq, n, H, Hk, D, causal, lists, parts):
    """p and ds of two fp16 parts leave their fp32 errors: of p at most 2^-15 (scores' sums of 16 magnitudes 2^-23, 8 steps;
    exponents below 64, 2^-22), of d_o.v - delta 2^-19 of some 10 times its size, in sums whose terms and errors are of
    random sign: 2^-14 of a result's 2-norm (one part would leave 2^-12)."""
    import torch
    from tests.grad_util import attention_backward, attention_forward, check
    g = _gen(n + nq)
    q = torch.randn((S, nq, H, D), device="cuda", generator=g).half()
    r = S * n if lists else n
    k = (torch.randn((r, Hk, D), device="cuda", generator=g) + 0.5 * torch.randn((1, Hk, D), device="cuda", generator=g)).half()
    v = torch.randn((r, Hk, D), device="cuda", generator=g).half()
    d_o = (torch.randn((S, nq, H, D), device="cuda", generator=g) * 0.1).half()
    rows = torch.arange(r, device="cuda", dtype=torch.int32).view(S, n) if lists else None
    pos = (n - nq + torch.arange(nq, device="cuda")).repeat(S, 1).to(torch.int32) if causal else None
    B, T = (S, nq) if lists else (1, S * nq)
    see = torch.ones((B, T, n), dtype=torch.bool, device="cuda")
    if causal:
        see = torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(B, T, 1)
    q1, d1, k1, v1 = q.view(B, T, H, D), d_o.view(B, T, H, D), k.view(B, n, Hk, D), v.view(B, n, Hk, D)
    o, lse = attention_forward(q1, k1, v1, see, D ** -0.5)
    want, bound = attention_backward(q1, k1, v1, see, D ** -0.5, o, lse, d1)
    got = skv.attn_backward(h, q, k, v, o.view(S, nq, H, D), lse.view(S, nq, H), d_o, Hk=Hk, q_pos=pos, kv_rows=rows)
    assert h.status() == 0
    for name, x, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        w, b = w.reshape(x.shape), b.reshape(x.shape)
        check(x, w, b, name)
        if (parts == "all" or name == "dq") and (n > 1 or name == "dv"):      # (one key: dq and dk are 0 but for delta's rounding)
            assert float((x.double() - w).norm()) <= 2.0 ** -14 * float(w.norm()), name

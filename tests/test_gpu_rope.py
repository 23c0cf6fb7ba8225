"""Norm and rotation of queries and keys, the same into cache rows, and the gradients, against 64 bits.

Bounds.  A rotated value is f (a cos - b sin) of normed a, b: the norm's sum of D squares in fp32 (a tree of at most 8
serial steps and 4 levels), one rsqrt (2^-22) and two products leave 2^-20 of |a|; cos and sin are good to 2^-23 and
the products and the sum add 2^-22: 2^-19 of |f| (|a| + |b|) leaves room for all; then half a step of the type.  Gradients of a
normed row add two sums of D products: 2^-18 of their magnitudes.  Weights' gradients are fp32 sums of N products
in runs of at most N / 64 + 1000 ones: bounded by (N / 64 + 1000) 2^-24 of the sum of magnitudes, far above what sums of random
sign give.
"""
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


def _case(n, H, Hk, D, R, axes, dtype, far, seed=0, interleaved=False):
    import torch
    g = _gen(seed * 31 + n + D)
    x = (torch.randn((n, H + 2 * Hk, D), device="cuda", generator=g) * 3).to(dtype)
    pos = torch.randint(0, far + 1, (axes, n), device="cuda", generator=g).to(torch.int32)
    half = R // 2
    freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))).float()
    axis = torch.randint(0, axes, (half,), device="cuda", generator=g).to(torch.int32)
    w = [1 + 0.3 * torch.randn(D, device="cuda", generator=g) for _ in "qk"]
    return x, pos, freq, axis, w


def _spec(skv, D, freq, axis, axes, interleaved, **kw):
    return skv.Rope(D, freq, axis=axis if axes > 1 else None, n_axes=axes, interleaved=interleaved, **kw)


def _near(got, want, mags, what):
    from tests.grad_util import check
    check(got, want, mags, what)


def _turn_bound(x, w, pos, freq, axis, inter, factor):
    """2^-19 of |f| (|a| + |b|) for pairs, of |y| for what passes."""
    import torch
    from tests.grad_util import rope_forward
    x = x.double()
    y = x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    R = 2 * freq.numel()
    i = torch.arange(R // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    m = y.abs().clone()
    m[..., a] = m[..., b] = abs(factor) * (y[..., a].abs() + y[..., b].abs())
    return rope_forward(x, w, pos, freq, axis, inter, factor), m * 2.0 ** -19


CASES = [
    # n, H, Hk, D, R, axes, norm, interleaved, far
    (1, 4, 1, 64, 64, 1, False, False, 4095),
    (1, 32, 8, 128, 128, 1, True, False, 1 << 20),
    (7, 5, 1, 128, 64, 1, True, True, 100),
    (33, 1, 0, 128, 128, 1, True, False, 2 ** 31 - 1),      # queries alone, the farthest positions
    (130, 0, 1, 64, 32, 2, False, True, 1000),              # keys alone
    (257, 16, 16, 64, 64, 3, True, True, 200),
    (100, 3, 2, 64, 16, 4, True, False, 50),
    (65, 8, 2, 128, 0, 1, True, False, 10),                 # no rotation
    (40, 2, 2, 64, 38, 1, False, True, 65536),              # an odd number of pairs
    (1000, 24, 8, 128, 96, 1, False, False, 131072),
]


@pytest.mark.parametrize("xt,ot", [("float16", "float16"), ("bfloat16", "float32"), ("float32", "float16"), ("float32", "bfloat16")])
@pytest.mark.parametrize("n,H,Hk,D,R,axes,norm,inter,far", CASES)
def test_rope(skv, h, n, H, Hk, D, R, axes, norm, inter, far, xt, ot):
    import torch
    x, pos, freq, axis, w = _case(n, H, Hk, D, R, axes, getattr(torch, xt), far)
    spec = _spec(skv, D, freq, axis, axes, inter, factor=1.25)
    ws = w if norm else [None, None]
    q, k = x[:, :H] if H else None, x[:, H:H + Hk] if Hk else None
    got = skv.rope(h, spec, q, k, pos, q_weight=ws[0] if H else None, k_weight=ws[1] if Hk else None, o_dtype=getattr(torch, ot))
    assert h.status() == 0
    for name, a, b, wt in (("q", q, got[0], ws[0]), ("k", k, got[1], ws[1])):
        if a is None:
            assert b is None
            continue
        want, bound = _turn_bound(a, wt, pos, freq, axis if axes > 1 else axis * 0, inter, 1.25)
        _near(b, want, bound, name)


@pytest.mark.parametrize("gt,xt", [("float16", "float16"), ("float32", "float32"), ("bfloat16", "bfloat16"), ("float32", "float16")])
@pytest.mark.parametrize("n,H,Hk,D,R,axes,norm,inter,far", CASES)
def test_rope_backward(skv, h, n, H, Hk, D, R, axes, norm, inter, far, gt, xt):
    import torch
    from tests.grad_util import check, rope_forward
    x, pos, freq, axis, w = _case(n, H, Hk, D, R, axes, getattr(torch, xt), far, seed=1)
    spec = _spec(skv, D, freq, axis, axes, inter, factor=0.75)
    ws = w if norm else [None, None]
    g = _gen(3)
    dy = [(torch.randn((n, m, D), device="cuda", generator=g) * 0.1).to(getattr(torch, gt)) for m in (H, Hk)]
    q, k = x[:, :H] if H else None, x[:, H:H + Hk] if Hk else None
    got = skv.rope_backward(h, spec, dy[0] if H else None, dy[1] if Hk else None, pos, q=q if norm else None, k=k if norm else None,
                            q_weight=ws[0] if H else None, k_weight=ws[1] if Hk else None, x_dtype=getattr(torch, xt))
    assert h.status() == 0
    ax = axis if axes > 1 else axis * 0
    for i, (a, d, wt) in enumerate(((q, dy[0], ws[0]), (k, dy[1], ws[1]))):
        if a is None:
            assert got[i] is None and got[2 + i] is None
            continue
        xa = a.double().requires_grad_()
        wa = None if wt is None else wt.double().requires_grad_()
        y = rope_forward(xa, wa, pos, freq, ax, inter, 0.75)
        grads = torch.autograd.grad(y, [xa] if wa is None else [xa, wa], d.double())
        # |u| as large as a pair's two gradients together; r (|u| + |x r| mean |u x r|)
        half = R // 2
        j = torch.arange(half, device="cuda")
        ia, ib = (2 * j, 2 * j + 1) if inter else (j, j + half)
        m = d.double().abs().clone()
        m[..., ia] = m[..., ib] = 0.75 * (d.double()[..., ia].abs() + d.double()[..., ib].abs())
        if wt is None:
            check(got[i], grads[0], m * 2.0 ** -19, "dx")
            assert got[2 + i] is None
            continue
        r = 1 / torch.sqrt(a.double().square().mean(-1, keepdim=True) + 1e-6)
        xr = a.double().abs() * r
        u = m * wt.double().abs()
        check(got[i], grads[0], r * (u + xr * (u * xr).mean(-1, keepdim=True)) * 2.0 ** -18, "dx")
        N = n * a.shape[1]
        check(got[2 + i], grads[1], (m * xr).sum((0, 1)) * ((N / 64 + 1000) * 2.0 ** -24), "dw")


def test_packed_rows_padding_and_given_results(skv, h):
    """Rows of a packed projection [S, n, heads, D]; gradients into a packed one; padding tokens hold NaN."""
    import torch
    from tests.grad_util import check
    S, n, H, Hk, D = 2, 37, 4, 2, 128
    x, pos, freq, axis, w = _case(S * n, H, Hk, D, 128, 1, torch.float16, 5000)
    pad = torch.zeros(S * n, dtype=torch.bool, device="cuda")
    pad[30:37] = pad[70:] = True
    pos[0, pad] = -1
    x[pad] = math.nan
    x = x.view(S, n, H + 2 * Hk, D)
    spec = skv.Rope(D, freq)
    q, k = x[:, :, :H], x[:, :, H:H + Hk]
    out = skv.rope(h, spec, q, k, pos.view(S, n), q_weight=w[0], k_weight=w[1])
    for a, b, wt in ((q, out[0], w[0]), (k, out[1], w[1])):
        assert b.shape == a.shape
        flat, res = a.reshape(S * n, -1, D), b.reshape(S * n, -1, D)
        assert (res[pad] == 0).all()
        want, bound = _turn_bound(flat[~pad], wt, pos[:, ~pad], freq, axis * 0, False, 1.0)
        check(res[~pad], want, bound, "packed")
    g = _gen(1)
    dq = torch.randn((S, n, H, D), device="cuda", generator=g).half()
    dk = torch.randn((S, n, Hk, D), device="cuda", generator=g).half()
    dq.view(S * n, H, D)[pad] = math.nan
    dk.view(S * n, Hk, D)[pad] = math.inf
    packed = torch.full((S, n, H + 2 * Hk, D), 7.0, dtype=torch.float16, device="cuda")
    a = skv.rope_backward(h, spec, dq, dk, pos, q=q, k=k, q_weight=w[0], k_weight=w[1], dq=packed[:, :, :H], dk=packed[:, :, H:H + Hk])
    b = skv.rope_backward(h, spec, dq, dk, pos, q=q.contiguous(), k=k.contiguous(), q_weight=w[0], k_weight=w[1])
    for u, v in zip(a, b):
        assert torch.equal(u, v) and torch.isfinite(v).all()
    assert (packed[:, :, H + Hk:] == 7).all()
    assert (b[0].view(S * n, H, D)[pad] == 0).all() and (b[1].view(S * n, Hk, D)[pad] == 0).all()
    live = [t.reshape(S * n, -1, D)[~pad].contiguous() for t in (dq, dk, q, k)]
    c = skv.rope_backward(h, spec, live[0], live[1], pos[:, ~pad].contiguous(), q=live[2], k=live[3], q_weight=w[0], k_weight=w[1])
    assert torch.equal(c[0], b[0].view(S * n, H, D)[~pad])
    # the sums run over the same rows in another order
    assert torch.allclose(c[2], b[2], rtol=1e-4, atol=1e-3) and torch.allclose(c[3], b[3], rtol=1e-4, atol=1e-3)
    assert h.status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kt,vt", [("F16", "F16"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0"), ("Q8_0", "Q8_0")])
@pytest.mark.parametrize("n,H", [(1, 4), (45, 6), (300, 0)])
def test_append_stores_what_rope_and_kv_append_store(skv, h, D, kt, vt, n, H):
    """The same bytes as rope (fp32 results) followed by kv_append, in a window and a pinned tail; rows of no token and
    of padding keep theirs."""
    import torch
    Hk, rows0, rows1 = 2, 200, 250
    x, pos, freq, axis, w = _case(n, H, Hk, D, D, 1, torch.float32, 9999, seed=4)
    g = _gen(8)
    at = torch.randperm(rows0 + rows1, device="cuda", generator=g)[:n].to(torch.int32)
    if n > 40:
        at[3], pos[0, 5] = -1, -7
    q, k, v = x[:, :H] if H else None, x[:, H:H + Hk], x[:, H + Hk:]
    spec = skv.Rope(D, freq)
    kt, vt = getattr(skv, kt), getattr(skv, vt)

    def caches():
        out = []
        for t in (kt, vt):
            b = Hk * skv.segment_bytes(t, D)
            out += [torch.full((rows0, b), 0x5a, dtype=torch.uint8, device="cuda"), torch.full((rows1, b), 0x5a, dtype=torch.uint8).pin_memory()]
        return out

    a, b = caches(), caches()
    got_q = skv.rope_append(h, spec, q, k, v, pos, at, a[0], a[2], a[1], a[3], q_weight=w[0] if H else None, k_weight=w[1], k_type=kt, v_type=vt)
    yq, yk = skv.rope(h, spec, q, k, pos, q_weight=w[0] if H else None, k_weight=w[1], o_dtype=torch.float32)
    at2 = torch.where(pos[0] < 0, -1, at).to(torch.int32)
    skv.kv_append(h, yk, at2, b[0], b[1], type_=kt)
    skv.kv_append(h, v.contiguous(), at2, b[2], b[3], type_=vt)
    assert h.status() == 0
    for s, t in zip(a, b):
        assert torch.equal(s.cpu(), t.cpu())
    if H:
        assert torch.equal(got_q, yq.half())
    else:
        assert got_q is None
    assert (a[0] != 0x5a).any() or (a[1] != 0x5a).any()


def test_append_beyond_the_cache_sets_the_status_bit(skv, h):
    import torch
    x, pos, freq, axis, w = _case(4, 2, 1, 64, 64, 1, torch.float16, 10)
    K = torch.zeros((3, 128), dtype=torch.uint8, device="cuda")
    V = K.clone()
    at = torch.tensor([0, 3, 2, -5], dtype=torch.int32, device="cuda")
    skv.rope_append(h, skv.Rope(64, freq), x[:, :2], x[:, 2:3], x[:, 3:], pos, at, K, V)
    with pytest.raises(skv.SplitKVError) as e:
        h.status()
    assert e.value.status == 8
    assert (K[0] != 0).any() and (K[1] == 0).all() and (K[2] != 0).any()
    assert h.status() == 0


def test_values_that_are_not_finite_stay_in_their_rows(skv, h):
    import torch
    x, pos, freq, axis, w = _case(9, 2, 1, 128, 128, 1, torch.float16, 100)
    y = x.clone()
    y[4, 1, 7], y[6, 2, 0] = math.nan, math.inf
    spec = skv.Rope(128, freq)
    a = skv.rope(h, spec, x[:, :2], x[:, 2:3], pos, q_weight=w[0], k_weight=w[1])
    b = skv.rope(h, spec, y[:, :2], y[:, 2:3], pos, q_weight=w[0], k_weight=w[1])
    same = [torch.ones(t.shape[:2], dtype=torch.bool, device="cuda") for t in a]
    same[0][4, 1], same[1][6, 0] = False, False
    for s, u, v in zip(same, a, b):
        assert torch.equal(u[s], v[s]) and torch.isnan(v[~s]).any()


def test_graph_stream_and_repeats(skv):
    import torch
    h = skv.Handle(0)
    x, pos, freq, axis, w = _case(500, 8, 2, 128, 128, 1, torch.float16, 100)
    spec, side = skv.Rope(128, freq), torch.cuda.Stream()
    q, k = x[:, :8], x[:, 8:10]
    dq, dk = q.contiguous() * 0.01, k.contiguous() * 0.01

    def both():
        a = skv.rope(h, spec, q, k, pos, q_weight=w[0], k_weight=w[1], stream=side)
        return a + skv.rope_backward(h, spec, dq, dk, pos, q=q, k=k, q_weight=w[0], k_weight=w[1], stream=side)

    torch.cuda.synchronize()
    ref = both()
    graph = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
        out = both()
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(both(), out):
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    assert not torch.equal(ref[4], out[4]) or torch.equal(ref[0], out[0])
    h.close()


def test_no_tokens(skv, h):
    import torch
    x, pos, freq, axis, w = _case(0, 2, 1, 64, 64, 1, torch.float16, 10)
    spec = skv.Rope(64, freq)
    a = skv.rope(h, spec, x[:, :2], x[:, 2:3], pos, q_weight=w[0], k_weight=w[1])
    assert a[0].shape == (0, 2, 64)
    b = skv.rope_backward(h, spec, a[0], a[1], pos, q=x[:, :2], k=x[:, 2:3], q_weight=w[0], k_weight=w[1])
    assert (b[2] == 0).all() and (b[3] == 0).all()


def test_a_training_step_of_attention(skv, h):
    """Projections -> norm and rotation -> attention -> its gradients -> gradients of norm and rotation, as used together,
    against autograd in 64 bits; every rounding in between is half a step of fp16 of q, k, v, dq, dk: 2^-8 of the norms
    is far above them."""
    import torch
    from tests.grad_util import rope_forward
    n, H, Hk, D = 200, 4, 2, 128
    x, pos, freq, axis, w = _case(n, H, Hk, D, D, 1, torch.float16, 0, seed=5)
    pos = torch.arange(n, device="cuda", dtype=torch.int32).view(1, n)
    spec = skv.Rope(D, freq)
    d_o = (torch.randn((1, n, H, D), device="cuda", generator=_gen(2)) * 0.1).half()
    xq, xk, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:].contiguous() / 3
    q, k = skv.rope(h, spec, xq, xk, pos, q_weight=w[0], k_weight=w[1])
    o, lse = skv.attn_partial(h, q.view(1, n, H, D), k, v, Hk=Hk, q_pos=pos)
    dq, dk, dv = skv.attn_backward(h, q.view(1, n, H, D), k, v, o, lse, d_o, Hk=Hk, q_pos=pos, g_dtype=torch.float16)
    got = skv.rope_backward(h, spec, dq.view(n, H, D), dk, pos, q=xq, k=xk, q_weight=w[0], k_weight=w[1]) + (dv,)
    assert h.status() == 0
    leaves = [t.double().requires_grad_() for t in (xq, xk, w[0], w[1], v)]
    yq, yk = rope_forward_grad(leaves[0], leaves[2], pos, freq), rope_forward_grad(leaves[1], leaves[3], pos, freq)
    s = torch.einsum("thd,nhd->htn", yq, yk.repeat_interleave(H // Hk, 1)) / D ** 0.5
    s = s.masked_fill(~(torch.arange(n, device="cuda").view(1, n) <= pos.view(n, 1)), -math.inf)
    y = torch.einsum("htn,nhd->thd", torch.softmax(s, -1), leaves[4].repeat_interleave(H // Hk, 1))
    want = torch.autograd.grad(y, leaves, d_o[0].double())
    for name, a, b in zip(("dxq", "dxk", "dwq", "dwk", "dv"), got, want):
        off = float((a.double() - b).norm() / b.norm())
        assert off <= 2.0 ** -8, (name, off)


def rope_forward_grad(x, w, pos, freq):
    """Half-split rotation of normed rows by differentiable steps."""
    import torch
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    th = (pos.double().view(-1, 1) * freq.double()).unsqueeze(1)
    a, b = y.chunk(2, -1)
    return torch.cat((a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos()), -1)


def test_rows_far_into_a_cache_and_a_projection(skv, h):
    """Cache rows and token strides whose offsets pass 32 bits."""
    import torch
    from tests.grad_util import check
    H, Hk, D, n = 2, 1, 128, 5
    rows = (1 << 32) // 256 + 100                                # 4 GiB of fp16 rows and a little
    K = torch.zeros((rows, Hk, D), dtype=torch.float16, device="cuda")
    V = torch.zeros((rows, Hk, D), dtype=torch.float16, device="cuda")
    stride = (1 << 30) + 64                                      # elements; the last token starts beyond 2^32
    flat = torch.empty(4 * stride + 4 * D, dtype=torch.float16, device="cuda")
    x = flat.as_strided((n, H + 2 * Hk, D), (stride, D, 1))
    g = _gen(3)
    x.copy_(torch.randn(x.shape, device="cuda", generator=g))
    pos = torch.arange(n, device="cuda", dtype=torch.int32).view(1, n)
    freq = (10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)).float()
    at = (rows - 1 - 2 * torch.arange(n, device="cuda")).to(torch.int32)
    spec = skv.Rope(D, freq)
    q = skv.rope_append(h, spec, x[:, :H], x[:, H:H + 1], x[:, H + 1:], pos, at, K, V)
    assert h.status() == 0
    zero = torch.zeros(64, dtype=torch.int32, device="cuda")
    for a, b in ((x[:, :H], q), (x[:, H:H + 1], K[at.long()])):
        want, bound = _turn_bound(a, None, pos, freq, zero, False, 1.0)
        check(b, want, bound, "far")
    assert torch.equal(V[at.long()], x[:, H + 1:])
    assert int((K.view(rows, -1) != 0).any(1).sum()) == n
    dq = skv.rope_backward(h, spec, q, None, pos, dq=x[:, :H])[0]
    assert dq.data_ptr() == x.data_ptr()
    # turned there and back: two roundings of fp16 and what they pass through a turn
    back = skv.rope_backward(h, spec, q, None, pos, x_dtype=torch.float32)[0]
    assert torch.equal(back.half(), dq)

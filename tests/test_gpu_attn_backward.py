"""Gradients of attention against the formulas in 64 bits, value by value within bounds derived from the kernels'
arithmetic (grad_util), and against differences of the forward call."""
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


def _inputs(S, nq, n, H, Hk, D, seed=0, shared=True, do="f16", amp=1.5):
    import torch
    g = _gen(seed * 7919 + nq * 31 + n)
    f16 = torch.float16
    q = (torch.randn((S, nq, H, D), device="cuda", generator=g) * amp).to(f16)
    rows = n if shared else S * n
    k = (torch.randn((rows, Hk, D), device="cuda", generator=g) + torch.randn((1, Hk, D), device="cuda", generator=g)).to(f16)
    v = torch.randn((rows, Hk, D), device="cuda", generator=g).to(f16)
    d_o = torch.randn((S, nq, H, D), device="cuda", generator=g) * 0.1
    return q, k, v, d_o.to(f16) if do == "f16" else d_o


def _want(q, k, v, see, o, lse, d_o, d_lse=None, scale=None):
    from tests.grad_util import attention_backward
    return attention_backward(q, k, v, see, q.shape[-1] ** -0.5 if scale is None else scale, o, lse, d_o, d_lse)


def _forward(q, k, v, see, scale=None):
    from tests.grad_util import attention_forward
    return attention_forward(q, k, v, see, q.shape[-1] ** -0.5 if scale is None else scale)


def _check3(got, want, bound, what):
    from tests.grad_util import check
    for name, x, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        if x is not None:
            check(x, w.reshape(x.shape), b.reshape(x.shape), f"{what} {name}")


DENSE = [
    # S, nq, n, H, Hk, D, causal
    (1, 1, 1, 1, 1, 64, False),
    (1, 1, 1, 2, 1, 128, True),
    (1, 64, 256, 4, 1, 64, True),
    (1, 128, 128, 2, 2, 128, False),
    (1, 127, 129, 2, 1, 128, True),
    (1, 300, 300, 5, 1, 128, True),          # five query heads a KV head
    (2, 33, 257, 6, 2, 64, False),           # two sequences share the keys
    (3, 7, 500, 8, 2, 128, True),            # few tokens: several heads in a tile
    (1, 1, 1000, 32, 8, 128, False),         # one token
    (1, 1, 3001, 16, 1, 64, True),
    (1, 1000, 1, 4, 2, 128, False),          # one key
    (1, 513, 1025, 4, 4, 128, True),
    (1, 200, 90, 3, 1, 128, True),           # more tokens than keys: the first see nothing
    (2, 100, 640, 40, 8, 128, True),
    (1, 40, 70, 130, 1, 64, False),          # more heads than a tile has rows
]


@pytest.mark.parametrize("g16", [True, False])
@pytest.mark.parametrize("S,nq,n,H,Hk,D,causal", DENSE)
def test_dense(skv, h, S, nq, n, H, Hk, D, causal, g16):
    import torch
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D)
    pos = None
    see = torch.ones((1, S * nq, n), dtype=torch.bool, device="cuda")
    if causal:
        pos = (n - nq + torch.arange(nq, device="cuda")).repeat(S, 1).to(torch.int32)
        see = torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(1, S * nq, 1)
    q1, d1 = q.view(1, S * nq, H, D), d_o.view(1, S * nq, H, D)
    o, lse = _forward(q1, k[None], v[None], see)
    want, bound = _want(q1, k[None], v[None], see, o, lse, d1)
    got = skv.attn_backward(h, q, k, v, o.view(S, nq, H, D), lse.view(S, nq, H), d_o, Hk=Hk, q_pos=pos,
                            g_dtype=torch.float16 if g16 else torch.float32)
    assert h.status() == 0
    _check3(got, want, bound, f"{(S, nq, n, H, Hk, D, causal)}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_lists(skv, h, D, per_head, causal):
    """Ragged sequences of one cache: rows in no order, padding behind and inside the lists, rows of no list hold NaN."""
    import torch
    S, nq, n, H, Hk = 3, 150, 300, 6, 2
    g = _gen(5)
    q, _, _, d_o = _inputs(S, nq, n, H, Hk, D, seed=3)
    rows = 1200
    k = torch.full((rows, Hk, D), math.nan, dtype=torch.float16, device="cuda")
    v = torch.full((rows, Hk, D), math.nan, dtype=torch.float16, device="cuda")
    lists = torch.full((S, Hk, n), -1, dtype=torch.int32, device="cuda")
    lens = [300, 129, 0]
    for s in range(S):
        for hk in range(Hk):
            own = torch.randperm(rows, device="cuda", generator=g)[:lens[s]] if per_head or hk == 0 else None
            lists[s, hk, :lens[s]] = own.to(torch.int32) if own is not None else lists[s, 0, :lens[s]]
    lists[0, :, 5] = -1                                       # a hole
    lists[0, :, 128:260] = -1                                 # a whole tile of them
    on = lists.permute(1, 0, 2).reshape(Hk, -1)
    for hk in range(Hk):
        r = on[hk][on[hk] >= 0].long()
        k[r, hk] = torch.randn((len(r), D), device="cuda", generator=g).to(torch.float16)
        v[r, hk] = torch.randn((len(r), D), device="cuda", generator=g).to(torch.float16)
    given = lists if per_head else lists[:, 0].contiguous()
    pos, lim = None, torch.full((S, nq), n, device="cuda")
    if causal:
        pos = torch.stack([torch.arange(nq, device="cuda") * 2 + 1, torch.arange(nq, device="cuda") - 20,
                           torch.arange(nq, device="cuda")]).to(torch.int32)
        lim = pos + 1
    wants, bounds, os, ls = [], [], [], []
    for hk in range(Hk):                                      # each KV head by itself: its own list
        r = lists[:, hk].long().clamp_min(0)
        kk, vv = (torch.where((lists[:, hk] >= 0).unsqueeze(-1), x[r, hk], 0.0).unsqueeze(2) for x in (k, v))
        see = (lists[:, hk] >= 0).unsqueeze(1) & (torch.arange(n, device="cuda") < lim.unsqueeze(-1))
        heads = slice(hk * H // Hk, (hk + 1) * H // Hk)
        o, lse = _forward(q[:, :, heads], kk, vv, see)
        w, b = _want(q[:, :, heads], kk, vv, see, o, lse, d_o[:, :, heads])
        wants.append(w), bounds.append(b), os.append(o), ls.append(lse)
    o, lse = torch.cat(os, 2).contiguous(), torch.cat(ls, 2).contiguous()
    got = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, kv_rows=given, kv_rows_per_head=per_head, q_pos=pos,
                            g_dtype=torch.float16)
    assert h.status() == 0
    assert got[1].shape == (S, n, Hk, D)
    _check3(got, [torch.cat(x, 2) for x in zip(*wants)], [torch.cat(x, 2) for x in zip(*bounds)], "lists")
    gone = (lists < 0).permute(0, 2, 1)
    assert (got[1][gone] == 0).all() and (got[2][gone] == 0).all() and (got[0][2] == 0).all()


def test_forward_and_backward_of_partitions(skv, h):
    """Two partitions, merged: each one's share from the merged o and lse; the shares of dq add up."""
    import torch
    S, nq, n, cut, H, Hk, D = 2, 70, 700, 301, 8, 2, 128
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D, seed=9)
    pos = (torch.arange(nq, device="cuda") * 9 + 5).repeat(S, 1).to(torch.int32)
    see = torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(1, S * nq, 1)
    parts = [skv.attn_partial(h, q, k, v, Hk=Hk, kv_begin=a, kv_end=b, q_pos=pos) for a, b in ((0, cut), (cut, n))]
    o, lse = skv.attn_combine(h, torch.stack([x[0].view(-1, D) for x in parts]), torch.stack([x[1].view(-1) for x in parts]))
    o, lse = o.view(S, nq, H, D), lse.view(S, nq, H)
    a = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, kv_end=cut, q_pos=pos)
    b = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, kv_begin=cut, q_pos=pos)
    assert h.status() == 0
    q1 = q.view(1, S * nq, H, D)
    want, bound = _want(q1, k[None], v[None], see, o.view(1, S * nq, H, D), lse.view(1, S * nq, H), d_o.view(1, S * nq, H, D))
    got = a[0] + b[0], torch.cat((a[1], b[1])), torch.cat((a[2], b[2]))
    # (dq is the sum of two results: twice the bound's parts that go by the largest value)
    _check3(got, want, [x * 2 for x in bound[:1]] + list(bound[1:]), "partitions")


@pytest.mark.parametrize("do", ["f16", "f32"])
def test_gradient_of_lse_scale_and_strides(skv, h, do):
    """d_lse beside d_o, another scale, rows of k and v inside wider ones, a position offset."""
    import torch
    S, nq, n, H, Hk, D = 1, 190, 333, 4, 2, 64
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D, seed=2, do=do)
    g = _gen(77)
    wide = torch.full((n, 2 * Hk * D + 24), math.nan, dtype=torch.float16, device="cuda")
    wide[:, :Hk * D], wide[:, Hk * D + 8:2 * Hk * D + 8] = k.view(n, -1), v.view(n, -1)
    kk, vv = wide, wide[:, Hk * D + 8:]
    pos = torch.randint(900, 1400, (S, nq), device="cuda", generator=g).to(torch.int32)
    see = 1000 + torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(1, nq, 1)
    o, lse = _forward(q, k[None], v[None], see, 0.3)
    d_lse = torch.randn((S, nq, H), device="cuda", generator=g)
    want, bound = _want(q, k[None], v[None], see, o, lse, d_o, d_lse, 0.3)
    got = skv.attn_backward(h, q, kk, vv, o, lse, d_o, Hk=Hk, q_pos=pos, key_pos0=1000, d_lse=d_lse, scale=0.3, kv_end=n,
                            k_row_bytes=wide.stride(0) * 2, v_row_bytes=wide.stride(0) * 2)
    assert h.status() == 0
    assert int((~see.any(-1)).sum()) > 0
    _check3(got, want, bound, "d_lse")


@pytest.mark.parametrize("D", [64, 128])
def test_fp32_gradients_of_every_size(skv, h, D):
    """Rows of d_o from 2^-90 to 2^60: dq of each row keeps its bits; all of one size: dk and dv do."""
    import torch
    nq, n, H, Hk = 260, 200, 2, 1
    q, k, v, d_o = _inputs(1, nq, n, H, Hk, D, seed=4, do="f32")
    see = torch.ones((1, nq, n), dtype=torch.bool, device="cuda")
    o, lse = _forward(q, k[None], v[None], see)
    for e in (-90, 0, 60):
        x = d_o * 2.0 ** e
        want, bound = _want(q, k[None], v[None], see, o, lse, x)
        _check3(skv.attn_backward(h, q, k, v, o, lse, x, Hk=Hk), want, bound, f"2^{e}")
    e = torch.randint(-60, 41, (1, nq, H, 1), device="cuda", generator=_gen(1))
    x = d_o * torch.exp2(e.float())
    want, bound = _want(q, k[None], v[None], see, o, lse, x)
    _check3(skv.attn_backward(h, q, k, v, o, lse, x, Hk=Hk), want, bound, "mixed")
    z = torch.zeros_like(d_o)
    assert all((t == 0).all() for t in skv.attn_backward(h, q, k, v, o, lse, z, Hk=Hk))
    assert h.status() == 0


@pytest.mark.parametrize("nq,n,H,Hk,D", [(17000, 130, 2, 1, 128), (70, 17000, 2, 2, 128), (300, 34000, 1, 1, 64)])
def test_long_sums(skv, h, nq, n, H, Hk, D):
    """Values of one sign over more than 128 tiles (the accumulators are emptied in between), and over few rows (split
    into pieces)."""
    import torch
    q, k, v, d_o = _inputs(1, nq, n, H, Hk, D, seed=6, amp=0.3)
    q, k, v, d_o = q.abs(), k.abs(), v.abs(), d_o.abs()
    see = torch.ones((1, nq, n), dtype=torch.bool, device="cuda")
    o, lse = _forward(q, k[None], v[None], see)
    want, bound = _want(q, k[None], v[None], see, o, lse, d_o)
    got = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk)
    assert h.status() == 0
    _check3(got, want, bound, "long")


def test_what_is_not_seen_is_not_looked_at(skv, h):
    """Padding tokens (lse = -inf) and keys behind the last position hold NaN and infinities."""
    import torch
    S, nq, n, H, Hk, D = 2, 200, 400, 4, 2, 128
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D, seed=8)
    pos = (torch.arange(nq, device="cuda") + 60).repeat(S, 1).to(torch.int32)
    pos[0, 150:], pos[1, 3:9] = -1, -1
    see = (torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(1, S * nq, 1))
    q1 = q.view(1, S * nq, H, D)
    o, lse = _forward(q1, k[None], v[None], see)
    want, bound = _want(q1, k[None], v[None], see, o, lse, d_o.view(1, S * nq, H, D))
    bad = pos.view(S, nq) < 0
    k[260:], v[260:] = math.nan, math.inf
    q[bad], d_o[bad] = math.nan, math.inf
    o = o.view(S, nq, H, D).clone()
    o[bad] = math.nan
    got = skv.attn_backward(h, q, k, v, o, lse.view(S, nq, H), d_o, Hk=Hk, q_pos=pos, g_dtype=torch.float16)
    assert h.status() == 0
    _check3(got, want, bound, "unseen")
    assert (got[0][bad] == 0).all() and (got[1][260:] == 0).all() and (got[2][260:] == 0).all()


def test_parts_repeats_streams_and_graphs(skv):
    """The parts alone give what they give together (cut into other pieces, so not bit for bit); repeated calls, another
    stream, a captured and replayed call on new inputs, and a second handle at the same time give the same bits."""
    import torch
    S, nq, n, H, Hk, D = 1, 333, 777, 8, 2, 128
    h, h2 = skv.Handle(0), skv.Handle(0)
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D, seed=11)
    see = torch.ones((1, nq, n), dtype=torch.bool, device="cuda")
    o, lse = _forward(q, k[None], v[None], see)
    ref = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk)
    dq = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, need_dkv=False)
    dkv = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, need_dq=False)
    assert dq[1] is None and dkv[0] is None
    want, bound = _want(q, k[None], v[None], see, o, lse, d_o)
    _check3(ref, want, bound, "together")
    _check3((dq[0], dkv[1], dkv[2]), want, bound, "alone")
    for part in (dict(need_dkv=False), dict(need_dq=False)):
        for x, y in zip(skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, **part), dq if "need_dkv" in part else dkv):
            assert x is y is None or torch.equal(x, y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    one = skv.attn_backward(h2, q, k, v, o, lse, d_o, Hk=Hk, stream=side)
    two = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk)
    torch.cuda.synchronize()
    for a, b, c in zip(ref, one, two):
        assert torch.equal(a, b) and torch.equal(a, c)
    outs = [torch.empty_like(x) for x in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
        skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, dq=outs[0], dk=outs[1], dv=outs[2], stream=side)
    d_o.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk), outs):
        assert torch.equal(a, b)
    h.close(), h2.close()


def test_growth_during_capture_is_refused(skv):
    import torch
    h = skv.Handle(0)
    q, k, v, d_o = _inputs(1, 64, 64, 2, 1, 64)
    o, lse = skv.attn_partial(h, q, k, v, Hk=1)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out = [torch.empty((1, 64, 2, 64), device="cuda"), torch.empty((64, 1, 64), device="cuda"), torch.empty((64, 1, 64), device="cuda")]
    fresh = skv.Handle(0)
    with pytest.raises(skv.SplitKVError) as e:
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            skv.attn_backward(fresh, q, k, v, o, lse, d_o, Hk=1, dq=out[0], dk=out[1], dv=out[2], stream=side)
    assert e.value.status == 5
    torch.cuda.synchronize()
    fresh.close(), h.close()


def test_empty_range(skv, h):
    import torch
    q, k, v, d_o = _inputs(1, 5, 8, 2, 1, 64)
    o, lse = torch.zeros((1, 5, 2, 64), device="cuda"), torch.full((1, 5, 2), -math.inf, device="cuda")
    dq, dk, dv = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=1, kv_begin=3, kv_end=3)
    assert (dq == 0).all() and dk.shape == dv.shape == (0, 1, 64)


@pytest.mark.parametrize("nq,n,H,Hk,D,causal", [
    (2048, 2048, 1, 1, 64, True),            # both kinds of CTAs cut into pieces
    (1500, 1500, 1, 1, 128, False),
    (2100, 6000, 16, 1, 64, False),          # pieces of dk and dv longer than a stretch of 128 tiles
    (1100, 34000, 4, 2, 64, True),           # pieces of dq longer than one
])
@pytest.mark.parametrize("g16", [True, False])
def test_pieces(skv, h, nq, n, H, Hk, D, causal, g16):
    import torch
    q, k, v, d_o = _inputs(1, nq, n, H, Hk, D, seed=31)
    pos, see = None, torch.ones((1, nq, n), dtype=torch.bool, device="cuda")
    if causal:
        pos = (n - nq + torch.arange(nq, device="cuda")).to(torch.int32).view(1, nq)
        see = torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(1, nq, 1)
    o, lse = _forward(q, k[None], v[None], see)
    want, bound = _want(q, k[None], v[None], see, o, lse, d_o)
    kw = dict(Hk=Hk, q_pos=pos, g_dtype=torch.float16 if g16 else torch.float32)
    got = skv.attn_backward(h, q, k, v, o, lse, d_o, **kw)
    assert h.status() == 0
    _check3(got, want, bound, "pieces")
    again = skv.attn_backward(h, q, k, v, o, lse, d_o, **kw)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_against_differences(skv, h):
    """sum(o * w) + sum(lse * u) of the forward call, moved along random directions of q, k and v (fp32 o and lse: a
    difference over a step of 2^-4 is good to the step's square and to the call's 1e-5)."""
    import torch
    S, nq, n, H, Hk, D = 1, 64, 160, 4, 2, 128
    q, k, v, _ = _inputs(S, nq, n, H, Hk, D, seed=13, amp=0.5)
    g = _gen(14)
    w = torch.randn((S, nq, H, D), device="cuda", generator=g)
    u = torch.randn((S, nq, H), device="cuda", generator=g)
    pos = (torch.arange(nq, device="cuda") + n - nq).view(1, nq).to(torch.int32)
    see = torch.arange(n, device="cuda").view(1, 1, n) <= pos.view(1, nq, 1)
    from tests.grad_util import attention_forward
    o, lse = skv.attn_partial(h, q, k, v, Hk=Hk, q_pos=pos)
    grads = skv.attn_backward(h, q, k, v, o, lse, w, Hk=Hk, q_pos=pos, d_lse=u)

    def value(q, k, v):
        o, lse = attention_forward(q.double(), k.double()[None], v.double()[None], see, D ** -0.5)
        return float((o.double() * w).sum() + (lse.double() * u).sum())

    step = 2.0 ** -7
    for i, x in enumerate((q, k, v)):
        way = torch.randn(x.shape, device="cuda", generator=g).double()
        args = [[t.double() for t in (q, k, v)] for _ in "ab"]
        args[0][i] = args[0][i] + step * way
        args[1][i] = args[1][i] - step * way
        slope = (value(*args[0]) - value(*args[1])) / (2 * step)
        got = float((grads[i].double() * way).sum())
        # fp16 operands: 2^-11 of each product, of random sign; 1e-3 of the gradient's and direction's norms is far above
        room = 1e-3 * float(grads[i].double().norm() * way.norm())
        assert abs(slope - got) <= room, (i, slope, got, room)


@pytest.mark.parametrize("lists", [False, True])
def test_rows_far_into_a_cache(skv, h, lists):
    """Keys whose offsets pass 32 bits: the end of a cache of a little over 4 GiB, as a range and by lists."""
    import torch
    S, nq, n, H, Hk, D = 1, 40, 200, 2, 1, 128
    rows = (1 << 32) // 256 + 300
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D, seed=21)
    K = torch.full((rows, Hk, D), math.nan, dtype=torch.float16, device="cuda")
    V = torch.full((rows, Hk, D), math.nan, dtype=torch.float16, device="cuda")
    K[rows - n:], V[rows - n:] = k, v
    see = torch.ones((1, nq, n), dtype=torch.bool, device="cuda")
    o, lse = _forward(q, k[None], v[None], see)
    want, bound = _want(q, k[None], v[None], see, o, lse, d_o)
    if lists:
        at = torch.arange(rows - n, rows, device="cuda", dtype=torch.int32).view(1, n)
        got = skv.attn_backward(h, q, K, V, o, lse, d_o, Hk=Hk, kv_rows=at)
    else:
        got = skv.attn_backward(h, q, K, V, o, lse, d_o, Hk=Hk, kv_begin=rows - n)
    assert h.status() == 0
    _check3(got, want, bound, "far")


def test_a_set_status_bit_does_not_disturb(skv):
    """Bits that other calls leave in the status word (an append beyond its cache) do not end a gradient's waits."""
    import torch
    h = skv.Handle(0)
    q, k, v, d_o = _inputs(1, 300, 500, 4, 2, 128, seed=22)
    o, lse = skv.attn_partial(h, q, k, v, Hk=2)
    ref = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=2)
    assert h.status() == 0
    skv.kv_append(h, torch.zeros((1, 2, 128), device="cuda"), torch.tensor([600], dtype=torch.int32, device="cuda"), k.clone())
    got = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=2)
    with pytest.raises(skv.SplitKVError) as e:
        h.status()
    assert e.value.status == 8
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    h.close()


def test_many_heads_and_sequences(skv, h):
    """More KV heads times sequences than fit a wave, lists of other lengths than the tokens, one token each."""
    import torch
    S, nq, n, H, Hk, D = 9, 1, 333, 80, 40, 64
    q, k, v, d_o = _inputs(S, nq, n, H, Hk, D, seed=23, shared=False)
    lists = torch.arange(S * n, device="cuda", dtype=torch.int32).view(S, n)
    see = torch.ones((S, nq, n), dtype=torch.bool, device="cuda")
    kk, vv = k.view(S, n, Hk, D), v.view(S, n, Hk, D)
    o, lse = _forward(q, kk, vv, see)
    want, bound = _want(q, kk, vv, see, o, lse, d_o)
    got = skv.attn_backward(h, q, k, v, o, lse, d_o, Hk=Hk, kv_rows=lists)
    assert h.status() == 0
    _check3(got, want, bound, "many")

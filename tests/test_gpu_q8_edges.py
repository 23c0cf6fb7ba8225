"""The calls over 8-bit pages at their edges, against definitions in 64 bits: scales of
either sign and far apart, rows beside pages that they do not see, rows that one key decides,
very long lists and selections, lengths beyond their lists, and the borders between the forms
of the choice."""
import numpy as np
import pytest

import q8_rows as r
import q8_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    import split_kv_flash_attn_gb300 as skv
    x = skv.Handle(0)
    yield x
    x.close()


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _q(rng, S, nq, H, D):
    return rng.standard_normal((S, nq, H, D)).astype(np.float16)


# ------------------------------------------------------- scales of either sign

def _signed(rng, lens, Hk, D, extra):
    c = u.Cache(rng, lens, Hk, D, extra=extra)
    c.ks *= rng.choice([-1, 1], c.n_pages).astype(np.float32)
    c.vs *= rng.choice([-1, 1], c.n_pages).astype(np.float32)
    return c


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("D,Hk,n,lens,size", [
    # rows that grow the scale, that do not, and that are zeros
    (128, 2, 3, [10, 63, 1, 64], 30.0), (64, 3, 20, [5, 40, 127], 0.01), (128, 1, 7, [33, 2], 0.0), (64, 2, 70, [61, 0, 100], 1.0)])
def test_append_to_pages_of_a_negative_scale(h, D, Hk, n, lens, size, f16):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(D + n)
    c = _signed(rng, lens, Hk, D, n)
    pool, ids, kv_len = c.on_gpu()
    held = c.k[c.ids[0, 0, 0], 0].astype(np.float64) * float(c.ks[c.ids[0, 0, 0]])
    x = (rng.standard_normal((2, len(lens), n, Hk, D)) * size).astype(np.float16 if f16 else np.float32)
    for _ in range(2):                                # again: the same bytes
        skv.q8_append(h, pool, _dev(x[0]), _dev(x[1]), ids, kv_len)
        r.append(c, x[0], x[1])
        for name, want in (("k", c.k), ("v", c.v), ("k_scale", c.ks), ("v_scale", c.vs)):
            got = getattr(pool, name).cpu().numpy()
            assert np.array_equal(got, want), f"{name} differs in {np.count_nonzero(got != want)} places"
    # what was held is still there, to half a step of the new scale
    p = c.ids[0, 0, 0]
    assert np.abs(c.k[p, 0] * float(c.ks[p]) - held).max() <= 0.5001 * c.ks[p]
    assert h.status() == 0


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("D,Hk,n,lens,size", [(128, 2, 3, [10, 63, 1, 64], 30.0), (64, 3, 20, [5, 40, 127], 0.01), (128, 1, 70, [33, 2], 1.0)])
def test_extremes_of_pages_of_a_negative_scale(h, D, Hk, n, lens, size, f16):
    """Recoding with a negative factor exchanges the smallest and the largest codes."""
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(D + n + 1)
    c = _signed(rng, lens, Hk, D, n)
    pool, ids, kv_len = c.on_gpu()
    x = (rng.standard_normal((2, len(lens), n, Hk, D)) * size).astype(np.float16 if f16 else np.float32)
    skv.q8_append(h, pool, _dev(x[0]), _dev(x[1]), ids, kv_len)
    r.append(c, x[0], x[1])
    assert np.array_equal(pool.k_min.cpu().numpy(), c.lo) and np.array_equal(pool.k_max.cpu().numpy(), c.hi)
    # and a selection of the pages written, whose scales are positive now
    c.lens += n
    c.ks = np.abs(c.ks)
    pool.k_scale.abs_()
    q = _q(rng, len(lens), 1, 4 * Hk, D)
    got = skv.q8_select(h, pool, _dev(q), ids, kv_len + n, n_sel=2, n_first=0, n_last=0)
    assert np.array_equal(got.cpu().numpy(), u.select(c, q, 2, 0, 0))
    assert h.status() == 0


@pytest.mark.parametrize("lens,nq,H,Hk,D,n", [([3000, 700], 1, 8, 2, 128, 6), ([64 * 1500], 1, 4, 1, 64, 100), ([2000], 5, 12, 2, 64, 4),
                                              ([64 * 300], 1, 150, 1, 128, 20), ([64 * 40, 0], 1, 1, 1, 64, 7)])
def test_selection_over_scales_of_either_sign(h, lens, nq, H, Hk, D, n):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(sum(lens) + D)
    c = _signed(rng, lens, Hk, D, 0)
    c.ks[c.ids[0, 0, 5]] = 0.0
    c.ks[c.ids[0, 0, 6]] = -0.0
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, len(lens), nq, H, D)
    q_pos = (c.lens[:, None] - nq + np.arange(nq)[None]).astype(np.int32) if nq > 1 else None
    got = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=n, n_first=0, n_last=0, q_pos=None if q_pos is None else _dev(q_pos))
    assert np.array_equal(got.cpu().numpy(), r.select(c, q, n, 0, 0, q_pos))
    assert h.status() == 0


def test_the_bound_of_a_negative_scale_is_one(h):
    """The page of the best key under the coded query is picked when every other page's bound is lower."""
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(3)
    c = u.Cache(rng, [64 * 40], 1, 128)
    c.k //= 8
    c.ks[:] = -0.03
    q = _q(rng, 1, 1, 1, 128)
    cq = u.code(q[0, 0, 0], np.float32(np.abs(q).astype(np.float64).max() / 127)).astype(int)
    c.k[c.ids[0, 0, 17], 9] = np.clip(-cq, -127, 127)    # one key along the query, its codes against it
    c.extremes()
    pool, ids, kv_len = c.on_gpu()
    got = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=1, n_first=0, n_last=0).cpu().numpy()
    assert got.tolist() == [[[[17]]]]


# ------------------------------------------------ values that a row does not see

@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("D,nq,H,Hk", [(128, 90, 4, 2), (64, 300, 1, 1), (128, 3, 8, 2)])
def test_a_far_value_scale_behind_a_row_s_limit(h, D, nq, H, Hk, f16):
    """Tokens that see the first page of a tile, whose other page holds values 2^30 as large: each row
    within what its own keys give (fp16: as half a step of its own weights and results)."""
    import split_kv_flash_attn_gb300 as skv
    import torch
    rng = np.random.default_rng(D + nq)
    c = u.Cache(rng, [640, 200], Hk, D)
    near, far = c.ids[:, :, 0:10:2], c.ids[:, :, 1:10:2]
    c.vs[near[near >= 0]] *= np.float32(2.0 ** (-15 if not f16 else -3))
    c.vs[far[far >= 0]] *= np.float32(2.0 ** (15 if not f16 else 27))
    q_pos = rng.integers(0, 640, (2, nq)).astype(np.int32)
    q_pos[:, : nq if f16 else nq // 2] = rng.integers(0, 64, (2, nq if f16 else nq // 2))   # (far values are beyond fp16)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 2, nq, H, D)
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(q_pos), o_dtype=torch.float16 if f16 else None)
    r.check(o, lse, r.attention(c, q, q_pos=q_pos), f16=f16)
    assert h.status() == 0


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("nq,causal", [(1, False), (3, True), (40, False), (40, True)])
def test_far_scales_row_by_row(h, nq, causal, f16):
    """Lists whose value scales lie up to 2^40 apart, absent pages, zero and negative scales: every row
    within its own bound (a bound over all rows would pass zeros for the smaller ones)."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(nq + causal)
    c = u.Cache(rng, [700, 640, 128, 300], 2, 128)
    c.ids[0, 0, 3] = -1
    c.ids[0, 1, 0] = -5
    c.ids[2, 1, :2] = -1
    for s in range(4):
        for k in range(2):
            p = c.ids[s, k][c.ids[s, k] >= 0]
            c.vs[p] *= np.float32(2.0 ** (-12 if f16 else -40) * rng.random()) * rng.choice([-1, 1], len(p)).astype(np.float32)
            if k:                                     # and far from one another within a list
                c.vs[p] *= (2.0 ** rng.integers(-4 if f16 else -30, 10, len(p))).astype(np.float32)
    c.vs[c.ids[1, 0, 1]] = 0.0
    c.ks[c.ids[1, 1, 4]] = 0.0
    c.ks[c.ids[0, 0, 1]] *= -1
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 4, nq, 8, 128)
    q_pos = (c.lens[:, None] - nq + np.arange(nq)[None]).astype(np.int32) if causal else None
    if causal:
        q_pos[:, ::2] = rng.integers(0, 700, q_pos[:, ::2].shape)
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=None if q_pos is None else _dev(q_pos),
                         o_dtype=torch.float16 if f16 else None)
    r.check(o, lse, r.attention(c, q, q_pos=q_pos), f16=f16)
    assert h.status() == 0


# ------------------------------------------------------- rows that one key decides

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("masked", [True, False])
def test_fp32_rows_of_one_key(h, D, masked):
    """Rows of one visible key (or of one key whose score leaves the others nothing) in units of
    1 to 10 tiles of 128 keys, one unit a CTA: o is that key's value.

    Relative bound.  The weight in two fp16 parts 2^-22; the truncated sum of their products, and of
    the weights, 2^-23 each; the value's scale through log2 (one step of a number below 8, times ln 2:
    2^-21.5) and 2^x (2^-22), their difference's rounding (2^-23); seven more fp32 roundings of 2^-24:
    in all 2^-19.3, so 2^-19."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(D)
    Hk = 8
    S = max(1, torch.cuda.get_device_properties(0).multi_processor_count // Hk)
    for tiles in (1, 4, 8, 10):
        n = 128 * tiles
        c = u.Cache(rng, [n] * S, Hk, D)
        c.ks[:] = 0.05
        key = rng.integers(0, n, S)
        q = np.zeros((S, 40, Hk, D), np.float16)
        q_pos = np.full((S, 40), n - 1, np.int32)
        if masked:
            key[:] = 0
            q_pos[:, :39] = 0
        else:
            for s in range(S):
                # the key along the query, all others at least 80 lower: 2^-115 of its weight
                sg = rng.choice([-1, 1], D)
                q[s] = (sg * 10).astype(np.float16)
                for k in range(Hk):
                    c.k[c.ids[s, k, key[s] // 64], key[s] % 64] = 127 * sg
        c.extremes()
        pool, ids, kv_len = c.on_gpu()
        o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(q_pos))
        o = o.double().cpu().numpy()
        for s in range(S):
            for k in range(Hk):
                p = c.ids[s, k, key[s] // 64]
                want = c.v[p, key[s] % 64].astype(np.float64) * float(c.vs[p])
                if not masked:
                    w = np.concatenate([c.k[c.ids[s, k, b]] for b in range(n // 64)]).astype(np.float64) @ q[s, 0, k].astype(np.float64)
                    w *= float(c.ks[p]) / np.sqrt(D)
                    w = np.sort(w)
                    assert w[-1] - w[-2] > 80
                off = np.abs(o[s, :39, k] - want).max() / np.abs(want).max()
                assert off <= 2.0 ** -19, f"{tiles} tiles, sequence {s}, head {k}: off by {off:.2e}"
    assert h.status() == 0


# ------------------------------------------------------- fp16 results over long lists

@pytest.mark.parametrize("D", [64, 128])
def test_fp16_results_over_long_lists(h, D):
    """Values of one sign over 524288 keys, a unit for every SM: the tensor core's truncated sums must
    not show beside the roundings to fp16 of the weights and of the result, half a step (2^-11) each."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    n, Hk, nq = 1 << 19, 8, 64
    S = max(1, torch.cuda.get_device_properties(0).multi_processor_count // Hk)
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    k = torch.randint(-60, 61, (n // 64, 64, D), device="cuda", generator=g, dtype=torch.int8)
    v = torch.randint(1, 128, (n // 64, 64, D), device="cuda", generator=g, dtype=torch.int8)
    ks, vs = (torch.full((n // 64,), x, device="cuda") for x in (0.02, 0.01))
    pool = skv.Q8Pool(k, v, ks, vs, k.amin(1), k.amax(1))
    ids = torch.arange(n // 64, device="cuda", dtype=torch.int32).expand(S, Hk, -1).contiguous()   # (one list for all)
    q = torch.randn((S, nq, Hk, D), device="cuda", generator=g).half()
    o, _ = skv.q8_attn(h, pool, q, ids, torch.full((S,), n, dtype=torch.int32, device="cuda"), o_dtype=torch.float16)
    assert h.status() == 0
    kk = k.view(n, D).double() * float(ks[0])
    for s in (0, S - 1):
        x = q[s, ::16].reshape(-1, D).double()
        want = torch.softmax(x @ kk.T * D ** -0.5, -1) @ (v.view(n, D).double() * float(vs[0]))
        off = ((o[s, ::16].reshape(-1, D).double() - want).abs() / want).max().item()
        # scores, as in q8_util: 2 (D + 4) 2^-23 A and 2^-18
        A = ((x.abs() @ kk[:8192].abs().T).max() * D ** -0.5).item()
        assert off <= 2.0 ** -10 + 2 * (D + 4) * 2.0 ** -23 * A + 2.0 ** -18


@pytest.mark.parametrize("D", [64, 128])
def test_fp16_results_of_long_pieces_across_units(h, D):
    """160 units of 80 to 330 tiles, more than there are SMs, so that pieces of over 128 tiles begin and end
    within units: fp16 results, log sums and weights beside the fp32 call's."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(D)
    S, Hk, H, nq, n_pages = 20, 8, 16, 40, 700
    lens = rng.integers(10000, 42000, S).astype(np.int32)
    cap = int(-(-lens.max() // 64))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()   # noqa: E731
    k = rng.integers(-60, 61, (n_pages, 64, D)).astype(np.int8)
    v = rng.integers(1, 128, (n_pages, 64, D)).astype(np.int8)
    pool = skv.Q8Pool(dev(k), dev(v), dev(rng.uniform(0.01, 0.03, n_pages).astype(np.float32)),
                      dev(rng.uniform(0.005, 0.02, n_pages).astype(np.float32)), dev(k.min(1)), dev(k.max(1)))
    ids = rng.integers(-1, n_pages, (S, Hk, cap)).astype(np.int32)     # (pages in several lists, some absent)
    q = _dev(_q(rng, S, nq, H, D))
    pos = _dev((lens[:, None] - nq + np.arange(nq)[None]).astype(np.int32))
    res = []
    for t in (torch.float32, torch.float16):
        mass = torch.zeros((S, Hk, cap), device="cuda")
        res.append((*skv.q8_attn(h, pool, q, dev(ids), dev(lens), q_pos=pos, mass=mass, o_dtype=t), mass))
    (o, lse, mass), (oo, ll, mm) = res
    # values of one sign, so sum p |v| = |o|: half a step for the weights and one for the result
    assert ((oo.double() - o.double()).abs() <= 2.0 ** -10 * o.double().abs() + 2.0 ** -17 * 127 * 0.02).all()
    # the same scores, summed in other stretches: 2^-22 of the log sums, 2^-20 for their sums
    assert ((ll - lse).abs() <= 2.0 ** -22 * lse.abs() + 2.0 ** -20).all()
    assert ((mm - mass).abs() <= 2.0 ** -16 * mass + 2.0 ** -20).all()
    one = skv.q8_attn(h, pool, q[7:8].contiguous(), dev(ids[7:8]), dev(lens[7:8]), q_pos=pos[7:8].contiguous())[0]
    assert ((one - o[7:8]).abs() <= 2.0 ** -17 * 127 * 0.02).all()
    assert h.status() == 0


# ------------------------------------------------------- lengths beyond their lists

@pytest.mark.parametrize("nq,cap", [(1, 4), (3, 4), (1, 1500)])
def test_selection_reports_a_length_beyond_its_list(h, nq, cap):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(12)
    c = u.Cache(rng, [cap * u.PAGE, 100], 2, 64, cap=cap)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 2, nq, 4, 64)
    kv_len[0] += 1                                    # cut to the list
    got = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=2)
    assert np.array_equal(got.cpu().numpy(), u.select(c, q, 2, 1, 1))
    with pytest.raises(skv.SplitKVError, match="0x4"):
        h.status()
    kv_len[0] -= 1
    skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=2)
    assert h.status() == 0


@pytest.mark.parametrize("S,nq", [(2, 1), (2, 3), (40, 1)])
def test_attention_over_a_selection_reports_a_length_beyond_its_list(h, S, nq):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(13)
    c = u.Cache(rng, [4 * u.PAGE] * S, 2, 64, cap=4)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, S, nq, 4, 64)
    sel = rng.integers(-1, 6, (S, nq, 2, 3)).astype(np.int32)
    kv_len[S - 1] += 1
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, sel=_dev(sel))
    u.check(o, lse, u.attention(c, q, sel=sel))
    with pytest.raises(skv.SplitKVError, match="0x4"):
        h.status()
    kv_len[S - 1] -= 1
    skv.q8_attn(h, pool, _dev(q), ids, kv_len, sel=_dev(sel))
    assert h.status() == 0


# ------------------------------------------------------- very many page visits

def test_selections_of_more_visits_than_2_to_the_30(h):
    """Nine tokens of 1024 heads on one KV head and selections that are padding but for a few pages: 1.2e9 visits."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(14)
    H, nq, n_sel = 1024, 9, 1 << 21
    c = u.Cache(rng, [400], 1, 64)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 1, nq, H, 64)
    few = [(0, 5), (1000003, 0), (n_sel - 1, 2)]
    sel = torch.full((1, nq, 1, n_sel), -1, dtype=torch.int32, device="cuda")
    for at, b in few:
        sel[..., at] = b
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, sel=sel)
    assert h.status() == 0
    want = np.broadcast_to(np.array([b for _, b in few], np.int32), (1, nq, 1, 3))
    u.check(o, lse, u.attention(c, q, sel=want))


# ------------------------------------------------------- the borders of the choice

@pytest.mark.parametrize("cap", [1024, 1025, 6144, 6145, 16384, 16385])
@pytest.mark.parametrize("full", [True, False])
def test_selection_at_the_borders_of_its_forms(h, cap, full):
    """Lists of as many pages as one form of the choice holds and of one more, filled to the last
    page or not, beside an empty one."""
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(cap)
    n = cap * u.PAGE - (0 if full else 65)
    c = u.Cache(rng, [n, 0], 1, 64, cap=cap)
    pool, ids, kv_len = c.on_gpu()
    assert ids.shape[2] == cap
    q = _q(rng, 2, 1, 2, 64)
    for n_sel in (1, 100, cap - 1):
        got = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=n_sel, n_first=0, n_last=1)
        assert np.array_equal(got.cpu().numpy(), u.select(c, q, n_sel, 0, 1))
    assert h.status() == 0


# ------------------------------------------------------- results in fp16

@pytest.mark.parametrize("lens,nq,H,Hk,D,sel", [([1000, 3, 517], 1, 16, 2, 128, False), ([5000], 2, 4, 1, 64, False), ([3000, 640], 5, 8, 1, 128, True)])
def test_fp16_results_of_up_to_eight_rows_are_the_fp32_ones_rounded(h, lens, nq, H, Hk, D, sel):
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(nq + H)
    c = u.Cache(rng, lens, Hk, D)
    pool, ids, kv_len = c.on_gpu()
    q = _dev(_q(rng, len(lens), nq, H, D))
    s = _dev(rng.integers(-1, 12, (len(lens), nq, Hk, 9)).astype(np.int32)) if sel else None
    o, lse = skv.q8_attn(h, pool, q, ids, kv_len, sel=s)
    oo, ll = skv.q8_attn(h, pool, q, ids, kv_len, sel=s, o_dtype=torch.float16)
    assert torch.equal(oo, o.half()) and torch.equal(ll, lse)


@pytest.mark.parametrize("lens,nq,H,Hk,D", [([4000, 900], 3, 8, 2, 128), ([4000], 200, 4, 2, 128), ([2500, 77], 60, 2, 1, 64)])
def test_fp16_results_of_more_rows(h, lens, nq, H, Hk, D):
    """One fp16 number a weight and one a result, half a step (2^-11) of each: no further from the fp32
    result than 2^-11 (sum p |v| + |o|), and 2^-17 for what the two differ by before."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(nq)
    c = u.Cache(rng, lens, Hk, D)
    pool, ids, kv_len = c.on_gpu()
    q = _dev(_q(rng, len(lens), nq, H, D))
    o, _ = skv.q8_attn(h, pool, q, ids, kv_len)
    oo, _ = skv.q8_attn(h, pool, q, ids, kv_len, o_dtype=torch.float16)
    pool.v.copy_(pool.v.abs())
    size, _ = skv.q8_attn(h, pool, q, ids, kv_len)    # sum p |v| (the scales are positive)
    vmax = 127 * float(c.vs.max())
    assert ((oo.double() - o.double()).abs() <= 2.0 ** -11 * (size.double() + o.double().abs()) + 2.0 ** -17 * vmax).all()

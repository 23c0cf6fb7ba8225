"""The calls over 8-bit pages on the GPU against their definitions in 64 bits:
appends code for code, attention within the arithmetic's bounds, selections and
evictions index for index, and the calls together as a server makes them."""
import numpy as np
import pytest

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


def _causal(c, nq):
    return (c.lens[:, None] - nq + np.arange(nq)[None]).astype(np.int32)


# --------------------------------------------------------------------- appends

@pytest.mark.parametrize("D,Hk,n,lens,f16", [
    (128, 2, 1, [0, 1, 63, 64, 65, 127], False), (64, 3, 1, [5, 62, 128], True),
    (128, 1, 64, [0, 1, 64, 100], True), (64, 2, 130, [0, 37, 63], False),
    (128, 2, 200, [3], False), (128, 8, 7, [60, 61, 0, 200], True)])
def test_append_codes(h, D, Hk, n, lens, f16):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(D + Hk * 10 + n)
    c = u.Cache(rng, lens, Hk, D, extra=n)
    pool, ids, kv_len = c.on_gpu()
    x = rng.standard_normal((2, len(lens), n, Hk, D)) * rng.choice([0.1, 1.0, 6.0], (2, len(lens), n, Hk, 1))
    x = x.astype(np.float16 if f16 else np.float32)
    for _ in range(2):                                # again: the same bytes
        skv.q8_append(h, pool, _dev(x[0]), _dev(x[1]), ids, kv_len)
        u.append(c, x[0], x[1])
        for name, want in (("k", c.k), ("v", c.v), ("k_scale", c.ks), ("v_scale", c.vs), ("k_min", c.lo), ("k_max", c.hi)):
            got = getattr(pool, name).cpu().numpy()
            assert np.array_equal(got, want), f"{name} differs in {np.count_nonzero(got != want)} places"
    assert h.status() == 0


def test_append_special_values_and_ragged_counts(h):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(5)
    D, Hk, lens = 64, 1, [10, 64, 0, 3, 70, 1]
    c = u.Cache(rng, lens, Hk, D, extra=20)
    c.vs[c.ids[3, 0, 0]] = np.float32(1e-41)          # a subnormal scale already there
    pool, ids, kv_len = c.on_gpu()
    x = rng.standard_normal((2, 6, 20, Hk, D)).astype(np.float32)
    x[0, 0, 3, 0, 5], x[0, 0, 4, 0, 6], x[0, 0, 5, 0, 7] = np.inf, -np.inf, np.nan
    x[1, 1] = 0.0                                     # nothing but zeros: scale 0
    x[:, 2] *= np.float32(2e-43)                      # subnormal values, scale of a few units
    x[1, 3] *= np.float32(1e-40)
    x[0, 4] *= np.float32(1e37)
    x[0, 5] = (np.arange(D) + 0.5).astype(np.float32) # exact ties against a scale of 1
    x[0, 5, :, 0, 0] = 127.0
    c.ks[c.ids[5, 0, 0]] = 1.0
    pool.k_scale[int(c.ids[5, 0, 0])] = 1.0
    n_new = np.array([20, 7, 20, 5, -3, 20], np.int32)
    skv.q8_append(h, pool, _dev(x[0]), _dev(x[1]), ids, kv_len, n_new=_dev(n_new))
    u.append(c, x[0], x[1], n_new)
    for name, want in (("k", c.k), ("v", c.v), ("k_scale", c.ks), ("v_scale", c.vs), ("k_min", c.lo), ("k_max", c.hi)):
        assert np.array_equal(getattr(pool, name).cpu().numpy(), want), name
    assert h.status() == 0


def test_append_of_more_pages_than_one_grid_has(h):
    """The tokens of one call, and of two that part at a page's border: the same bytes."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    n, cut, D = 2097152 + 300, 64 * 20000, 64
    cap = n // u.PAGE + 2
    x = torch.randn((2, 1, n, 1, D), device="cuda", dtype=torch.float16)
    ids = torch.randperm(cap, device="cuda").to(torch.int32).view(1, 1, cap)
    pools = []
    for parts in ([(0, n)], [(0, cut), (cut, n)]):
        pool = skv.Q8Pool.empty(cap, D)
        for t in (pool.k, pool.v, pool.k_scale, pool.v_scale, pool.k_min, pool.k_max):
            t.zero_()
        for a, b in parts:
            skv.q8_append(h, pool, x[0, :, a:b].contiguous(), x[1, :, a:b].contiguous(), ids,
                          torch.tensor([a], dtype=torch.int32, device="cuda"))
        pools.append(pool)
    for name in ("k", "v", "k_scale", "v_scale", "k_min", "k_max"):
        assert torch.equal(getattr(pools[0], name), getattr(pools[1], name)), name
    page = int(ids[0, 0, (n - 1) // u.PAGE])
    want = x[0, 0, (n - 1) // u.PAGE * u.PAGE:, 0].float()
    rows = want.shape[0]
    # half a step of the scale, and fp32 products
    assert ((pools[0].k[page, :rows].float() * pools[0].k_scale[page] - want).abs().max()
            <= pools[0].k_scale[page] * 0.5001)
    assert h.status() == 0


def test_append_without_a_page_is_reported(h):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(6)
    c = u.Cache(rng, [60, 5], 1, 64, cap=2)           # the first list has no second page
    pool, ids, kv_len = c.on_gpu()
    before = pool.k.clone()
    x = rng.standard_normal((2, 10, 1, 64)).astype(np.float32)
    skv.q8_append(h, pool, _dev(x), _dev(x), ids, kv_len)
    with pytest.raises(skv.SplitKVError, match="0x2"):
        h.status()
    u.append(c, x, x)
    assert np.array_equal(pool.k.cpu().numpy(), c.k) and not np.array_equal(before.cpu().numpy(), c.k)
    ids[0, 0, 1] = c.n_pages                          # outside the pool: not written either
    skv.q8_append(h, pool, _dev(x), _dev(x), ids, kv_len)
    with pytest.raises(skv.SplitKVError, match="0x2"):
        h.status()
    assert np.array_equal(pool.k.cpu().numpy(), c.k)


# ------------------------------------------------------------------- attention

ATTN = [
    # S lens, nq, H, Hk, D, causal
    ([1], 1, 1, 1, 64, False), ([256], 1, 4, 1, 64, False), ([63, 64, 65, 0, 1], 1, 8, 2, 128, False),
    ([1000, 3, 517], 1, 10, 2, 128, False), ([300], 1, 16, 1, 128, False), ([777, 0, 12], 3, 8, 2, 64, True),
    ([130, 40], 5, 6, 2, 128, True), ([4097], 1, 40, 8, 128, False), ([2000, 64], 2, 24, 8, 64, True),
    ([90], 40, 2, 2, 128, True), ([5, 200], 9, 20, 4, 128, True), ([321], 1, 71, 1, 64, False),
]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("lens,nq,H,Hk,D,causal", ATTN)
def test_attention(h, lens, nq, H, Hk, D, causal, f16):
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(sum(lens) + H + D)
    c = u.Cache(rng, lens, Hk, D)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, len(lens), nq, H, D)
    q_pos = _causal(c, nq) if causal else None
    ref = u.attention(c, q, q_pos=q_pos)
    mass = torch.ones((len(lens), Hk, c.cap), device="cuda")
    for m in (None, mass):
        o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=None if q_pos is None else _dev(q_pos), mass=m,
                             o_dtype=torch.float16 if f16 else torch.float32)
        u.check(o, lse, ref, f16=f16)
    # a page's weight: at most nq*H/Hk probabilities, each off by e = tol_o / (2 vmax) relative, and fp32 sums
    tol = (ref[3] / (2 * ref[5]) if ref[5] else 0) * nq * H / Hk + nq * H / Hk * 2.0 ** -20 + 2.0 ** -22
    assert np.abs(mass.double().cpu().numpy() - 1.0 - ref[2]).max() <= tol
    assert h.status() == 0


# many rows a KV head: tiles of 128 rows in pairs, the last pair of some with one
PREFILL = [
    ([64], 33, 1, 1, 128, False), ([300], 64, 8, 2, 64, True), ([1000, 0, 300], 150, 8, 2, 128, True),
    ([700, 20], 33, 16, 1, 128, False), ([2000], 70, 40, 8, 64, True), ([5000, 129], 64, 8, 4, 128, True),
    ([40], 100, 6, 2, 128, True), ([260] * 9, 72, 4, 1, 64, False), ([70, 0, 131] * 100, 34, 1, 1, 64, True),
    ([65] * 1100, 33, 1, 1, 64, False),
    # units of more tiles than fp32 results take at a time, one or less of them a CTA
    ([1300, 2500] + [1300] * 38, 33, 4, 4, 64, True), ([1400] * 20, 33, 8, 8, 128, False),
    # few units of many pieces
    ([30000], 34, 3, 1, 128, True), ([17000, 0, 9000], 40, 2, 1, 64, True),
]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("lens,nq,H,Hk,D,causal", PREFILL)
def test_attention_many_rows(h, lens, nq, H, Hk, D, causal, f16):
    test_attention(h, lens, nq, H, Hk, D, causal, f16)


@pytest.mark.parametrize("f16", [False, True])
def test_many_rows_any_positions(h, f16):
    """Query positions in no order, beyond the keys and before them; absent pages."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(41)
    c = u.Cache(rng, [900, 130], 2, 128)
    c.ids[0, 0, 5] = -1
    c.ids[0, 1, 0] = c.ids[0, 1, 1] = -1
    c.ids[1, 0, :3] = -1                              # nothing at all for this head
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 2, 90, 8, 128)
    q_pos = rng.integers(-50, 1100, (2, 90)).astype(np.int32)
    ref = u.attention(c, q, q_pos=q_pos)
    mass = torch.zeros((2, 2, c.cap), device="cuda")
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(q_pos), mass=mass, o_dtype=torch.float16 if f16 else None)
    u.check(o, lse, ref, f16=f16)
    tol = (ref[3] / (2 * ref[5]) + 2.0 ** -20) * 90 * 4
    assert np.abs(mass.double().cpu().numpy() - ref[2]).max() <= tol
    assert h.status() == 0


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_absent_pages_and_far_scales(h, nq):
    """Padding inside a list, scales that differ by 2^40 and zero scales, large scores."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(11)
    c = u.Cache(rng, [700, 640, 128], 2, 128)
    c.ids[0, 0, 3] = -1
    c.ids[0, 1, 0] = -5
    c.ids[2, 1, :2] = -1                              # nothing left for this head
    c.vs *= (2.0 ** rng.integers(-40, 1, c.n_pages)).astype(np.float32)
    c.vs[c.ids[1, 0, 0]] = 0.0
    c.ks[c.ids[1, 1, 4]] = 0.0
    c.ks[c.ids[1, 0, 2]] *= 20
    c.ks[c.ids[0, 0, 1]] *= -1                        # the pool's scales may have either sign
    c.vs[c.ids[0, 1, 2]] *= -1
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 3, nq, 8, 128)
    mass = torch.zeros((3, 2, c.cap), device="cuda")
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, mass=mass)
    ref = u.attention(c, q)
    u.check(o, lse, ref)
    assert np.array_equal(mass.cpu().numpy() == 0, ref[2] < 2.0 ** -100)
    assert h.status() == 0


def test_attention_reports_bad_lists(h):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(12)
    c = u.Cache(rng, [200, 100], 1, 64, cap=4)
    c.ids[0, 0, 1] = c.n_pages + 7                    # outside the pool: reads as absent
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 2, 1, 4, 64)
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len)
    u.check(o, lse, u.attention(c, q))
    with pytest.raises(skv.SplitKVError, match="0x4"):
        h.status()
    c.ids[0, 0, 1] = -1
    c.lens[:] = [200, -3]
    o, lse = skv.q8_attn(h, pool, _dev(q), _dev(c.ids), _dev(c.lens))
    c.lens[1] = 0
    u.check(o, lse, u.attention(c, q))
    assert h.status() == 0
    long = c.lens.copy()
    long[0] = 4 * u.PAGE + 1                          # longer than its list: cut to it
    c.lens[0] = 4 * u.PAGE
    o, lse = skv.q8_attn(h, pool, _dev(q), _dev(c.ids), _dev(long))
    u.check(o, lse, u.attention(c, q))
    with pytest.raises(skv.SplitKVError, match="0x4"):
        h.status()


@pytest.mark.parametrize("lens,nq,H,Hk,D,n", [([1000, 64, 0], 1, 8, 2, 128, 5), ([640, 333], 4, 8, 1, 64, 3), ([2000], 2, 40, 2, 128, 40)])
def test_attention_over_a_selection(h, lens, nq, H, Hk, D, n):
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(n)
    c = u.Cache(rng, lens, Hk, D)
    c.ids[0, 0, 2] = -1
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, len(lens), nq, H, D)
    q_pos = _causal(c, nq)
    sel = rng.integers(-1, max(lens) // u.PAGE + 3, (len(lens), nq, Hk, n)).astype(np.int32)
    sel[0, 0, 0, 0] = sel[0, 0, 0, -1] = 1            # the same page twice counts twice
    sel[0, -1, 0, :2] = 2 ** 30                       # far behind the list
    ref = u.attention(c, q, q_pos=q_pos, sel=sel)
    mass = torch.zeros((len(lens), Hk, c.cap), device="cuda")
    runs = []
    for _ in range(2):
        mass.zero_()
        o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(q_pos), sel=_dev(sel), mass=mass)
        u.check(o, lse, ref)
        runs.append(mass.clone())
    assert torch.equal(runs[0], runs[1])
    tol = (ref[3] / (2 * ref[5]) + 2.0 ** -20) * nq * H / Hk
    assert np.abs(mass.double().cpu().numpy() - ref[2]).max() <= tol
    assert h.status() == 0


@pytest.mark.parametrize("nq,lens", [(1, [700, 0, 40]), (3, [3000, 64, 65]), (70, [700, 5, 130]), (70, [1300] * 40)])
@pytest.mark.parametrize("f16", [False, True])
def test_a_query_with_nan_gives_nan_in_its_own_row(h, nq, lens, f16):
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(nq)
    c = u.Cache(rng, lens, 2, 128)
    pool, ids, kv_len = c.on_gpu()
    q = _dev(_q(rng, len(lens), nq, 8, 128))
    pos = _dev(_causal(c, nq)) if nq > 1 else None
    o_type = torch.float16 if f16 else None
    o, lse = skv.q8_attn(h, pool, q, ids, kv_len, q_pos=pos, o_dtype=o_type)
    q[0, nq // 2, 5, 17] = float("nan")
    q[2, nq - 1, 0, 3] = float("nan")
    oo, ll = skv.q8_attn(h, pool, q, ids, kv_len, q_pos=pos, o_dtype=o_type)
    bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    bad[0, nq // 2, 5] = bad[2, nq - 1, 0] = True
    assert ll[bad].isnan().all() and oo[bad].isnan().all()
    assert torch.equal(ll[~bad], lse[~bad]) and torch.equal(oo[~bad], o[~bad])
    assert h.status() == 0


def test_fp32_results_over_long_lists(h):
    """Values of one sign, where every truncated addition loses the same way: 2^-18 of
    the largest value (u.check's bound where scores are small) over 128 tiles."""
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(62)
    c = u.Cache(rng, [16384] * 5, 8, 64)
    c.v = rng.integers(64, 128, c.v.shape).astype(np.int8)
    c.ks[:] = 1e-4
    c.vs[:] = 0.01
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 5, 33, 8, 64)
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len)
    ref = list(u.attention(c, q))
    u.check(o, lse, ref)
    assert h.status() == 0


@pytest.mark.parametrize("G,nq,sel", [(2, 600, False), (1, 30, False), (2, 600, True)])
def test_weights_in_several_launches(h, G, nq, sel):
    """Lists so long that the pages' log sums of all tokens exceed the scratch of one
    launch: results, weights and log sums as of one."""
    import split_kv_flash_attn_gb300 as skv
    import torch
    rng = np.random.default_rng(G + nq)
    cap = 65536 if nq > 30 else 1 << 21
    c = u.Cache(rng, [400], 1, 64, cap=cap)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 1, nq, G, 64)
    pos = rng.integers(-5, 450, (1, nq)).astype(np.int32)
    n_sel = 60000                                     # (with the padding)
    s = None
    if sel:
        s = np.full((1, nq, 1, n_sel), -1, np.int32)
        s[..., 1], s[..., -1] = 2, 0
    mass = torch.zeros((1, 1, cap), device="cuda")
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(pos), mass=mass, sel=None if s is None else _dev(s))
    ref = u.attention(c, q, q_pos=pos, sel=s)
    u.check(o, lse, ref)
    tol = (ref[3] / (2 * ref[5]) + 2.0 ** -20) * nq * G
    assert np.abs(mass.double().cpu().numpy() - ref[2]).max() <= tol
    assert h.status() == 0


# --------------------------------------------------------------- the selection

@pytest.mark.parametrize("lens,nq,H,Hk,D,n,first,last,causal", [
    ([1000], 1, 4, 1, 128, 4, 1, 1, False), ([5000, 64, 0, 1], 1, 8, 2, 64, 16, 0, 0, False),
    ([777, 2500], 3, 10, 2, 128, 7, 2, 2, True), ([300], 20, 4, 4, 64, 3, 1, 2, True),
    ([4096], 1, 80, 1, 64, 10, 0, 1, False), ([64 * 2000], 1, 2, 1, 64, 300, 1, 1, False), ([64 * 7000 - 3], 1, 1, 1, 64, 77, 0, 1, False),
    ([64 * 17000], 1, 1, 1, 64, 2000, 1, 2, False), ([130], 2, 8, 8, 128, 8, 1, 1, True), ([9000], 1, 2, 2, 128, 1, 0, 1, False),
    # lists at the border of what the last CTA of the scores chooses from, one of them empty, and more heads than it takes at once
    ([64 * 4092, 0, 64 * 3000 - 1], 1, 4, 2, 128, 500, 1, 1, False), ([64 * 4095], 1, 1, 1, 64, 4000, 0, 1, False),
    ([64 * 900, 5], 1, 130, 1, 64, 20, 0, 0, True)])
def test_selection(h, lens, nq, H, Hk, D, n, first, last, causal):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(sum(lens) + n)
    c = u.Cache(rng, lens, Hk, D)
    if c.cap > 8:
        c.ids[0, 0, 3] = -1                           # absent
        c.ids[0, 0, 6] = c.ids[0, 0, 4]               # the same page twice: the same score
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, len(lens), nq, H, D)
    q[0, 0, 0] = 0                                    # a query of zeros: all its bounds are 0
    if H // Hk == 1:
        q[0, 0] = 0                                   # ... for every head: all ties
    q_pos = _causal(c, nq) if causal else None
    got = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=n, n_first=first, n_last=last,
                        q_pos=None if q_pos is None else _dev(q_pos))
    want = u.select(c, q, n, first, last, q_pos)
    assert np.array_equal(got.cpu().numpy(), want)
    assert h.status() == 0


def test_selection_of_many_tokens_in_long_lists(h):
    """More keys than the scratch of one launch holds: the tokens go in several."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(9)
    S, nq, H, D, cap = 2, 700, 2, 64, 65536
    c = u.Cache(rng, [700, 333], 1, D, cap=cap)
    pool, ids, kv_len = c.on_gpu()
    q = _dev(_q(rng, S, nq, H, D))
    pos = _dev(rng.integers(-5, 800, (S, nq)).astype(np.int32))
    got = skv.q8_select(h, pool, q, ids, kv_len, n_sel=4, q_pos=pos)
    for t in (0, 255, 511, 512, 513, 699):            # token by token, the same
        one = skv.q8_select(h, pool, q[:, t:t + 1].contiguous(), ids, kv_len, n_sel=4, q_pos=pos[:, t:t + 1].contiguous())
        assert torch.equal(got[:, t:t + 1], one), t
    want = u.select(c, q[:, -3:].cpu().numpy(), 4, 1, 1, pos[:, -3:].cpu().numpy())
    assert np.array_equal(got[:, -3:].cpu().numpy(), want)
    assert h.status() == 0


def test_selection_bounds_every_score(h):
    """The bound is one: the page of the best key under the coded query is always picked."""
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(3)
    c = u.Cache(rng, [64 * 40], 1, 128)
    c.ks[:] = 0.03
    best = 17
    q = _q(rng, 1, 1, 1, 128)
    cq = u.code(q[0, 0, 0], np.float32(np.abs(q).astype(np.float64).max() / 127))
    c.k[c.ids[0, 0, best], 9] = np.clip(cq.astype(int) * 2, -127, 127)   # one key along the query
    c.extremes()
    pool, ids, kv_len = c.on_gpu()
    got = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=8, n_first=0, n_last=0).cpu().numpy()[0, 0, 0]
    scores = np.array([(c.k[p].astype(int) @ cq.astype(int)).max() for p in c.ids[0, 0, :40]])
    bounds = np.array([np.maximum(cq.astype(int) * c.lo[p].astype(int), cq.astype(int) * c.hi[p].astype(int)).sum()
                       for p in c.ids[0, 0, :40]])
    assert np.all(bounds >= scores)
    assert np.all(np.sort(bounds)[::-1][:8] == np.sort(bounds[got])[::-1])


# ------------------------------------------------------------------- evictions

@pytest.mark.parametrize("lens,Hk,cap,keep,first,last", [
    ([64 * 20], 1, 25, 5, 1, 1), ([1000, 64, 0, 63, 5000], 2, 90, 8, 2, 3), ([700], 3, 11, 1, 0, 1), ([700], 3, 11, 11, 0, 2),
    ([64 * 3000 - 5, 64 * 1500], 2, 3000, 700, 1, 4), ([64 * 49000, 64 * 10], 1, 49500, 200, 1, 1),
    ([64 * 9000, 64 * 16000 - 1], 1, 16384, 5000, 3, 3), ([64 * 1024], 2, 1024, 1023, 1, 1), ([64 * 6000], 1, 6144, 2, 1, 1)])
def test_eviction(h, lens, Hk, cap, keep, first, last):
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(keep + cap)
    S = len(lens)
    ids = rng.permutation(S * Hk * cap).astype(np.int32).reshape(S, Hk, cap)
    ids[rng.random(ids.shape) < 0.1] = -1
    mass = rng.choice(np.array([0.0, -0.0, 0.25, 1.0, np.inf, np.nan, 3.5], np.float32), ids.shape)
    mass = np.where(rng.random(ids.shape) < 0.5, mass, rng.random(ids.shape)).astype(np.float32)
    got = skv.q8_evict(h, _dev(ids), _dev(mass), _dev(np.array(lens, np.int32)), n_keep=keep, n_first=first, n_last=last)
    want = u.evict(ids, mass, lens, keep, first, last)
    for name, a, b in zip(("page_ids", "mass", "kv_len", "freed"), got, want):
        assert np.array_equal(a.cpu().numpy(), b, equal_nan=name == "mass"), name
    assert h.status() == 0


# ------------------------------------------------------------- the calls together

def test_a_server_s_steps(h):
    """Prompt, decode steps with accumulated weight, sparse steps, eviction, reuse of the freed pages."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(77)
    Hk, H, D, S = 2, 8, 128, 2
    c = u.Cache(rng, [0, 0], Hk, D, extra=1400, spare=0)
    pool, ids, kv_len = c.on_gpu()
    pool.k.fill_(99)                                  # pages need not be cleared
    pool.k_scale.fill_(7.0)
    c.k[:], c.ks[:] = 99, 7.0
    mass = torch.zeros((S, Hk, c.cap), device="cuda")
    ref_mass = np.zeros((S, Hk, c.cap))

    def append(n, n_new=None):
        x = rng.standard_normal((2, S, n, Hk, D)).astype(np.float16)
        skv.q8_append(h, pool, _dev(x[0]), _dev(x[1]), ids, kv_len, n_new=None if n_new is None else _dev(n_new))
        u.append(c, x[0], x[1], n_new)
        kv_len.add_(n if n_new is None else _dev(n_new))
        c.lens += n if n_new is None else n_new

    append(700, np.array([700, 333], np.int32))
    q = _q(rng, S, 30, H, D)                          # the prompt's last tokens
    pos = _causal(c, 30)
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(pos), mass=mass)
    ref = u.attention(c, q, q_pos=pos)
    u.check(o, lse, ref)
    ref_mass += ref[2]
    for step in range(4):
        append(1)
        q = _q(rng, S, 1, H, D)
        sel = None
        if step % 2:
            sel = skv.q8_select(h, pool, _dev(q), ids, kv_len, n_sel=4)
            assert np.array_equal(sel.cpu().numpy(), u.select(c, q, 4, 1, 1))
        o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, sel=sel, mass=mass)
        ref = u.attention(c, q, sel=None if sel is None else sel.cpu().numpy())
        u.check(o, lse, ref)
        ref_mass += ref[2]
    assert np.allclose(mass.cpu().numpy(), ref_mass, rtol=1e-4, atol=1e-4)
    m = mass.cpu().numpy()
    ids2, mass2, len2, freed = skv.q8_evict(h, ids, mass, kv_len, n_keep=6, n_first=1, n_last=2)
    w = u.evict(c.ids, m, c.lens, 6, 1, 2)
    for a, b in zip((ids2, mass2, len2, freed), w):
        assert np.array_equal(a.cpu().numpy(), b)
    c.ids, c.lens = w[0], w[2]
    ids, kv_len = ids2, len2
    # the freed pages go behind what each list still holds
    for s in range(S):
        for k in range(Hk):
            free = w[3][s, k][w[3][s, k] >= 0]
            row = c.ids[s, k]
            n = int((row >= 0).sum())
            assert np.all(row[:n] >= 0)
            row[n:n + len(free)] = free
    ids.copy_(_dev(c.ids))
    append(200)
    q = _q(rng, S, 2, H, D)
    pos = _causal(c, 2)
    o, lse = skv.q8_attn(h, pool, _dev(q), ids, kv_len, q_pos=_dev(pos))
    u.check(o, lse, u.attention(c, q, q_pos=pos))
    assert h.status() == 0


def test_partitions_merge(h):
    """8-bit pages for old tokens and fp16 rows for recent ones: two partials, one combine."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(8)
    Hk, H, D = 2, 8, 128
    c = u.Cache(rng, [500], Hk, D)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 1, 1, H, D)
    K = rng.standard_normal((100, Hk, D)).astype(np.float16)
    V = rng.standard_normal((100, Hk, D)).astype(np.float16)
    o1, l1 = skv.q8_attn(h, pool, _dev(q), ids, kv_len)
    o2, l2 = skv.attn_partial(h, _dev(q), _dev(K.reshape(100, -1)), _dev(V.reshape(100, -1)), Hk=Hk)
    o, lse = skv.attn_combine(h, torch.stack([o1.view(H, D), o2.view(H, D)]), torch.stack([l1.view(H), l2.view(H)]))
    ro, rl, _, tol, tol_l, vmax = u.attention(c, q)
    for x in range(H):
        k = x // (H // Hk)
        w = K[:, k].astype(np.float64) @ q[0, 0, x].astype(np.float64) / np.sqrt(D)
        z = np.logaddexp(rl[0, 0, x], np.logaddexp.reduce(w))
        want = np.exp(rl[0, 0, x] - z) * ro[0, 0, x] + np.exp(w - z) @ V[:, k].astype(np.float64)
        assert np.abs(o[x].double().cpu().numpy() - want).max() <= tol + 2e-3 * max(vmax, np.abs(V).max())
        assert abs(lse[x].item() - z) <= tol_l + 1e-4


# ----------------------------------------------------------- streams and graphs

def test_graph_replays_follow_the_inputs(h):
    """A captured step replayed on other lengths, queries and lists, with a graph
    captured before and one after the workspace grew."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(21)
    hh = skv.Handle(0)
    Hk, H, D = 2, 8, 128
    c = u.Cache(rng, [400, 900], Hk, D)
    pool, ids, kv_len = c.on_gpu()
    q = _dev(_q(rng, 2, 1, H, D))
    mass = torch.zeros((2, Hk, c.cap), device="cuda")

    def step():
        sel = skv.q8_select(hh, pool, q, ids, kv_len, n_sel=5)
        return skv.q8_attn(hh, pool, q, ids, kv_len, sel=sel) + skv.q8_attn(hh, pool, q, ids, kv_len, mass=mass) + (sel,)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    hh.reserve(64 << 20)                              # the workspace moves; the graph keeps its own
    junk = torch.full((32 << 20,), 1.0, device="cuda")
    for lens in ([400, 900], [1, 0], [833, 64]):
        c.lens[:] = lens
        c.extremes()
        pool.k_min.copy_(_dev(c.lo))
        pool.k_max.copy_(_dev(c.hi))
        kv_len.copy_(_dev(c.lens))
        qq = _q(rng, 2, 1, H, D)
        q.copy_(_dev(qq))
        g.replay()
        torch.cuda.synchronize()
        want = u.select(c, qq, 5, 1, 1)
        assert np.array_equal(out[4].cpu().numpy(), want)
        u.check(out[0], out[1], u.attention(c, qq, sel=want))
        u.check(out[2], out[3], u.attention(c, qq))
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    del junk
    assert hh.status() == 0
    hh.close()


def test_a_captured_prompt_step(h):
    """Append, attention of many rows in fp32 and fp16, weights and eviction in one graph,
    replayed on other tokens and lengths."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(25)
    hh = skv.Handle(0)
    Hk, H, D, n = 2, 8, 128, 70
    c = u.Cache(rng, [300, 1100], Hk, D, extra=n)
    pool, ids, kv_len = c.on_gpu()
    after = kv_len + n
    x = torch.zeros((2, 2, n, Hk, D), dtype=torch.float16, device="cuda")
    q = torch.zeros((2, n, H, D), dtype=torch.float16, device="cuda")
    pos = torch.zeros((2, n), dtype=torch.int32, device="cuda")
    mass = torch.zeros((2, Hk, c.cap), device="cuda")

    def step():
        skv.q8_append(hh, pool, x[0], x[1], ids, kv_len)
        a = skv.q8_attn(hh, pool, q, ids, after, q_pos=pos, mass=mass)
        b = skv.q8_attn(hh, pool, q, ids, after, q_pos=pos, o_dtype=torch.float16)
        return a + b + skv.q8_evict(hh, ids, mass, after, n_keep=6, n_first=1, n_last=2)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for lens in ([300, 1100], [0, 63], [129, 640]):
        c.lens[:] = lens
        kv_len.copy_(_dev(c.lens))
        xx = rng.standard_normal((2, 2, n, Hk, D)).astype(np.float16)
        x.copy_(_dev(xx))
        c.k, c.v, c.ks, c.vs = (t.cpu().numpy().copy() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale))
        u.append(c, xx[0], xx[1])
        c.lens += n
        after.copy_(_dev(c.lens))
        qq, pp = _q(rng, 2, n, H, D), _causal(c, n)
        q.copy_(_dev(qq))
        pos.copy_(_dev(pp))
        mass.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(pool.k.cpu().numpy(), c.k) and np.array_equal(pool.v_scale.cpu().numpy(), c.vs)
        ref = u.attention(c, qq, q_pos=pp)
        u.check(out[0], out[1], ref)
        u.check(out[2], out[3], ref, f16=True)
        for a, b in zip(out[4:], u.evict(c.ids, mass.cpu().numpy(), c.lens, 6, 1, 2)):
            assert np.array_equal(a.cpu().numpy(), b)
    assert hh.status() == 0
    hh.close()


def test_two_handles_on_two_streams_at_once(h):
    """Calls that overlap on the GPU, each with its handle: the results of one after the other."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(26)
    hh = skv.Handle(0)
    jobs = []
    for hd, lens, nq in ((h, [9000, 4000, 1], 1), (hh, [3000, 7000], 70)):
        c = u.Cache(rng, lens, 4, 128)
        pool, ids, kv_len = c.on_gpu()
        q, pos = _dev(_q(rng, len(lens), nq, 16, 128)), _dev(_causal(c, nq))

        def job(hd=hd, pool=pool, ids=ids, kv_len=kv_len, q=q, pos=pos):
            sel = skv.q8_select(hd, pool, q, ids, kv_len, n_sel=9, q_pos=pos)
            return (sel, *skv.q8_attn(hd, pool, q, ids, kv_len, q_pos=pos),
                    *skv.q8_attn(hd, pool, q, ids, kv_len, q_pos=pos, sel=sel))
        jobs.append((job, torch.cuda.Stream()))
    want = [job() for job, _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (job, st) in enumerate(jobs):
            with torch.cuda.stream(st):
                got[i].append(job())
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))
    assert h.status() == 0 and hh.status() == 0
    hh.close()


def test_capture_does_not_grow_scratch():
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(22)
    hh = skv.Handle(0)
    c = u.Cache(rng, [400], 1, 64)
    pool, ids, kv_len = c.on_gpu()
    q = _dev(_q(rng, 1, 1, 4, 64))
    g = torch.cuda.CUDAGraph()
    o = torch.empty((1, 1, 4, 64), device="cuda")
    lse = torch.empty((1, 1, 4), device="cuda")
    err = None
    with torch.cuda.graph(g):
        o.zero_()
        try:
            skv.q8_attn(hh, pool, q, ids, kv_len, o=o, lse=lse)
        except skv.SplitKVError as e:
            err = e
    assert err is not None and "SKV_ECAPTURE" in str(err)
    hh.close()


def test_runs_on_the_stream_it_is_given(h):
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(23)
    c = u.Cache(rng, [1500], 2, 128)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 1, 1, 8, 128)
    qd, zero = _dev(q), torch.zeros((1, 1, 8, 128), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.zeros(64 << 20, device="cuda")
        for _ in range(10):
            big.add_(1.0)                             # holds the stream for a while
        zero.copy_(qd)
        o, lse = skv.q8_attn(h, pool, zero, ids, kv_len)
    s.synchronize()
    u.check(o, lse, u.attention(c, q))


@pytest.mark.parametrize("raw", [False, True])
def test_results_belong_to_the_stream_of_the_call(h, raw):
    """Memory freed on the current stream, on which work with it is still queued, is
    not what a call on another stream writes its results to."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(24)
    c = u.Cache(rng, [640], 2, 128)
    pool, ids, kv_len = c.on_gpu()
    q = _q(rng, 1, 1, 8, 128)
    qd = _dev(q)
    mass = torch.rand((1, 2, c.cap), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    big = torch.zeros(64 << 20, device="cuda")
    old = [torch.empty(1024 * k, device="cuda") for k in (1, 2, 4) for _ in range(4)]
    for _ in range(20):
        big.add_(1.0)
    for x in old:
        x.fill_(7.0)                                  # behind big's additions
    del old, x
    st = s.cuda_stream if raw else s
    sel = skv.q8_select(h, pool, qd, ids, kv_len, n_sel=4, stream=st)
    o, lse = skv.q8_attn(h, pool, qd, ids, kv_len, stream=st)
    kept = skv.q8_evict(h, ids, mass, kv_len, n_keep=6, stream=st)
    torch.cuda.synchronize()
    assert np.array_equal(sel.cpu().numpy(), u.select(c, q, 4, 1, 1))
    u.check(o, lse, u.attention(c, q))
    for a, b in zip(kept, u.evict(c.ids, mass.cpu().numpy(), c.lens, 6, 1, 1)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_offsets_beyond_32_bits(h):
    """A pool whose codes pass 2^31 bytes, read and written at its end."""
    import torch
    import split_kv_flash_attn_gb300 as skv
    rng = np.random.default_rng(31)
    n = (1 << 31) // (64 * 128) + 40
    small = u.Cache(rng, [500], 1, 128, extra=70, shuffle=False, spare=0)
    pool = skv.Q8Pool.empty(n, 128)
    off = n - small.n_pages
    for name, x in (("k", small.k), ("v", small.v), ("k_scale", small.ks), ("v_scale", small.vs), ("k_min", small.lo), ("k_max", small.hi)):
        getattr(pool, name)[off:] = _dev(x)
    ids = small.ids.copy()
    ids[ids >= 0] += off
    x = rng.standard_normal((2, 1, 70, 1, 128)).astype(np.float32)
    kv_len = _dev(small.lens)
    skv.q8_append(h, pool, _dev(x[0]), _dev(x[1]), _dev(ids), kv_len)
    u.append(small, x[0], x[1])
    small.lens += 70
    kv_len += 70
    assert np.array_equal(pool.k[off:].cpu().numpy(), small.k)
    q = _q(rng, 1, 1, 4, 128)
    sel = skv.q8_select(h, pool, _dev(q), _dev(ids), kv_len, n_sel=3)
    assert np.array_equal(sel.cpu().numpy(), u.select(small, q, 3, 1, 1))
    o, lse = skv.q8_attn(h, pool, _dev(q), _dev(ids), kv_len)
    u.check(o, lse, u.attention(small, q))
    assert h.status() == 0
    del pool
    torch.cuda.empty_cache()

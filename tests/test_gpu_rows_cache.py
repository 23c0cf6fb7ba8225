"""Rows into caches by skv.rope_append, byte for byte what rope (fp32 results) and kv_append store: layouts of the cache,
orders of pairs and types of rows that differ in how a lane's values reach their places."""
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


def _case(skv, n, H, Hk, D, R, axes, dtype, inter, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 101 + n + D + R)
    x = (torch.randn((n, H + 2 * Hk, D), device="cuda", generator=g) * 3).to(dtype)
    pos = torch.randint(0, 10000, (axes, n), device="cuda", generator=g).to(torch.int32)
    half = R // 2
    freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))).float()
    axis = torch.randint(0, axes, (half,), device="cuda", generator=g).to(torch.int32) if axes > 1 else None
    w = [1 + 0.3 * torch.randn(D, device="cuda", generator=g) for _ in "qk"]
    return skv.Rope(D, freq, axis=axis, n_axes=axes, interleaved=inter), x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], pos, w, g


def test_parts_of_a_packed_cache(skv, h):
    """K and V side by side in one cache [rows, 2, Hk, D], each with the cache's pitch; positions up to its last row."""
    import torch
    n, H, Hk, D, rows = 41, 4, 2, 64, 50
    spec, q, k, v, pos, w, g = _case(skv, n, H, Hk, D, D, 1, torch.float16, False)
    at = torch.randperm(rows, device="cuda", generator=g)[:n].to(torch.int32)
    at[0], pitch = rows - 1, 4 * Hk * D
    at[1:] = torch.where(at[1:] == rows - 1, -1, at[1:])
    packed = torch.full((rows, 2, Hk, D), 7.0, dtype=torch.float16, device="cuda")
    K, V = (torch.full((rows, Hk, D), 7.0, dtype=torch.float16, device="cuda") for _ in "kv")
    a = skv.rope_append(h, spec, q, k, v, pos, at, packed[:, 0], packed[:, 1], k_weight=w[1], k_row_bytes=pitch, v_row_bytes=pitch)
    b = skv.rope_append(h, spec, q, k, v, pos, at, K, V, k_weight=w[1])
    assert h.status() == 0
    assert torch.equal(a, b) and torch.equal(packed[:, 0], K) and torch.equal(packed[:, 1], V)
    assert int((K != 7).any(-1).any(-1).sum()) == int((at >= 0).sum())
    o = [skv.attn_partial(h, a.view(1, n, H, D), x, y, Hk=Hk, kv_end=rows, k_row_bytes=p, v_row_bytes=p)
         for x, y, p in ((packed[:, 0], packed[:, 1], pitch), (K, V, pitch // 2))]
    assert torch.equal(o[0][0], o[1][0]) and torch.equal(o[0][1], o[1][1])


# n, H, Hk, D, R, axes, interleaved, norm: partial rotation moves a lane's two groups of four apart in another pattern for each R
FORMS = [
    (37, 3, 2, 128, 128, 1, True, True),
    (37, 2, 5, 64, 64, 3, True, False),
    (65, 4, 2, 128, 96, 1, False, True),
    (33, 1, 3, 128, 8, 2, False, True),
    (20, 2, 2, 64, 16, 4, False, False),
    (45, 2, 1, 64, 38, 1, True, True),           # an odd number of pairs
    (9, 0, 2, 128, 0, 1, False, True),           # no rotation
    (70, 2, 2, 64, 0, 1, True, True),
    (1, 8, 2, 128, 64, 3, False, True),
]


@pytest.mark.parametrize("xt", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("kt,vt,pad", [("F16", "F16", 0), ("F16", "F16", 4), ("Q8_0", "Q4_0", 2), ("Q4_0", "Q8_0", 0), ("F16", "Q8_0", 12)])
@pytest.mark.parametrize("n,H,Hk,D,R,axes,inter,norm", FORMS)
def test_forms_store_what_rope_and_kv_append_store(skv, h, n, H, Hk, D, R, axes, inter, norm, kt, vt, pad, xt):
    """Rows `pad` bytes longer than their heads too (fp16 rows of 4-byte alignment, blocks at any even byte): what stands
    between them stays."""
    import torch
    spec, q, k, v, pos, w, g = _case(skv, n, H, Hk, D, R, axes, getattr(torch, xt), inter, seed=3)
    rows0, rows1 = 40, 60
    at = torch.randperm(rows0 + rows1, device="cuda", generator=g)[:n].to(torch.int32)
    if n > 10:
        at[3], pos[0, 5] = -1, -7
    kt, vt = getattr(skv, kt), getattr(skv, vt)
    step = [Hk * skv.segment_bytes(t, D) + pad for t in (kt, vt)]

    def caches():
        out = []
        for s in step:
            out += [torch.full((rows0, s), 0x5a, dtype=torch.uint8, device="cuda"), torch.full((rows1, s), 0x5a, dtype=torch.uint8).pin_memory()]
        return out

    a, b = caches(), caches()
    wq, wk = (w[0] if norm and H else None), (w[1] if norm else None)
    got = skv.rope_append(h, spec, q if H else None, k, v, pos, at, a[0], a[2], a[1], a[3], q_weight=wq, k_weight=wk, k_type=kt, v_type=vt,
                          k_row_bytes=step[0], v_row_bytes=step[1])
    yq, yk = skv.rope(h, spec, q if H else None, k, pos, q_weight=wq, k_weight=wk, o_dtype=torch.float32)
    at2 = torch.where(pos[0] < 0, -1, at).to(torch.int32)
    skv.kv_append(h, yk, at2, b[0], b[1], type_=kt, row_bytes=step[0])
    skv.kv_append(h, v.float().contiguous(), at2, b[2], b[3], type_=vt, row_bytes=step[1])
    assert h.status() == 0
    for s, t in zip(a, b):
        assert torch.equal(s.cpu(), t.cpu())
    for i, s in enumerate(step):
        if pad:
            assert (a[2 * i][:, s - pad:] == 0x5a).all() and (a[2 * i + 1][:, s - pad:] == 0x5a).all()
    assert got is None if not H else torch.equal(got, yq.half())
    assert int(sum((x.cpu() != 0x5a).any(1).sum() for x in a[:2])) == int((at2 >= 0).sum())


def test_a_replayed_graph_turns_what_its_inputs_hold_then(skv):
    """Rows doubled after the capture: normed rows stay what they were, their gradients halve.  A replay that went by the
    old rows would leave these.  The power of two changes no rounding; eps (1e-6 beside a mean square of 4 and more) shifts
    1/rms by less than 2^-22, and two rounded results of nearly the same value lie within two halves of a step: 2^-10 of
    the value (2^-24 below the normal range), and 2^-18 of the magnitudes that fp32 sums and products go through."""
    import torch
    h = skv.Handle(0)
    spec, q, k, v, pos, w, g = _case(skv, 300, 8, 2, 128, 128, 1, torch.float16, False, seed=5)
    base = torch.cat((q, k), 1)
    q, k = base[:, :8], base[:, 8:]
    dy = [torch.randn(t.shape, device="cuda", generator=g).half() for t in (q, k)]
    side = torch.cuda.Stream()

    def both():
        a = skv.rope(h, spec, q, k, pos, q_weight=w[0], k_weight=w[1], stream=side)
        return a + skv.rope_backward(h, spec, dy[0], dy[1], pos, q=q, k=k, q_weight=w[0], k_weight=w[1], stream=side)

    torch.cuda.synchronize()
    ref = both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
        out = both()
    base.mul_(2)
    for x in out:
        x.fill_(7)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    again = both()
    torch.cuda.synchronize()
    for x, y in zip(again, out):
        assert torch.equal(x, y)
    half = [x.double() / 2 for x in (q, k)]                  # the rows as they were
    for i in (0, 1):
        y, z = ref[i].double(), out[i].double()
        assert ((z - y).abs() <= y.abs() * 2.0 ** -10 + 2.0 ** -24 + (y.abs() + y.roll(64, -1).abs()) * 2.0 ** -18).all()
    for i in (0, 1):
        r = 1 / torch.sqrt(half[i].square().mean(-1, keepdim=True) + 1e-6)
        assert float(r.max()) < 0.5
        u, xr = (dy[i].double().abs() + dy[i].double().roll(64, -1).abs()) * w[i].double().abs(), half[i].abs() * r
        size = r * (u + xr * (u * xr).mean(-1, keepdim=True))
        y, z = ref[2 + i].double() / 2, out[2 + i].double()
        assert ((z - y).abs() <= y.abs() * 2.0 ** -10 + 2.0 ** -24 + size * 2.0 ** -18).all()
        assert float((z - 2 * y).norm()) > 0.4 * float((2 * y).norm())
    h.close()

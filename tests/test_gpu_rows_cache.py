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

"""A bit that one call leaves in the device status word (an append beyond its cache) does not end the waits of later calls:
their results are those of a clear word, bit for bit, until the word is read."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import split_kv_flash_attn_gb300 as m
    return m


def _rows(skv, t, n, Hk, D, g):
    """A cache of n rows of a type, filled by kv_append."""
    import torch
    h = skv.Handle(0)
    out = torch.zeros((n, Hk * skv.segment_bytes(t, D)), dtype=torch.uint8, device="cuda")
    skv.kv_append(h, torch.randn((n, Hk, D), device="cuda", generator=g), torch.arange(n, device="cuda", dtype=torch.int32), out, type_=t)
    assert h.status() == 0
    h.close()
    return out


CASES = [
    # query tokens, K type, V type, by a list
    (256, "F16", "F16", False),              # TMA tiles
    (256, "F16", "F16", True),               # copied rows
    (256, "Q8_0", "Q8_0", False),            # decoded rows
    (256, "Q8_0", "Q4_0", False),            # two query tiles a CTA
    (1, "Q8_0", "Q4_0", False),              # whole rows of one token
    (1, "F16", "F16", True),
]


@pytest.mark.parametrize("nq,kt,vt,lists", CASES)
def test_attention_after_an_append_beyond_the_cache(skv, nq, kt, vt, lists):
    import torch
    S, n, H, Hk, D = 1, 6000, 32, 8, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(nq + n)
    kt, vt = getattr(skv, kt), getattr(skv, vt)
    K, V = _rows(skv, kt, n, Hk, D, g), _rows(skv, vt, n, Hk, D, g)
    q = torch.randn((S, nq, H, D), device="cuda", generator=g).half()
    rows = torch.randperm(n, device="cuda", generator=g).to(torch.int32).view(1, n) if lists else None
    h = skv.Handle(0)

    def call():
        return skv.attn_partial(h, q, K, V, Hk=Hk, k_type=kt, v_type=vt, kv_rows=rows, kv_end=n)

    ref = call()
    assert h.status() == 0
    one = torch.zeros((1, Hk, D), device="cuda")
    skv.kv_append(h, one, torch.tensor([n], dtype=torch.int32, device="cuda"), K.clone(), type_=kt)
    got = [call() for _ in range(3)]
    with pytest.raises(skv.SplitKVError) as e:
        h.status()
    assert e.value.status == 8                               # the append's bit, and no wait that gave up
    for o, lse in got:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert h.status() == 0
    h.close()

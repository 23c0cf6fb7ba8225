"""The calls over 8-bit pages at their edges, against definitions in 64 bits: scales of
either sign, rows beside pages that they do not see, rows that one key decides, lengths
beyond their lists, and the borders between the forms of the choice."""
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

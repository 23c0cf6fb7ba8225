"""What the Python calls for rows around attention say of tensors' memory before anything is launched: rows, positions and
cache regions whose strides, shapes or types do not hold what the call would read or write.  On CPU tensors, with a library
that records its arguments."""
import pytest

torch = pytest.importorskip("torch")

import split_kv_flash_attn_gb300 as skv
from split_kv_flash_attn_gb300 import _lib

F16, F32, I32, U8 = torch.float16, torch.float32, torch.int32, torch.uint8


class Handle:
    device, _h, ptr = -1, None, None

    def check(self, rc):
        assert rc == 0


class Lib:
    """Stands for the library: keeps each call's arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture()
def lib(monkeypatch):
    x = Lib()
    monkeypatch.setattr(_lib, "lib", lambda: x)
    return x


def refused(f, *args, **kw):
    with pytest.raises(skv.SplitKVError) as e:
        f(*args, **kw)
    assert e.value.status == 1
    return str(e.value)


# (storage shape, shape, strides, leading shape): tokens that are broadcast, or lie closer together than their heads
BROADCAST = [
    ((1, 1, 4, 128), (2, 5, 4, 128), (0, 0, 128, 1), (2, 5)),
    ((2, 1, 4, 128), (2, 5, 4, 128), (512, 0, 128, 1), (2, 5)),
    ((1, 5, 4, 128), (2, 5, 4, 128), (0, 512, 128, 1), (2, 5)),
    ((1, 4, 128), (5, 4, 128), (0, 128, 1), (5,)),
    ((1, 1, 128), (5, 1, 128), (0, 128, 1), (5,)),
    ((1, 1, 128), (5, 1, 128), (0, 0, 1), (5,)),
    ((2, 1, 1, 128), (2, 1, 1, 128), (0, 128, 128, 1), (2, 1)),
    ((9, 128), (5, 4, 128), (128, 128, 1), (5,)),            # overlapping windows of heads
    ((16, 128), (5, 4, 128), (256, 128, 1), (5,)),
]


@pytest.mark.parametrize("store,shape,strides,lead", BROADCAST)
def test_tokens_that_overlap_are_refused(lib, store, shape, strides, lead):
    base = torch.zeros(store, dtype=F16)
    x = base.flatten().as_strided(shape, strides)
    refused(skv._token_rows, "q", x, lead, 128, F16, -1)
    spec, pos = skv.Rope(128, torch.zeros(64)), torch.zeros(lead, dtype=I32)
    whole = torch.zeros(shape, dtype=F16)
    K = torch.zeros((64, shape[-2] * 128), dtype=F16)
    for q, k in ((x, whole), (whole, x), (x, None), (None, x)):
        refused(skv.rope, Handle(), spec, q, k, pos, stream=0)
    refused(skv.rope_append, Handle(), spec, x, whole, whole, pos, pos, K, K, stream=0)
    refused(skv.rope_append, Handle(), spec, None, whole, x, pos, pos, K, K, stream=0)
    refused(skv.rope_backward, Handle(), spec, whole, None, pos, dq=x, stream=0)
    refused(skv.rope_backward, Handle(), spec, None, whole, pos, k=x, k_weight=torch.zeros(128), stream=0)
    assert not lib.calls


def test_token_strides_that_hold_their_heads():
    """One token may have any stride; packed, padded and single rows have theirs."""
    x = torch.zeros((5, 9, 128), dtype=F16)
    rows = skv._token_rows
    assert rows("q", x, (5,), 128, F16, -1) == (9, 9 * 128)
    assert rows("q", x[:, 2:5], (5,), 128, F16, -1) == (3, 9 * 128)
    assert rows("q", x[::2, :4], (3,), 128, F16, -1) == (4, 18 * 128)
    assert rows("q", x[:1].expand(1, 9, 128), (1,), 128, F16, -1)[0] == 9
    one = torch.zeros((1, 1, 4, 128), dtype=F16)
    assert rows("q", one, (1, 1), 128, F16, -1) == (4, 512)
    assert rows("q", one[0].as_strided((1, 4, 128), (0, 128, 1)), (1,), 128, F16, -1)[0] == 4
    assert rows("q", x[:, :1], (5,), 128, F16, -1) == (1, 9 * 128)
    assert rows("q", x[:0], (0,), 128, F16, -1)[0] == 9
    assert rows("q", x[:, :0], (5,), 128, F16, -1)[0] == 0

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


def _append(lib, Hk=2, D=64, n=3, **kw):
    """rope_append of n tokens; the recorded cache regions (type, row bytes, address and rows of both) of k and v."""
    x = torch.zeros((n, Hk, D), dtype=F16)
    args = dict(k_dst0=None, v_dst0=None, stream=0)
    args.update(kw)
    at = torch.zeros((n,), dtype=I32)
    skv.rope_append(Handle(), skv.Rope(D, torch.zeros(D // 2)), None, x, x, at, at, **args)
    name, a = lib.calls[-1]
    assert name == "skv_rope_append"
    return [tuple(getattr(d._obj, f) for f in ("type", "row_bytes", "dst0", "n_rows0", "dst1", "n_rows1")) for d in (a[17], a[18])]


def test_cache_regions_as_tensors_hold_them(lib):
    Hk, D, row = 2, 64, 256
    kv = torch.zeros((10, 2, Hk, D), dtype=F16)
    K, V = kv[:, 0], kv[:, 1]
    flat = torch.zeros(10 * row, dtype=U8)
    # contiguous regions of any shape, their rows counted by bytes
    k, v = _append(lib, k_dst0=flat, v_dst0=torch.zeros((7, Hk, D), dtype=F16), k_dst1=flat[:5 * row])
    assert k == (skv.F16, row, flat.data_ptr(), 10, flat.data_ptr(), 5) and v[1] == row and v[3:] == (7, None, 0)
    # parts of a packed cache, with their pitch: every row of them
    k, v = _append(lib, k_dst0=K, v_dst0=V, k_row_bytes=2 * row, v_row_bytes=2 * row)
    assert k == (skv.F16, 2 * row, K.data_ptr(), 10, None, 0) and v == (skv.F16, 2 * row, V.data_ptr(), 10, None, 0)
    assert V.data_ptr() == K.data_ptr() + row
    # every other row, one row, none
    assert _append(lib, k_dst0=K[::2], v_dst0=V[:5], k_row_bytes=4 * row, v_row_bytes=2 * row)[0][3] == 5
    assert _append(lib, k_dst0=K[:1], v_dst0=V[:0], k_row_bytes=2 * row, v_row_bytes=2 * row)[1][3] == 0
    # an explicit count up to the memory's end, whose last row needs no padding behind it
    assert _append(lib, k_dst0=K, v_dst0=V, k_row_bytes=2 * row, v_row_bytes=2 * row, n_rows0=10)[1][3] == 10
    assert _append(lib, k_dst0=flat, v_dst0=flat, n_rows0=4)[0][3] == 4
    q8, q4 = (torch.zeros((9, Hk * skv.segment_bytes(t, D)), dtype=U8) for t in (skv.Q8_0, skv.Q4_0))
    k, v = _append(lib, k_dst0=q8, v_dst0=q4, k_type=skv.Q8_0, v_type=skv.Q4_0)
    assert k[:2] == (skv.Q8_0, 136) and v[:2] == (skv.Q4_0, 72) and k[3] == v[3] == 9


def test_cache_regions_that_would_be_written_wrongly_are_refused(lib):
    Hk, D, row = 2, 64, 256
    kv = torch.zeros((10, 2, Hk, D), dtype=F16)
    K, V, good = kv[:, 0], kv[:, 1], torch.zeros((10, Hk, D), dtype=F16)
    flat = torch.zeros(10 * row, dtype=U8)
    bad = [
        dict(k_dst0=K, v_dst0=good), dict(k_dst0=good, v_dst0=V),                    # a pitch that the call does not know of
        dict(k_dst0=K, v_dst0=good, n_rows0=10),
        dict(k_dst0=good, v_dst0=good, k_dst1=K), dict(k_dst0=good, v_dst0=good, v_dst1=V),
        dict(k_dst0=K, v_dst0=good, k_row_bytes=row), dict(k_dst0=K, v_dst0=good, k_row_bytes=3 * row),      # another one than the tensor's
        dict(k_dst0=good.transpose(0, 1), v_dst0=good, k_row_bytes=row), dict(k_dst0=good.transpose(1, 2), v_dst0=good, k_row_bytes=row),
        dict(k_dst0=good[:, :, :32], v_dst0=good, k_row_bytes=row),
        dict(k_dst0=K[:, :1], v_dst0=good, k_row_bytes=2 * row),                     # rows of fewer heads
        dict(k_dst0=torch.zeros((1, Hk, D), dtype=F16).expand(10, Hk, D), v_dst0=good, k_row_bytes=row),     # one row for all
        dict(k_dst0=torch.zeros((1, Hk, D), dtype=F16).expand(10, Hk, D), v_dst0=good, k_row_bytes=0),
        dict(k_dst0=good, v_dst0=good, n_rows0=11), dict(k_dst0=flat, v_dst0=good, k_row_bytes=2 * row, n_rows0=6),    # more rows than memory
        dict(k_dst0=K, v_dst0=V, k_row_bytes=2 * row, v_row_bytes=2 * row, n_rows0=11),
        dict(k_dst0=good, v_dst0=good, k_dst1=good, n_rows1=11),
        dict(k_dst0=good, v_dst0=good, k_row_bytes=128), dict(k_dst0=good, v_dst0=good, k_row_bytes=-row),   # rows that hold no Hk heads
        dict(k_dst0=good.float(), v_dst0=good), dict(k_dst0=good, v_dst0=good.bfloat16()),                   # values of another type
        dict(k_dst0=good, v_dst0=good, k_type=skv.Q8_0), dict(k_dst0=good, v_dst0=good, k_type=7),
    ]
    for kw in bad:
        refused(_append, lib, **kw)
    assert not lib.calls


def test_cache_regions_on_another_device_are_refused(lib):
    """A region is the handle's device's or (page-locked) host memory."""
    class Far:
        """A tensor of another device, as far as the check looks."""

        def __init__(self, x):
            self.x = x

        def get_device(self):
            return 5

        def __getattr__(self, name):
            return getattr(self.x, name)

    good = torch.zeros((10, 2, 64), dtype=F16)
    for kw in (dict(k_dst0=Far(good), v_dst0=good), dict(k_dst0=good, v_dst0=good, v_dst1=Far(good))):
        assert "device" in refused(_append, lib, **kw)


def test_positions_by_shape(lib):
    """[n_axes, tokens], tokens as the rows have them or in one line, without the axis where there is one."""
    x = torch.zeros((6, 4, 2, 64), dtype=F16)
    y, f = torch.zeros_like(x), torch.zeros(32)
    one, three = skv.Rope(64, f), skv.Rope(64, f, axis=torch.arange(32, dtype=I32) % 3)
    K = torch.zeros((50, 2, 64), dtype=F16)

    def calls(spec, pos, at=torch.zeros((6, 4), dtype=I32)):
        return [lambda: skv.rope(Handle(), spec, x, x, pos, q_out=y, k_out=y, stream=0),
                lambda: skv.rope_append(Handle(), spec, x, x, x, pos, at, K, K, q_out=y, stream=0),
                lambda: skv.rope_backward(Handle(), spec, x, x, pos, dq=y, dk=y, stream=0)]

    zeros = lambda *s: torch.zeros(s, dtype=I32)
    for spec, shapes in ((one, [(6, 4), (24,), (1, 6, 4), (1, 24)]), (three, [(3, 6, 4), (3, 24)])):
        for s in shapes:
            for call in calls(spec, zeros(*s)):
                call()
    n = len(lib.calls)
    for spec, shapes in ((one, [(4, 6), (24, 1), (6, 4, 1), (2, 12), (1, 4, 6), (6, 1, 4)]),
                         (three, [(6, 4, 3), (24, 3), (72,), (3, 4, 6), (6, 3, 4), (1, 72), (3, 1, 24)])):
        for s in shapes:
            for call in calls(spec, zeros(*s)):
                assert "positions" in refused(call)
    # cache rows: as positions of one axis, whatever the rotation has
    for spec, pos in ((one, zeros(6, 4)), (three, zeros(3, 24))):
        for s in ((4, 6), (24, 1), (12, 2), (3, 24), (3, 6, 4)):
            assert "positions" in refused(calls(spec, pos, zeros(*s))[1])
        for s in ((6, 4), (24,), (1, 6, 4), (1, 24)):
            calls(spec, pos, zeros(*s))[1]()
    assert len(lib.calls) == n + 8


def test_rows_of_no_heads(lib):
    """No heads of k: refused, not divided by."""
    K = torch.zeros((10, 2, 64), dtype=F16)
    for kw in (dict(), dict(k_row_bytes=0, v_row_bytes=0)):
        refused(_append, lib, Hk=0, k_dst0=K, v_dst0=K, **kw)

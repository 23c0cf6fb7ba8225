"""The stated limits of the calls around attention: what lies just beyond each is refused on the host, before anything is
launched, on a zeroed handle."""
import ctypes
import os
import re

import pytest

A = 1 << 20                                            # an address that is never followed, 16-byte aligned
F32, F16 = 3, 0


@pytest.fixture(scope="module")
def lib():
    from split_kv_flash_attn_gb300 import build as b
    b.build()
    from split_kv_flash_attn_gb300 import _lib
    return _lib.load()


@pytest.fixture()
def hnd():
    return ctypes.create_string_buffer(1 << 16)


def _attn(lib, h, lists=0, n=100, **kw):
    from split_kv_flash_attn_gb300 import _lib
    d = dict(S=1, nq=16, H=1, Hk=1, D=128, scale=0.1, k_type=0, v_type=0, k_row_bytes=None, v_row_bytes=None)
    d.update(kw)
    for x in ("k_row_bytes", "v_row_bytes"):
        d[x] = d[x] or d["Hk"] * d["D"] * 2
    rc = lib.skv_attn_backward(h, _lib.SkvShape(*d.values()), A, A, A, None, 0, A if lists else None, n, 0, 0, n, A, A, F16, A, None, F16, A, A, A, None)
    return rc, lib.skv_last_error(h).decode()


ROWS = 1 << 22


@pytest.mark.parametrize("kw,word", [
    # query tiles of a KV head: rows of one head, of eight that share it, of several sequences over the same keys, of five
    # heads (128 tokens of one a tile, the fewest tiles), of more heads than a tile has rows
    (dict(nq=ROWS + 1), "tiles of query rows"),
    (dict(nq=ROWS // 8 + 1, H=8), "tiles of query rows"),
    (dict(S=4, nq=ROWS // 4 + 1), "tiles of query rows"),
    (dict(nq=32768 // 5 * 128 + 1, H=5), "tiles of query rows"),
    (dict(nq=ROWS // 256 + 1, H=256), "tiles of query rows"),
    (dict(lists=1, nq=ROWS + 1, n=10), "tiles of query rows"),
    # all tiles
    (dict(nq=128, H=65536, Hk=65536, n=32768 * 128), "too many tiles"),
    (dict(lists=1, S=1 << 12, nq=1, H=1024, Hk=1024, n=512 * 128), "too many tiles"),
    # ... whose number passes 64 bits, and whose heads alone do 31
    (dict(lists=1, S=1 << 30, nq=1, H=1 << 30, Hk=1 << 30, D=64, n=1024), "too many tiles"),
    (dict(lists=1, S=1 << 29, nq=1, H=1 << 30, Hk=1 << 30, D=64, n=31 * 128), "too many tiles"),
    (dict(lists=1, S=1 << 16, nq=1, H=1 << 16, Hk=1 << 16, n=1), "too many tiles"),
    # bytes
    (dict(k_row_bytes=1 << 39), "2^39"), (dict(v_row_bytes=1 << 39), "2^39"),
    (dict(lists=1, S=2, nq=1 << 20, H=4096, Hk=4096, n=10), "2^39"),
    # tokens, keys
    (dict(S=2, nq=(1 << 30) - 127), "2^31 - 256"), (dict(n=(1 << 31) - 255), "2^31 - 256"),
])
def test_beyond_the_limits_of_gradients(lib, hnd, kw, word):
    rc, msg = _attn(lib, hnd, **kw)
    assert rc == 2 and word in msg, (rc, msg)


def test_the_header_states_them():
    """The numbers that the code refuses by stand in the header."""
    import split_kv_flash_attn_gb300 as skv
    root = os.path.dirname(os.path.dirname(skv.__file__))
    header = open(os.path.join(root, "include", "splitkv.h")).read()
    text = re.sub(r"[\s*]+", " ", header[header.index("---- gradients of attention"):])
    tiles = int(re.search(r"kMaxQTiles = (\d+);", open(os.path.join(root, "split_kv_flash_attn_gb300", "csrc", "bwd.cuh")).read()).group(1))
    assert f"at most {tiles} tiles of query rows" in text and tiles * 128 == ROWS and "2^22 of them" in text
    assert "over all KV heads and lists together below 2^31" in text and "below 2^39 bytes" in text and "below 2^31 - 256" in text
    assert "smaller than about 2^-29" in text and "are more than about" not in text
    rows = re.sub(r"[\s*]+", " ", header[header.index("norm and rotation -----"):header.index("---- gradients of attention")])
    assert "n is below 2^31, H and Hk at most 65535" in rows

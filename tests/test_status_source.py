"""Which bits of the device status word end a wait, read from the source."""
import os
import re

import split_kv_flash_attn_gb300 as skv

CSRC = os.path.join(os.path.dirname(skv.__file__), "csrc")


def test_only_a_wait_that_gave_up_ends_others():
    """Bit 0 says so; the others (rows beyond a cache, bad pages) are no reason to drop a pipeline's work."""
    for name in sorted(os.listdir(CSRC)):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"if \(([^;]*?(?:\*abort_flag|volatile int \*>\(status\))[^;]*?)\) return false;", src):
            assert re.search(r"(?:\*abort_flag|\(status\)) & 1\)*$", m.group(1)), (name, m.group(0))
    assert "(*abort_flag & 1)" in open(os.path.join(CSRC, "tc.cuh")).read()


def test_prefill_waits_for_its_loads_and_products_whoever_gives_up():
    """A warp may give up after the one that issued has looked: what is in flight is waited for in any case, with a limit
    and no status word."""
    for name, n in (("prefill_kernel.cuh", 2), ("prefill_pairq.cuh", 1)):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        drains = list(re.finditer(r"mbar_wait\(bar\([^;]*nullptr, 100000000ull\)", src))
        assert len(drains) == n
        for d in drains:
            before = src[:d.start()].rstrip().splitlines()
            assert not any("s_abort" in line for line in before[-3:]), (name, before[-3:])

"""What the gradient kernels have to keep to when a bounded wait gives up, read from their source: such a failure is not
staged on a GPU.  A CTA that leaves with copies or products in flight lets them read and write shared and tensor memory
that are another CTA's by then."""
import os
import re

import pytest

import split_kv_flash_attn_gb300 as skv

CSRC = os.path.join(os.path.dirname(skv.__file__), "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def block(src, at):
    """The text from the brace at or after `at` to the one that closes it."""
    at = src.index("{", at)
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i + 1]
    raise AssertionError("unbalanced")


def roles(src):
    """The warps' parts of a stretch."""
    return re.split(r"\} else if \(warp == |\} else \{\s*const uint32_t lane_base|if \(warp == kCompute / 32\) \{", src)[1:]


DRAIN = r"tc::mbar_wait\(bar\((\w+)[^;]*nullptr, kDrainNs\)"


@pytest.mark.parametrize("name,vote", [("bwd_kv.cuh", "if (__syncthreads_or(s_abort)) {"), ("bwd_q.cuh", "if (gave_up) {")])
def test_loads_and_products_are_waited_for_whoever_gives_up(name, vote):
    src = source(name)
    # The CTA decides as a whole, behind the end of all warps' parts: somebody may give up after others have looked.
    assert src.count("__syncthreads_or(s_abort)") == 1 and src.count(vote) == 1
    assert vote.startswith("if (__sync") or "const bool gave_up = __syncthreads_or(s_abort);" in src
    assert not re.search(r"if \(s_abort\)", src) and len(re.findall(r"s_abort\)", src)) == len(re.findall(r"&s_abort\)|_or\(s_abort\)", src))
    leaving = block(src, src.index(vote))
    assert leaving.rstrip("} \n").endswith("break;")
    # with a limit, and no status word that would cut a wait short; nowhere else, so that no wait hangs on who knows what
    drains = re.findall(DRAIN, leaving)
    assert len(drains) == leaving.count("mbar_wait(")
    assert src.count("mbar_wait(") == len(drains) + 1        # and the one of CTAs without work
    # every barrier that loads complete on, as many loads as were asked for
    loaded = set(re.findall(r"(?:tma_load_\dd|bulk_load)\([^;]*bar\((\w+)(?: \+ \w+)?\)\);", src))
    assert len(loaded) == 3 and loaded <= set(drains), (loaded, drains)
    tma = roles(src)[0]
    assert re.search(r"\}\s*s_loads\[0\] = it0 \+ [qk]_out;\s*s_loads\[1\] = it0 \+ [ov]_out;\s*\}", tma)
    assert leaving.count("s_loads[0]") == leaving.count("s_loads[1]") == 2
    # products: a commit behind all of a thread's, by that thread, waited for
    issuing = [r for r in roles(src) if "mma_f16_" in r]
    if name == "bwd_kv.cuh":                                 # each stretch ends with it
        assert len(issuing) == 1 and re.search(r"\}\s*tc::mma_commit_if\(one, bar\(second \? B_ACC \+ 1 : B_ACC\)\);\s*\}", issuing[0])
        assert "B_ACC" in drains
    else:
        assert len(issuing) == 2 and all("tc::elect_one()" in r for r in issuing)
        assert "mma_commit_if(tc::elect_one(), bar(B_END +" in leaving and "B_END" in drains


@pytest.mark.parametrize("name", ["bwd_kv.cuh", "bwd_q.cuh"])
def test_ctas_without_work_wait_for_their_first_loads(name):
    src = source(name)
    early = [m.group(1) for m in re.finditer(r"if \((?:o_lo >= o_hi|j_lo >= j_hi) && tid == kCompute\) ([^;]*;)", src)]
    assert len(early) == 1 and re.match(DRAIN, early[0])

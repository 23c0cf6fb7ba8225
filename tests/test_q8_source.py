"""What the kernels over 8-bit pages have to keep to when a bounded wait gives up, read from
their source: such a failure is not staged on a GPU."""
import os
import re

import pytest

import split_kv_flash_attn_gb300 as skv

CSRC = os.path.join(os.path.dirname(skv.__file__), "csrc")


@pytest.mark.parametrize("name", ["q8_decode.cu", "q8_prefill.cu"])
def test_a_warp_votes_on_its_waits(name):
    """A lane whose wait gave up must not leave the others alone with products, shuffles and barriers of
    the whole warp: what comes of a wait is used in a vote, or by code that goes on all the same."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    bodies = re.split(r"auto wait = \[&\]", src)
    assert len(bodies) == 2
    uses = list(re.finditer(r"[^\n;{}]*[^\w:.]wait\([^\n;]*", bodies[1]))
    assert len(uses) >= 2
    for m in uses:
        line = m.group(0)
        # `have` of the prefill kernel's results is voted on in the statement behind it
        voted = "__all_sync" in line or re.search(r"\ball\(wait\(", line)
        later = re.match(r"\s*bool (\w+) = ", line)
        if later and not voted:
            rest = bodies[1][m.end():].lstrip("; \n")
            voted = rest.startswith(f"{later.group(1)} = __all_sync(0xffffffffu, {later.group(1)})")
        assert voted, line.strip()

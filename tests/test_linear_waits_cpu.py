"""The waits of the products' kernel as its source has them: what they guard against cannot be provoked without a wait that
runs out or a race, so the text itself is held to its two rules."""
import os
import re

import newton_schulz_stacked_gb300 as nss

CSRC = os.path.join(os.path.dirname(nss.__file__), "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_bounded_waits_are_decided_by_whole_warps():
    """Lanes time a wait by clocks of their own: what one of them decides, all have to."""
    found = 0
    for name in ("mb_linear.cu", "mb_linear.cuh"):
        text = _source(name)
        for call in re.finditer(r"mbar_wait(?:_cluster)?_or_abort\(", text):
            found += 1
            before = text[:call.start()].rstrip()
            assert re.search(r"__all_sync\(0xffffffffu,$", before), text[call.start() - 120:call.end() + 80]
    assert found >= 8


def test_slabs_of_dz_are_handed_over_through_a_barrier():
    """A lane acquires its slab's counter, another lane issues the load: a warp barrier, then the fence between generic and
    asynchronous accesses, stand between them."""
    text = _source("mb_linear.cuh")
    body = text[text.index("bool rows(const LinearAhead& A"):]
    body = body[body.index("load_acquire"):body.index("return true;", body.index("load_acquire"))]
    assert re.search(r"__syncwarp\(\);\s*fence_async_global\(\);\s*$", body), body


def test_every_block_has_all_producers_in_it():
    """A stage is released by what was loaded into it.  A block that some producer had no part in could be released, and the
    stage with it, twice before that producer looks: it would wait for a phase that has passed."""
    text = _source("mb_linear.cu")
    loop = text[text.index("for (int left = blocks; left > 0;"):]
    loop = loop[:loop.index("__syncwarp();")]
    loads = loop[loop.index("if (elect_lane())"):]
    depth, guards = 0, []
    for line in loads.splitlines():
        if "tma_load_3d_pair(to, f.map" in line:
            break
        guards = guards[:depth]
        if line.rstrip().endswith("{"):
            guards.append(line.strip())
        depth += line.count("{") - line.count("}")
    assert guards[:depth] == ["if (elect_lane()) {"], guards[:depth]
    assert re.search(r"if \(past_end\) mbar_arrive\(&full\[st\]\);\s*else mbar_expect_tx\(&full\[st\]", loop)

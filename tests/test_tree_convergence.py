"""The tree attention's softmax warps come to their scores converged (CPU): their lanes walk up the tree by themselves, as
far as each has to, and the loads from tensor memory behind it are the whole warp's.  Nothing but a warp-wide
synchronisation brings lanes together for certain."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_forward_06_gb300",
                      "csrc", "prefill_tc.cu")


def test_lanes_meet_between_their_masks_and_the_first_scores():
    with open(SOURCE) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    body = code[code.index("void softmax_wg("):]
    masks = body.index("tree_visible(")
    between = body[masks:body.index("tmem_ld32(tS", masks)]
    waits = [m.start() for m in re.finditer(r"wait_bounded\(", between)]
    assert waits and "__syncwarp()" in between[:waits[0]]
    # and the walk itself is the last thing that they do apart
    assert "tree_visible(" not in between[between.index("__syncwarp()"):]

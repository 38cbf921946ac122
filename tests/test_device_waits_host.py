"""Rules of the device code's waits that neither a compiler nor a run of it can show broken, read from the sources:
an order of memory accesses that happens to hold on one machine, and the ways out of a wait that runs out."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_moe_expert_router_gb300",
                    "csrc")


def _source(name):
    """The file without comments, white space as one blank."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", " ", text))


def _block(text, at):
    """The text from `at` to the brace that closes the first one behind it."""
    depth = 0
    for i in range(text.index("{", at), len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("unbalanced braces")


def test_a_wait_by_one_lane_orders_the_warps_accesses():
    """Where one lane waits on a barrier for its warp, a warp barrier follows before the others go on: a shuffle
    passes the result on but orders no memory."""
    body = _block(_source("tcgen05.cuh"), _source("tcgen05.cuh").index("bool stage_wait_warp("))
    assert re.search(r"stage_wait\w*(<\w+>)?\(bar, parity, err\);.*__syncwarp\(\);.*return", body)

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


def test_waits_for_another_ctas_signals_have_cluster_scope():
    """What another CTA of a cluster did before it signalled a barrier is ordered by a wait of cluster scope only (the
    default is the own CTA's), and by an arrival of that scope: all barriers but the one that a CTA's own copies of
    a tail complete."""
    waits = re.findall(r"\bstage_wait\w*(<true>)?\((\w+)", _source("linear.cu"))
    assert {bar for _, bar in waits} == {"full", "empty", "tail_full", "tail_done", "acc_full", "acc_empty", "vacant",
                                         "summed"}
    assert all(scope or bar == "tail_full" for scope, bar in waits)
    assert len(re.findall(r"mbar_wait<true>\(got,", _source("linear_small.cu"))) == 2
    arrivals = re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster", _source("tcgen05.cuh"))
    assert arrivals and all(".cluster.shared::cluster" in a for a in arrivals)
    release = _block(_source("tcgen05.cuh"), _source("tcgen05.cuh").index("void mbar_arrive_cluster_shared("))
    assert release.index("fence.release") < release.index("mbar_arrive_cluster_relaxed(")
    assert re.search(r"fence_proxy_async\(\); __syncwarp\(\); if \(lane == 0\) mbar_arrive_cluster_shared\(lead_done",
                     _source("linear.cu"))


def test_every_role_waits_for_the_launch_before_first():
    """A bounded wait of the products' kernel for a stage, an accumulator or a sum starts behind the wait for the
    launch before, whose rest would count against the limit.  (The loading thread's first waits are for stages that
    are still empty and return at once.)"""
    text = _source("linear.cu")
    kernel = _block(text, text.index("linear_kernel(const __grid_constant__ Args a,"))
    roles = kernel[kernel.index("if (warp < 4)"):]
    starts = [roles.index(m) for m in ("else if (warp == 1)", "else if (warp == 2)", "else if (kMode == kWeightGrad && warp == 3)",
                                       "else if (!kSplit)")]
    starts.append(roles.index("else {", starts[-1]))
    for at in starts:
        role = _block(roles, at)
        wait = re.search(r"(stage_wait\w*|mbar_wait)(<\w+>)?\(", role)
        assert 0 < role.find("grid_dependency_wait()") < (wait.start() if wait else len(role)), role[:60]


def test_copies_in_flight_land_after_a_wait_ran_out():
    """The kernel for few rows counts a chunk before it waits for it, so the copies that may still be in flight when
    that wait runs out begin with the last chunk counted, not behind it."""
    body = _source("linear_small.cu")
    chunk = _block(body, body.index("const auto chunk = "))
    assert chunk.index("stage_wait_warp(") < chunk.index("++used;") < chunk.index("__syncthreads_and(")
    drain = re.search(r"for \(int k = (used[^;]*); k < fetched; \+\+k\) mbar_wait\(full", chunk)
    assert drain and drain.group(1) == "used - 1"

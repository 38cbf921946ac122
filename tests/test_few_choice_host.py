"""The order of the shared memory accesses in a single token's choice, read from the source: a run of it that goes wrong
depends on how late a warp comes."""
import re

from test_device_waits_host import _block, _source


def test_all_warps_read_the_choice_by_rank_before_it_is_made_anew():
    """Where logits tie, every warp has to find a rank open before the one that makes the choice by rounds writes into
    the same place: a barrier of the CTA stands between the vote on it and the return."""
    text = _source("few.cu")
    by_rank = _block(text, text.index("bool choose_by_rank("))
    vote = re.search(r"(\w+) = __any_sync\(0xffffffffu, [^;]*r\.sel\[lane\] < 0\); if \(\1\) __syncthreads\(\); "
                     r"return !\1;", by_rank)
    assert vote and by_rank.rindex("r.sel[at] = i") < by_rank.rindex("__syncthreads();", 0, vote.start()) < vote.start()
    # and what the choice by rounds leaves is read behind a barrier
    form = _block(text, text.index("void form_routing("))
    assert re.search(r"!choose_by_rank\([^{]*\{ if \(warp == 0[^;]*;( if \(warp == 0[^;]*;)? __syncthreads\(\); \}", form)

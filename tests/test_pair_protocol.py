"""The 8-bit LM head's pairs of blocks: what the leader's commits still have on the
way to the other block's barriers when that block is done, checked on the CPU.

Each commit arrives once at a barrier of either block, some time later.  A block
that leaves with an arrival on the way gives its shared memory to the next block
before the arrival lands there.  The model counts, for the other block, the
arrivals on each of its barriers and the latest it waits for.
"""
import os

import pytest

from test_quarter_protocol import CSRC, body_of


def unseen(units, k_blocks, ring, drain):
    """The barriers of the leader's commits that the other block does not wait for, in order."""
    arrivals, waited = {}, {}

    def commit(bar):
        arrivals[bar] = arrivals.get(bar, 0) + 1

    def wait(bar, phase):  # phases count from 1
        waited[bar] = max(waited.get(bar, 0), phase)

    it = 0
    for u in range(units):
        for _ in range(k_blocks):
            s = it % ring
            commit(("empty", s))               # the leader, when the stage's MMAs are done
            wait(("empty", s), it // ring)     # the copy thread, before it fills the stage (phase 0: at once)
            it += 1
        commit(("acc_full", u & 1))
        wait(("acc_full", u & 1), u // 2 + 1)  # the epilogue
    commit(("mma_done", 0))
    if drain:
        for i in range(max(it - ring, 0), it):
            wait(("empty", i % ring), i // ring + 1)
        wait(("mma_done", 0), 1)
    return [bar for bar, n in arrivals.items() if waited.get(bar, 0) < n]


@pytest.mark.parametrize("units,k_blocks", [(1, 1), (1, 9), (2, 32), (5, 9), (17, 13)])
@pytest.mark.parametrize("ring", [5, 6])
def test_every_arrival_is_waited_for(units, k_blocks, ring):
    assert unseen(units, k_blocks, ring, drain=True) == []
    left = unseen(units, k_blocks, ring, drain=False)  # what the model is for: without it the last ones are not
    assert ("mma_done", 0) in left and len(left) == min(ring, units * k_blocks) + 1


def test_the_source_drains():
    body = body_of(open(os.path.join(CSRC, "linear.cu")).read(), "linear_partials8_pair_kernel")
    assert "const int64_t last = it > kRing ? it - kRing : 0;" in body
    copies = body[body.index("const int64_t last"):body.index("} else if (warp == 1)")]
    drain = copies[copies.index("for (int64_t i = last; i < it; ++i) {", copies.index("sm.full")):]
    assert "sm.empty[i % kRing], static_cast<unsigned>((i / kRing) & 1)" in drain
    assert "if (rank != 0) thread_wait_watch(&sm.mma_done, 0u" in drain
    assert body.rindex("cluster_sync()") > body.index(drain)

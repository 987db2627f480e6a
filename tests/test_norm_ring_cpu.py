"""CPU: the walk of the norm backward's ring of asynchronous copies
(k_rms_norm_bwd in norm.cu), restated group by group: each row that is read has
landed, no slot is filled before it has been read, and nothing is in flight
when a warp leaves."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "graph_sparse_head_gb300", "csrc", "norm.cu")


def kernel():
    s = open(SRC).read()
    at = s.index("__global__ void __launch_bounds__(kThreads) k_rms_norm_bwd(")
    return s[at:s.index("__global__", at + 10)]


def walk(ring, steps, drains):
    """Copies in flight when a warp with this many steps leaves."""
    slots, flight, read = [None] * ring, [], set()

    def fetch(row, slot):
        assert slots[slot] is None or slots[slot] in read  # what lay there has been read
        assert all(s != slot for _, s in flight)
        slots[slot] = row
        flight.append((row, slot))  # one group each

    for i in range(ring - 1):
        fetch(i, i)
    slot = 0
    for step in range(steps):
        fetch(step + ring - 1, slot - 1 if slot else ring - 1)
        del flight[:max(0, len(flight) - (ring - 1))]  # wait_group ring - 1: the youngest may still fly
        assert slots[slot] == step and (step, slot) not in flight
        read.add(step)
        slot = 0 if slot + 1 == ring else slot + 1
    return 0 if drains else len(flight)


@pytest.mark.parametrize("ring", [2, 4])
@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 5, 9, 40])
def test_nothing_flies_when_a_warp_leaves(ring, steps):
    k = kernel()
    assert len(re.findall(r'"cp.async.wait_group %0;" ::"n"\(kRing - 1\)', k)) == 1
    tail = k[k.index("cp.async.wait_group"):]
    drain = tail.find("cp.async.wait_all")
    drains = 0 <= drain < tail.index("if (!a.part) return;")  # before the first way out
    assert walk(ring, steps, drains) == 0


def test_the_walk_sees_a_missing_wait():
    assert walk(4, 7, False) == 3 and walk(2, 0, False) == 1

"""CPU: the binding's stage timing holds every stage that the library has (a read
clears the records, so that a stage left out would be lost), against a fake of
the library's call."""
import os
import re

import graph_sparse_head_gb300 as pmha
from graph_sparse_head_gb300 import _lib

CSRC = os.path.join(os.path.dirname(__file__), "..", "graph_sparse_head_gb300", "csrc")


class Fake:
    def __init__(self, stages):
        self.stages = stages

    def pmha_profile_read(self, most, names, launches, totals, n):
        n._obj.value = len(self.stages)
        for i, s in enumerate(self.stages[:most]):
            names[32 * i:32 * i + 32] = s.encode().ljust(32, b"\0")
            launches[i], totals[i] = i + 1, 0.5 * i
        return 0


def test_every_stage_is_read(monkeypatch):
    literals = set()
    for f in os.listdir(CSRC):
        literals |= set(re.findall(r'"([a-z][a-z0-9]*(?:_[a-z0-9]+)*)"', open(os.path.join(CSRC, f)).read()))
    stages = sorted(literals)  # a superset of the stages' names
    assert len(stages) > 32 and "ffn_block_backward" in stages
    monkeypatch.setattr(_lib, "load", lambda: Fake(stages))
    assert pmha.pmha_profile_read() == {s: (i + 1, 0.5 * i) for i, s in enumerate(stages)}

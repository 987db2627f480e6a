"""Gates that do not belong to the rows of a call are refused."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_gate_without_rows_is_no_missing_gate():
    x = torch.randn(6, 32, device=DEV)
    p = pmha.JoinParams(pre=torch.ones(32, device=DEV), gate=torch.empty(0, 32, device=DEV))
    for call in (lambda: pmha.pmha_join(p, x, x), lambda: pmha.pmha_join_checkpointed(p, x, x),
                 lambda: pmha.pmha_join_backward(p, x, x, x, x), lambda: pmha.pmha_join_backward_workspace_size(p, x)):
        with pytest.raises(ValueError, match="gate"):
            call()
    none = x[:0]  # no samples: no gates
    for gate in (p.gate, torch.ones(4, 32, device=DEV)[:0]):
        p.gate = gate
        s, n = pmha.pmha_join(p, none, none)
        got = pmha.pmha_join_backward(p, none, s, n, none)
        assert s.shape == (0, 32) and got["dgate"].shape == (0, 32) and bool((got["dpre"] == 0).all())

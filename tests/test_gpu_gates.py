"""Gates that do not belong to the rows of a call are refused."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests.test_gpu_encoder import make

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


@pytest.mark.parametrize("which", ["gate1", "gate2"])
def test_a_layer_refuses_gates_of_another_batch(which):
    """(G, E) with G neither 1 nor the batch, but a divisor of the tokens: some samples would take another's gate."""
    base, x, dy, _ = make(64, 256, 4, 32, 4, 40, "f32")
    args = (base.graph, base.attention, base.norm1, base.norm2, base.block)

    def layer(rows):
        return pmha.PackedEncoderLayer(*args, **{which: torch.rand(rows, 32, device=DEV)})

    mask = torch.zeros(4, 64, dtype=torch.bool, device=DEV)
    for rows in (2, 8, 256):
        wrong = layer(rows)
        for call in (lambda: wrong(x), lambda: wrong(x, key_padding_mask=mask), lambda: wrong.backward(x, dy),
                     lambda: wrong.forward_checkpointed(x)):
            with pytest.raises(ValueError, match=which):
                call()
    right = layer(4)
    _, kept = right.forward_checkpointed(x)
    with pytest.raises(ValueError, match=which):
        layer(2).backward_checkpointed(kept, dy)
    one = layer(1)  # one row for all samples is what (E,) is
    same = pmha.PackedEncoderLayer(*args, **{which: getattr(one, "join" + which[-1]).gate[0]})
    assert torch.equal(one(x), same(x))


def test_a_served_layer_refuses_gates_of_another_batch():
    base, x, _, _ = make(100, 800, 4, 128, 8, 256, "bf16", seed=5)
    layer = pmha.PackedEncoderLayer(base.graph, base.attention, base.norm1, base.norm2, base.block,
                                    gate2=torch.ones(2, 128, dtype=torch.bfloat16, device=DEV))
    for block in (pmha.FfnQuantizedParams.from_params(base.block), pmha.FfnMxParams.from_params(base.block)):
        with pytest.raises(ValueError, match="gate2"):
            layer.serve(x, block)

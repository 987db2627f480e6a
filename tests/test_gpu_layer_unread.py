"""The layer makes, keeps and computes again only what its joins read."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests.test_gpu_encoder import make
from tests.test_gpu_encoder_joins import BARS, close, joined, plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n,nnz,B,E,H,F,dt", [(64, 256, 2, 32, 4, 88, "f32"), (300, 3000, 2, 128, 8, 344, "bf16")])
def test_a_scale_alone_keeps_and_repeats_no_block(n, nnz, B, E, H, F, dt, monkeypatch):
    """With a residual scale and neither norm nor gate after the block, no gradient needs the block's output."""
    base, x, dy, spec = make(n, nnz, B, E, H, F, dt)
    layer = joined(base, 5, False, 0, 1.25)
    y, kept = layer.forward_checkpointed(x)
    assert kept.block is None
    assert torch.equal(y, layer(x))
    want, leaf = plain(layer, x, spec)
    want.backward(dy.double())
    close("y", y, want.detach(), 1.5 * BARS[dt][0])

    def never(*args, **kw):
        raise AssertionError("the block ran forward again")

    monkeypatch.setattr(pmha, "pmha_ffn_forward", never)
    grads = layer.backward(x, dy)
    from_kept = layer.backward_checkpointed(kept, dy)
    for name, v in leaf.items():
        if name == "bk" or v is None:
            continue  # bk: zero in exact arithmetic
        got = grads["dx" if name == "x" else "d" + name]
        close(name, got, v.grad, 1.5 * BARS[dt][1] * (5 if v.dim() == 1 else 1))
    assert from_kept.keys() == grads.keys()


def test_a_step_from_checkpoints_with_norm_or_gate_alone_keeps_the_block():
    base, x, dy, _ = make(64, 256, 2, 32, 4, 88, "f32")
    for post, gates in ((True, 0), (False, 1)):
        _, kept = joined(base, 5, post, gates, 1.0).forward_checkpointed(x)
        assert kept.block is not None


def test_serving_in_8_bits_normalises_a_join_once(monkeypatch):
    """The 8-bit norm takes the join's sum: the join itself leaves its norm out."""
    base, x, _, _ = make(100, 800, 2, 128, 8, 256, "bf16", seed=5)
    layer = joined(base, 9, True, 1)
    block = pmha.FfnQuantizedParams.from_params(base.block)
    n1, _ = pmha.pmha_rms_norm(x, layer.norm1, layer.eps)
    a, _ = pmha.pmha_forward(layer.graph, layer.attention, n1, n1, n1)
    s, _ = pmha.pmha_join(layer.join1, a, x)
    q, scale, _ = pmha.pmha_rms_norm_quantized(s, layer.norm2, layer.eps)
    want = pmha.pmha_join(layer.join2, pmha.pmha_ffn_forward_quantized(block, q, scale), s)[0]
    join, seen = pmha.pmha_join, []

    def spy(params, *args, **kw):
        seen.append(params.pre is None)
        return join(params, *args, **kw)

    monkeypatch.setattr(pmha, "pmha_join", spy)
    assert torch.equal(layer.serve(x, block), want)
    assert seen == [True, True]

"""8-bit checkpoints and 4-bit quantisation at odd widths on tensors past 2^32 values: the last rows are those of a call on
them alone, bit for bit."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"


@pytest.mark.parametrize("width", [171, 7])
def test_odd_widths_past_2_32_values(width):
    rows = (2 ** 32 + 2 ** 25) // width
    assert rows * width > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(4)
    base = torch.randn(4099, width, generator=g, device=DEV).bfloat16()
    x = base.repeat((rows + 4098) // 4099, 1)[:rows].contiguous()
    x[-1000:] = torch.randn(1000, width, generator=g, device=DEV).bfloat16() * 3
    tail = x[-1000:].clone()
    k, one = pmha.pmha_checkpoint(x), pmha.pmha_checkpoint(tail)
    assert torch.equal(k.codes[-1000:], one.codes) and torch.equal(k.scale[-1000:], one.scale)
    back = pmha.pmha_checkpoint_restore(k)
    assert torch.equal(back[-1000:], pmha.pmha_checkpoint_restore(one))
    first = pmha.pmha_checkpoint_restore(pmha.pmha_checkpoint(x[:5000].clone()))
    assert torch.equal(back[:5000], first)
    del back, k
    q = pmha.pmha_mx_quantize(x)
    assert torch.equal(q.codes[-1000:], pmha.pmha_mx_quantize(tail).codes)

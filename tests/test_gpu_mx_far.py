"""4-bit products of large scales whose sums are small: no infinity between."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def operands(rows, ex, ew):
    """Blocks whose largest values miss each other: products of 1/4 and 0 between scales 2^ex and 2^ew."""
    x, w = (torch.zeros(n, 64, dtype=torch.float64, device=DEV) for n in (rows, 16))
    x[:, 0], x[:, 2], w[:, 1], w[:8, 2] = 6.0, 0.5, 6.0, 0.5
    return pmha.pmha_mx_quantize((x * 2.0 ** ex).float()), pmha.pmha_mx_quantize((w * 2.0 ** ew).float())


@pytest.mark.parametrize("rows", [1, 3, 8, 40, 300])
@pytest.mark.parametrize("ex,ew", [(100, 28), (100, 27), (64, 64), (4, 124), (124, 4), (-60, -60), (-124, 120)])
def test_sums_next_to_the_largest_values_and_zeros(rows, ex, ew):
    x, w = operands(rows, ex, ew)
    y = pmha.pmha_mx_linear(x, w).double()
    assert bool((y[:, :8] == 2.0 ** (ex + ew - 2)).all()) and bool((y[:, 8:] == 0).all())


@pytest.mark.parametrize("rows", [1, 8, 40])
def test_a_gate_of_large_scales_that_is_zero(rows):
    """silu(0) = 0: the block's output is its bias and residual, the other factor being finite."""
    x, w = operands(rows, 100, 60)
    zero = pmha.MxTensor(w.codes[8:].contiguous().repeat(4, 1), pmha.pmha_mx_quantize(w.values()[8:].float().repeat(4, 1)).scale,
                         (32, 64))
    ones = pmha.pmha_mx_quantize(torch.ones(64, 32, device=DEV) * 2.0 ** -10)
    up = pmha.pmha_mx_quantize(torch.full((32, 64), 2.0 ** -90, device=DEV))
    residual = torch.ones(rows, 64, dtype=torch.bfloat16, device=DEV)
    y = pmha.pmha_ffn_forward_mx(pmha.FfnMxParams(zero, up, ones), x, residual=residual)
    assert torch.equal(y, residual)


@pytest.mark.parametrize("side", ["x", "w"])
def test_nan_scales_stay_nan(side):
    x, w = torch.ones(3, 64, device=DEV), torch.ones(16, 64, device=DEV)
    (x if side == "x" else w)[2, 40] = float("nan")
    y = pmha.pmha_mx_linear(pmha.pmha_mx_quantize(x), pmha.pmha_mx_quantize(w))
    bad = y.isnan()
    assert bool(bad[2].all() and not bad[:2].any()) if side == "x" else bool(bad[:, 2].all() and bad.sum() == 3)

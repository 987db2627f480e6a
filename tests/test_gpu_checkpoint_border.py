"""The scale of 8-bit groups next to its lower limit."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _stream_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("join", [False, True])
def test_scales_next_to_the_least_are_rounded_up_too(dtype, join):
    """The largest values on both sides of 127 times the first scales from 2^-100 on; those below share the least scale."""
    rows = []
    for k in range(-2, 6):
        border = torch.tensor(127 * 2.0 ** -100 * (1 + k / 128), dtype=torch.float64).to(dtype)
        for most in (torch.nextafter(border, border * 0), border, torch.nextafter(border, border * 2)):
            rows.append([float(most)] + [float(most) * i / 32 for i in range(31)])
    x = torch.tensor(rows, dtype=torch.float64, device=DEV).to(dtype)
    codes, scale = ref.kept(x)
    assert bool((x.double().abs().amax(-1) <= 127 * scale[:, 0]).all()) and len(scale.unique()) >= 6
    if join:
        k = pmha.pmha_join_checkpointed(pmha.JoinParams(), x, x, keep_residual=False)[2]
    else:
        k = pmha.pmha_checkpoint(x)
    assert torch.equal(k.scale.double(), scale) and torch.equal(k.codes.double(), codes)

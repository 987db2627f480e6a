"""MxTensor.values() of tensors without rows."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 64), (0, 33), (3, 0, 40), (1, 5)])
def test_values_of_any_number_of_rows(shape):
    x = torch.ones(shape, device="cuda:0", dtype=torch.bfloat16)
    v = pmha.pmha_mx_quantize(x).values()
    assert v.shape == shape and v.dtype == torch.float64 and bool((v == 1).all())

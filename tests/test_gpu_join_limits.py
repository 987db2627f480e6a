"""The join's backward pass near the limits that its checks allow."""
import ctypes

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from graph_sparse_head_gb300 import _lib

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"


def test_a_gate_for_each_of_almost_2_31_rows():
    """dpost sums 2^31 - 16 partial rows, whose last indices plus 32 leave 31 bits. Only the last 64 hold something."""
    lib, rows = _lib.load(), 2 ** 31 - 16
    one = torch.ones(rows, 1, dtype=torch.bfloat16, device=DEV)
    dsum = torch.zeros(rows, 1, dtype=torch.bfloat16, device=DEV)
    dsum[-64:] = 1.0
    post = torch.ones(8, dtype=torch.bfloat16, device=DEV)
    dpost = torch.zeros(8, device=DEV)
    p = _lib.PmhaJoinParams(1, 1, post.data_ptr(), one.data_ptr(), rows, 1.0, None, 1e-6)
    need = lib.pmha_join_backward_workspace_size(ctypes.byref(p), rows)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    st = lib.pmha_join_backward(ctypes.byref(p), rows, one.data_ptr(), None, None, None, dsum.data_ptr(), None, None,
                                dpost.data_ptr(), None, None, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0, lib.pmha_last_error()
    pmha.pmha_device_status()
    want = 64 / (1 + 1e-6) ** 0.5
    # a root within 2^-21 and its product
    assert abs(float(dpost[0].double()) - want) <= 2.0 ** -20 * want
    assert bool((dpost[1:] == 0).all())

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


def test_sums_of_many_like_rows():
    """2^24 partial rows of the same values: what the pairs' low parts lose must not grow with the rows."""
    rows, width = 2 ** 24 + 5, 8
    x = torch.tensor([1.0, 2.5, -0.75, 3.0, 0.25, -1.5, 2.0, 0.5], dtype=torch.bfloat16, device=DEV).repeat(rows, 1)
    ones = torch.ones(width, dtype=torch.bfloat16, device=DEV)
    p = pmha.JoinParams(post=ones, gate=torch.full_like(x, 1.0))
    got = pmha.pmha_join_backward(p, x, None, None, torch.ones_like(x), input_grads=False)
    each = got["dgate"].double()  # with a gate a row and ones for post: the partial rows themselves
    assert bool((each == each[0]).all())
    want = rows * each[0]
    assert bool(((got["dpost"].double() - want).abs() <= 2.0 ** -23 * want.abs()).all())

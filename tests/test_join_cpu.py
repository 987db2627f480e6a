"""Host-side checks of the join and of 8-bit checkpoints: every refusal returns its status and message before any device work."""
import ctypes

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from graph_sparse_head_gb300 import _lib
from graph_sparse_head_gb300 import build as pmha_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 5, 6
P = 1 << 20  # stands for a device address; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    pmha_build.build()
    return _lib.load()


def join(**kw):
    a = dict(dtype=1, width=64, post=20 * P, gate=21 * P, gates=2, residual_scale=1.0, pre=22 * P, eps=1e-6)
    a.update(kw)
    return _lib.PmhaJoinParams(*a.values())


def kept(at):
    return ctypes.byref(_lib.PmhaKept(at, at + P // 2))


BAD_PARAMS = [dict(dtype=2), dict(width=0), dict(width=(1 << 24) + 1), dict(eps=0.0), dict(eps=float("nan")),
              dict(residual_scale=float("inf")), dict(residual_scale=float("nan")), dict(gates=0), dict(gates=3),
              dict(gates=16), dict(gates=-1), dict(gate=None), dict(post=20 * P + 8), dict(gate=21 * P + 2),
              dict(pre=22 * P + 4)]


def forward(lib, p, **kw):
    a = dict(rows=8, branch=P, branch_kept=None, residual=2 * P, residual_kept=None, sum=3 * P, out=4 * P, keep_branch=None,
             keep_residual=None, stream=None)
    a.update(kw)
    return lib.pmha_join(ctypes.byref(p), *a.values())


@pytest.mark.parametrize("kw", BAD_PARAMS)
def test_bad_parameters(lib, kw):
    p = join(**kw)
    assert forward(lib, p) == INVALID and lib.pmha_last_error().startswith(b"pmha_join:")
    assert lib.pmha_join_backward_workspace_size(ctypes.byref(p), 8) == ctypes.c_size_t(-1).value
    assert lib.pmha_last_error().startswith(b"pmha_join_backward:")


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 31), dict(rows=7), dict(branch=None), dict(residual=None), dict(sum=None), dict(out=None),
    dict(branch_kept=kept(5 * P)), dict(residual_kept=kept(5 * P)), dict(branch=P + 8), dict(residual=2 * P + 2),
    dict(sum=P), dict(sum=2 * P + 16), dict(out=3 * P), dict(out=20 * P), dict(out=21 * P), dict(sum=22 * P),
    dict(keep_branch=kept(P)), dict(keep_branch=kept(5 * P), keep_residual=kept(5 * P)),
    dict(keep_branch=kept(4 * P)), dict(branch=None, branch_kept=kept(5 * P), keep_branch=kept(6 * P)),
    dict(residual=None, residual_kept=kept(5 * P), keep_residual=kept(6 * P)),
    dict(branch=None, branch_kept=kept(3 * P)), dict(keep_branch=kept(5 * P + 4)), dict(keep_branch=kept(0)),
])
def test_forward_refusals(lib, kw):
    assert forward(lib, join(), **kw) == INVALID
    assert lib.pmha_last_error().startswith(b"pmha_join:")


def test_forward_without_norms(lib):
    plain = dict(post=None, gate=None, gates=0)
    assert forward(lib, join(pre=None, **plain)) == INVALID  # out without pre
    assert forward(lib, join(pre=None), branch=None, out=None) == INVALID  # post without a branch
    assert forward(lib, join(), rows=0, branch=None, residual=None, sum=None, out=None) == 0
    assert lib.pmha_join(None, 8, P, None, 2 * P, None, 3 * P, 4 * P, None, None, None) == INVALID


def backward(lib, p, **kw):
    a = dict(rows=8, branch=P, branch_kept=None, sum=2 * P, dout=3 * P, dsum=4 * P, dbranch=5 * P, dresidual=6 * P,
             dpost=7 * P, dgate=8 * P, dpre=9 * P, workspace=16 * P, nbytes=1 << 30, stream=None)
    a.update(kw)
    return lib.pmha_join_backward(ctypes.byref(p), *a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=9), INVALID), (dict(branch=None), INVALID), (dict(branch_kept=kept(10 * P)), INVALID),
    (dict(sum=None), INVALID), (dict(dout=None), INVALID), (dict(dbranch=P), INVALID), (dict(dresidual=5 * P), INVALID),
    (dict(dresidual=4 * P + 16), INVALID), (dict(dpost=8 * P), INVALID), (dict(dpre=9 * P + 4), INVALID),
    (dict(dgate=21 * P), INVALID), (dict(dpost=20 * P), INVALID), (dict(dsum=4 * P + 8), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(nbytes=16), WORKSPACE), (dict(workspace=16 * P + 16), WORKSPACE),
])
def test_backward_refusals(lib, kw, status):
    assert backward(lib, join(), **kw) == status
    assert lib.pmha_last_error().startswith(b"pmha_join_backward:")


def test_backward_gradients_need_their_parameter(lib):
    assert backward(lib, join(post=None), branch=P) == INVALID
    assert backward(lib, join(gate=None, gates=0)) == INVALID
    assert backward(lib, join(pre=None), dout=None) == INVALID
    assert backward(lib, join(pre=None), dout=None, dpre=None, dsum=None) == INVALID
    nothing = dict(dbranch=None, dresidual=None, dpost=None, dgate=None, dpre=None, workspace=None, nbytes=0)
    assert backward(lib, join(), **nothing) == 0


def test_too_many_gates(lib):
    p = join(width=1 << 12, gates=1 << 24)
    assert lib.pmha_join_backward_workspace_size(ctypes.byref(p), 1 << 24) == ctypes.c_size_t(-1).value
    assert backward(lib, p, rows=1 << 24) == UNSUPPORTED


def test_backward_sizes(lib):
    n = lib.pmha_join_backward_workspace_size(ctypes.byref(join()), 100_000)
    assert n >= 2 * 64 * 4 and n % 512 == 0
    assert lib.pmha_join_backward_workspace_size(ctypes.byref(join()), 0) == 0


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(rows=-1), dict(width=0), dict(x=None), dict(x=P + 8), dict(k=None),
                                dict(k=kept(P)), dict(k=kept(0)), dict(k=kept(2 * P + 8))])
def test_checkpoint_refusals(lib, kw):
    a = dict(dtype=1, rows=8, width=64, x=P, k=kept(2 * P))
    a.update(kw)
    assert lib.pmha_checkpoint(*a.values(), None) == INVALID
    assert lib.pmha_last_error().startswith(b"pmha_checkpoint:")
    assert lib.pmha_checkpoint_restore(a["dtype"], a["rows"], a["width"], a["k"], a["x"], None) == INVALID
    assert lib.pmha_checkpoint_restore(1, 0, 64, None, None, None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: pmha.pmha_checkpoint(x), lambda: pmha.pmha_join(pmha.JoinParams(), x, x),
                 lambda: pmha.pmha_join_backward(pmha.JoinParams(), x, None, None, x),
                 lambda: pmha.Checkpoint(x, x, torch.float32)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="dout or dsum"):
        pmha.pmha_join_backward(pmha.JoinParams(), x, None, None)
    with pytest.raises(TypeError, match="kept"):
        pmha.pmha_join_checkpointed(pmha.JoinParams(), None, x)

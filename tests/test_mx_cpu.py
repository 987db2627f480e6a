"""Host-side checks of the operators in microscaled 4 bits: every refusal returns its status and message before any device work."""
import ctypes

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from graph_sparse_head_gb300 import _lib
from graph_sparse_head_gb300 import build as pmha_build

INVALID, WORKSPACE = 1, 6
P = 1 << 24  # stands for a device address; never dereferenced on the host
NO_SIZE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    pmha_build.build()
    return _lib.load()


def mx(at, scale=None):
    return _lib.PmhaMx(at, at + P // 2 if scale is None else scale)


def test_sizes(lib):
    assert lib.pmha_mx_code_bytes(3, 33) == 3 * 32 and lib.pmha_mx_scale_bytes(3, 33) == 512
    assert lib.pmha_mx_code_bytes(129, 256) == 129 * 128 and lib.pmha_mx_scale_bytes(129, 257) == 2 * 3 * 512
    assert lib.pmha_mx_code_bytes(0, 5) == 0 and lib.pmha_mx_scale_bytes(0, 5) == 0
    for bad in ((-1, 4), (1 << 31, 4), (4, 0), (4, (1 << 20) + 1), ((1 << 31) - 1, 1 << 20)):
        assert lib.pmha_mx_code_bytes(*bad) == NO_SIZE and lib.pmha_mx_scale_bytes(*bad) == NO_SIZE


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(rows=-1), dict(width=0), dict(width=(1 << 20) + 1), dict(x=None),
                                dict(x=P + 2), dict(out=None), dict(out=mx(2 * P + 8)), dict(out=mx(None, 3 * P)),
                                dict(out=mx(2 * P, 0)), dict(out=mx(P)), dict(out=mx(2 * P, P + 512)),
                                dict(out=mx(2 * P, 2 * P + 128))])
def test_quantize_refusals(lib, kw):
    a = dict(dtype=1, rows=8, width=64, x=P, out=mx(2 * P))
    a.update(kw)
    out = None if a["out"] is None else ctypes.byref(a["out"])
    assert lib.pmha_mx_quantize(a["dtype"], a["rows"], a["width"], a["x"], out, None) == INVALID
    assert lib.pmha_last_error().startswith(b"pmha_mx_quantize")
    assert lib.pmha_mx_quantize(1, 0, 64, None, None, None) == 0


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=0), dict(outputs=0), dict(outputs=(1 << 20) + 1), dict(width=1 << 20, outputs=1 << 20),
    dict(x=None), dict(w=None), dict(x=mx(P + 8)), dict(w=mx(2 * P, 3)), dict(out=None), dict(out=4 * P + 2),
    dict(bias=5 * P + 1), dict(residual=6 * P + 8), dict(out=P), dict(out=2 * P + P // 2), dict(out=5 * P),
    dict(residual=4 * P), dict(out=2 * P)])
def test_linear_refusals(lib, kw):
    a = dict(rows=8, width=64, outputs=32, x=mx(P), w=mx(2 * P), bias=5 * P, residual=6 * P, out=4 * P)
    a.update(kw)
    x, w = (None if t is None else ctypes.byref(t) for t in (a["x"], a["w"]))
    st = lib.pmha_mx_linear(a["rows"], a["width"], a["outputs"], x, w, a["bias"], a["residual"], a["out"], None)
    assert st == INVALID and lib.pmha_last_error().startswith(b"pmha_mx_linear")
    assert lib.pmha_mx_linear(0, 64, 32, None, None, None, None, None, None) == 0


def ffn(E=64, F=96, dtype=1, act=0, **kw):
    a = dict(wg=None, wu=None, wd=None, bg=10 * P, bu=11 * P, bd=12 * P)
    a.update(kw)
    return _lib.PmhaFfnParams(E, F, dtype, act, *a.values())


def test_block_refusals(lib):
    weights = _lib.PmhaFfnMx(mx(P), mx(2 * P), mx(3 * P))

    def call(p, w=weights, x=mx(4 * P), residual=5 * P, rows=20, out=6 * P, ws=7 * P, nbytes=P):
        return lib.pmha_ffn_forward_mx(None if p is None else ctypes.byref(p), None if w is None else ctypes.byref(w),
                                       None if x is None else ctypes.byref(x), residual, rows, out, ws, nbytes, None)

    for p in (None, ffn(dtype=0), ffn(act=2), ffn(E=0), ffn(F=0), ffn(E=1 << 20, F=1 << 20)):
        assert call(p) == INVALID and lib.pmha_last_error().startswith(b"pmha_ffn_forward_mx")
        if p is not None:
            assert lib.pmha_ffn_forward_mx_workspace_size(ctypes.byref(p), 20) == NO_SIZE
    good = ffn()
    bad = [dict(w=None), dict(x=None), dict(w=_lib.PmhaFfnMx(mx(P + 1), mx(2 * P), mx(3 * P))), dict(out=None),
           dict(out=6 * P + 2), dict(residual=5 * P + 2), dict(out=4 * P), dict(out=3 * P), dict(out=5 * P), dict(out=12 * P),
           dict(out=7 * P + 64), dict(rows=-1)]
    for kw in bad:
        assert call(good, **kw) == INVALID, kw
    assert call(ffn(bg=10 * P + 1)) == INVALID
    for kw in (dict(ws=None), dict(nbytes=64), dict(ws=7 * P + 16)):
        assert call(good, **kw) == WORKSPACE
    assert call(good, rows=0, x=None, out=None) == 0
    sizes = [lib.pmha_ffn_forward_mx_workspace_size(ctypes.byref(good), r) for r in range(300)]
    assert sizes[0] == 0 and sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pmha.pmha_mx_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        pmha.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8), (4, 64))
    with pytest.raises(TypeError, match="MxTensor"):
        pmha.pmha_mx_linear(x, x)
    with pytest.raises(TypeError, match="MxTensor"):
        pmha.pmha_ffn_forward_mx(pmha.FfnMxParams(x, x, x), x)
    with pytest.raises(TypeError, match="Checkpoint"):
        pmha.pmha_checkpoint_restore(x)
    for shape in ((), (4, 0)):
        with pytest.raises(ValueError, match="one value"):
            pmha.MxTensor(x, x, shape)

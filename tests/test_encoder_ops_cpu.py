"""Host-side checks of the encoder operators (norm, gated block, gradient
clipping): every refusal returns its status and message before any device work,
so that these run without a GPU; and the binding's checks on CPU tensors."""
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


def norm_args(**kw):
    a = dict(dtype=1, rows=8, width=64, x=P, residual=None, weight=None, eps=1e-6, sum=None, out=2 * P, out_q=None,
             scale=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(dtype=7), dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=(1 << 24) + 1), dict(eps=0.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-40), dict(out=None), dict(out_q=3 * P),
    dict(out_q=3 * P, scale=4 * P, x=None), dict(scale=3 * P), dict(x=P + 2), dict(residual=P + 8), dict(weight=P + 4),
    dict(sum=5 * P + 2), dict(out=P), dict(out=P + 512), dict(sum=2 * P + 16), dict(residual=2 * P),
    dict(weight=2 * P), dict(out_q=3 * P, scale=3 * P + 256),
])
def test_norm_refusals(lib, kw):
    assert lib.pmha_rms_norm(*norm_args(**kw)) == INVALID
    assert lib.pmha_last_error().startswith(b"pmha_rms_norm")


def test_norm_without_rows_does_nothing(lib):
    assert lib.pmha_rms_norm(*norm_args(rows=0, x=None, out=None)) == 0


def backward_args(**kw):
    a = dict(dtype=0, rows=8, width=64, x=P, weight=None, eps=1e-6, dout=2 * P, dsum=None, dx=3 * P, dweight=4 * P,
             workspace=8 * P, nbytes=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(eps=-1.0), INVALID), (dict(x=None), INVALID), (dict(dout=None), INVALID), (dict(dx=P), INVALID),
    (dict(dx=2 * P + 64), INVALID), (dict(dweight=3 * P), INVALID), (dict(dweight=P + 4), INVALID),
    (dict(weight=4 * P), INVALID), (dict(dsum=3 * P + 16), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(nbytes=16), WORKSPACE), (dict(workspace=8 * P + 16), WORKSPACE), (dict(dtype=2), INVALID),
])
def test_norm_backward_refusals(lib, kw, status):
    assert lib.pmha_rms_norm_backward(*backward_args(**kw)) == status


def test_norm_backward_sizes(lib):
    assert lib.pmha_rms_norm_backward_workspace_size(3, 8, 64) == 0
    n = lib.pmha_rms_norm_backward_workspace_size(1, 100000, 128)
    assert n >= 128 * 4 and n % 256 == 0
    assert lib.pmha_rms_norm_backward(*backward_args(dx=None, dweight=None)) == 0  # nothing asked for


def ffn(E=64, F=72, dtype=1, act=0, **kw):
    a = dict(wg=P, wu=2 * P, wd=3 * P, bg=None, bu=None, bd=None)
    a.update(kw)
    return _lib.PmhaFfnParams(E, F, dtype, act, *a.values())


BAD_PARAMS = [dict(E=0), dict(F=0), dict(E=(1 << 20) + 1), dict(E=1 << 20, F=1 << 20), dict(dtype=5), dict(act=2)]
BAD_POINTERS = [dict(wg=None), dict(wu=P + 8), dict(wd=None), dict(bg=P + 1), dict(bd=P + 1)]


@pytest.mark.parametrize("kw", BAD_PARAMS + BAD_POINTERS)
def test_ffn_parameter_refusals(lib, kw):
    p = ffn(**kw)
    b = ctypes.byref(p)
    assert lib.pmha_ffn_forward(b, 4 * P, None, 4, 5 * P, 6 * P, 1 << 40, None) == INVALID
    assert lib.pmha_ffn_backward(b, 4 * P, 5 * P, 4, 6 * P, None, 7 * P, 1 << 40, None) == INVALID
    if kw in BAD_PARAMS:
        assert lib.pmha_ffn_forward_workspace_size(b, 4) == ctypes.c_size_t(-1).value
        assert lib.pmha_ffn_backward_workspace_size(b, 4) == ctypes.c_size_t(-1).value


def test_ffn_call_refusals(lib):
    p = ffn()
    b = ctypes.byref(p)
    need = lib.pmha_ffn_forward_workspace_size(b, 1000)
    assert need % 256 == 0
    ok = dict(x=4 * P, residual=None, rows=1000, out=8 * P, ws=16 * P, n=need, stream=None)

    def call(**kw):
        return lib.pmha_ffn_forward(b, *{**ok, **kw}.values())

    assert call(x=None) == INVALID and call(out=None) == INVALID and call(x=4 * P + 2) == INVALID
    assert call(residual=P + 8) == INVALID and call(rows=-1) == INVALID and call(rows=(1 << 31) - 1) == INVALID
    assert call(out=4 * P) == INVALID and call(out=P) == INVALID and call(residual=8 * P) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE and call(ws=16 * P + 8) == WORKSPACE
    assert call(rows=0, x=None, out=None, ws=None, n=0) == 0
    assert lib.pmha_ffn_forward(None, *ok.values()) == INVALID


def test_ffn_backward_refusals(lib):
    p = ffn(bg=5 * P)
    b = ctypes.byref(p)
    need = lib.pmha_ffn_backward_workspace_size(b, 1000)
    assert 0 < need < 1 << 40
    # past a limit the workspace stops growing
    many = [lib.pmha_ffn_backward_workspace_size(b, r) for r in (10_000_000, 50_000_000)]
    assert many[1] <= 1.05 * many[0] < 4 << 30
    g = _lib.PmhaFfnGrads(wg=6 * P)
    ok = dict(x=8 * P, dout=9 * P, rows=1000, dx=10 * P, grads=ctypes.byref(g), ws=32 * P, n=need, stream=None)

    def call(**kw):
        return lib.pmha_ffn_backward(b, *{**ok, **kw}.values())

    assert call(x=None) == INVALID and call(dout=9 * P + 4) == INVALID and call(dx=8 * P) == INVALID
    assert call(grads=ctypes.byref(_lib.PmhaFfnGrads(wg=10 * P))) == INVALID  # over dx
    assert call(grads=ctypes.byref(_lib.PmhaFfnGrads(wg=P))) == INVALID  # over a weight
    assert call(grads=ctypes.byref(_lib.PmhaFfnGrads(bu=6 * P + 1))) == INVALID
    assert call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(dx=None, grads=None) == 0  # nothing asked for


def test_ffn_quantized_refusals(lib):
    q = _lib.PmhaFfnQuantized(P, 2 * P, 5 * P, 6 * P)
    ok = [8 * P, 9 * P, None, 4, 10 * P, 12 * P, 1 << 40, None]
    for kw, status in ((dict(E=72), UNSUPPORTED), (dict(F=68), UNSUPPORTED), (dict(dtype=0), INVALID)):
        p = ffn(**kw)
        assert lib.pmha_ffn_forward_quantized(ctypes.byref(p), ctypes.byref(q), *ok) == status
        assert lib.pmha_ffn_forward_quantized_workspace_size(ctypes.byref(p), 4) == ctypes.c_size_t(-1).value
    p = ffn(wg=None, wu=None)
    assert lib.pmha_ffn_forward_quantized(ctypes.byref(p), None, *ok) == INVALID
    for bad in (dict(wg=None), dict(wu=P + 8), dict(wg_scale=None), dict(wu_scale=P + 2)):
        z = _lib.PmhaFfnQuantized(**{**dict(wg=P, wu=2 * P, wg_scale=5 * P, wu_scale=6 * P), **bad})
        assert lib.pmha_ffn_forward_quantized(ctypes.byref(p), ctypes.byref(z), *ok) == INVALID
    assert lib.pmha_ffn_forward_quantized(ctypes.byref(p), ctypes.byref(q), 8 * P, None, *ok[2:]) == INVALID
    assert lib.pmha_ffn_forward_quantized(ctypes.byref(p), ctypes.byref(q), 8 * P, 10 * P, *ok[2:]) == INVALID  # out over scales


def clip(lib, grads, out=None, numel=None, dtype=None, max_norm=1.0, norm=64 * P, ws=128 * P, n=1 << 30):
    k = len(grads)
    arr = lambda t, v: None if v is None else (t * k)(*v)  # noqa: E731
    return lib.pmha_clip_grad_norm(k, arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, out),
                                   arr(ctypes.c_int64, numel or [64] * k), arr(ctypes.c_int, dtype or [0] * k), max_norm,
                                   norm, ws, n, None)


def test_clip_refusals(lib):
    assert clip(lib, [P, P]) == INVALID and b"given twice" in lib.pmha_last_error()
    assert clip(lib, [P, P + 128]) == INVALID  # overlapping
    assert clip(lib, [P], out=[P + 4]) == INVALID  # neither in place nor apart
    assert clip(lib, [P, 2 * P], out=[2 * P, P]) == INVALID
    assert clip(lib, [P, 2 * P], out=[3 * P, 3 * P]) == INVALID
    assert clip(lib, [64 * P]) == INVALID  # over the norm
    assert clip(lib, [None]) == INVALID and clip(lib, [P + 2]) == INVALID and clip(lib, [P + 1], dtype=[1]) == INVALID
    assert clip(lib, [P], dtype=[9]) == INVALID and clip(lib, [P], numel=[-1]) == INVALID
    for m in (-1.0, float("inf"), float("nan")):
        assert clip(lib, [P], max_norm=m) == INVALID
    assert clip(lib, [P], norm=None) == INVALID and clip(lib, [P], norm=64 * P + 2) == INVALID
    assert clip(lib, [P], ws=None) == WORKSPACE and clip(lib, [P], n=8) == WORKSPACE
    assert lib.pmha_clip_grad_norm(1, None, None, None, None, 1.0, 64 * P, 128 * P, 1 << 30, None) == INVALID
    assert lib.pmha_clip_grad_norm_workspace_size(-1) == 0
    assert lib.pmha_clip_grad_norm_workspace_size(1) < lib.pmha_clip_grad_norm_workspace_size(100000)


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 8), torch.ones(8)
    for call in (lambda: pmha.pmha_rms_norm(x, w, 1e-6), lambda: pmha.pmha_rms_norm_quantized(x, w, 1e-6),
                 lambda: pmha.pmha_rms_norm_backward(x, w, 1e-6, x), lambda: pmha.pmha_clip_grad_norm([x], 1.0),
                 lambda: pmha.pmha_clip_grad_norm([], 1.0), lambda: pmha.pmha_clip_grad_norm([None], 1.0),
                 lambda: pmha.pmha_ffn_forward(pmha.FfnParams(torch.zeros(8, 8), torch.zeros(8, 8), torch.zeros(8, 8)), x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        pmha.pmha_clip_grad_norm(["no tensor"], 1.0)


def test_quantize_rows():
    g = torch.Generator().manual_seed(0)
    w = torch.randn(6, 40, generator=g)
    w[2] = 0.0
    q, s = pmha.quantize_rows(w)
    assert q.dtype == torch.float8_e4m3fn and s.dtype == torch.float32 and s.shape == (6,)
    assert float(s[2]) == 2.0 ** -64 and not q[2].float().any()
    # half a step of 4 significant bits, below 2^-6 half a step of 2^-9
    back = q.float() * s[:, None]
    assert bool(((back - w).abs() <= 2.0 ** -4 * w.abs() + 2.0 ** -10 * s[:, None]).all())


@pytest.mark.parametrize("E,F", [(1, 1), (5, 7), (64, 72), (256, 1024), (1032, 200)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_a_workspace_for_many_rows_serves_fewer(lib, E, F, dtype):
    rows = sorted({1, 2, 16, 63, 64, 65, 100, 256, 257, 1000, 2047, 2048, 2049, 100_000, 1_000_000,
                   *(max(1, n // (E * F) + d) for n in (2048 * F, 1 << 21) for d in (-1, 0, 1))})
    b = ctypes.byref(ffn(E=E, F=F, dtype=dtype))
    for size in (lib.pmha_ffn_forward_workspace_size, lib.pmha_ffn_backward_workspace_size):
        n = [size(b, r) for r in rows]
        assert n == sorted(n)

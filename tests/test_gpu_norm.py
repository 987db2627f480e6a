"""Root-mean-square norm with the residual's addition, its 8-bit output and its
gradients against the formulas in 64 bits."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# widths of every kernel shape: lanes a row, pieces a lane, odd ones, one block a row
WIDTHS = [1, 2, 3, 7, 8, 24, 33, 64, 72, 100, 128, 130, 256, 257, 512, 520, 1000, 1023, 1024, 1025, 1032, 2048, 4099]
ROWS = [1, 2, 5, 67]


def make(rows, width, dtype, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed + 1000 * width + rows)
    x = torch.randn(rows, width, generator=g).to(dtype).to(DEV)
    r = (2 * torch.randn(rows, width, generator=g)).to(dtype).to(DEV) if residual else None
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(dtype).to(DEV)
    return x, r, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward(width, dtype):
    for rows in ROWS:
        for residual in (True, False):
            x, r, w = make(rows, width, dtype, residual=residual)
            for weight in (w, None):
                out, s = pmha.pmha_rms_norm(x, weight, ref.EPS, residual=r)
                kept = x if r is None else (x.float() + r.float()).to(dtype)
                assert (s is None) == (r is None) and (s is None or torch.equal(s, kept))
                y, _ = ref.norm(kept, weight)
                tol = ref.stat_tol(width) + ref.half_ulp(dtype)
                ref.assert_within("out", out, y, 1.01 * tol * y.abs() + 1e-40)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_quantized_is_the_formula_rounded_once(width, dtype):
    for rows in ROWS + [700]:
        x, r, w = make(rows, width, dtype, seed=5)
        q, scale, s = pmha.pmha_rms_norm_quantized(x, w, ref.EPS, residual=r)
        kept = (x.float() + r.float()).to(dtype)
        assert torch.equal(s, kept)
        y, _ = ref.norm(kept, w, eps=float(torch.tensor(ref.EPS, dtype=torch.float32)))
        rq, rscale = ref.quantized(y)
        assert torch.equal(scale, rscale)
        assert torch.equal(q.double(), rq)


def test_quantized_rows_of_zeros_and_infinities():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1.0
    q, scale, _ = pmha.pmha_rms_norm_quantized(x, None, ref.EPS)
    assert float(scale[0]) == 2.0 ** -64 and not q[0].float().any()
    assert scale[1].isnan() and scale[2].isnan() and q[1].float().isnan().all() and q[2].float().isnan().all()
    assert torch.equal(q[3].float(), torch.full((64,), 448.0, device=DEV))
    out, _ = pmha.pmha_rms_norm(x, None, ref.EPS)
    assert not out[0].any() and out[2].isnan().all()


def test_large_and_small_values():
    # squares of 2^60 and 2^-60 are float32 numbers; eps decides the small row
    x = torch.stack([torch.full((256,), 2.0 ** 60), torch.full((256,), 2.0 ** -60)]).to(DEV)
    out, _ = pmha.pmha_rms_norm(x, None, ref.EPS)
    y, _ = ref.norm(x, None)
    ref.assert_within("out", out, y, 2 * ref.stat_tol(256) * y.abs())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(width, dtype):
    for rows in (1, 3, 130, 2100):
        x, ds, w = make(rows, width, dtype, seed=9)
        dy = make(rows, width, dtype, seed=11)[0]
        for weight, dsum in ((w, ds), (w, None), (None, ds)):
            g = pmha.pmha_rms_norm_backward(x, weight, ref.EPS, dy, dsum=dsum)
            dx, mag, dw, dw_mag = ref.norm_backward(x, weight, dy, dsum)
            tol = 4 * ref.stat_tol(width) * mag + ref.half_ulp(dtype) * dx.abs()
            ref.assert_within("dx", g["dx"], dx, 1.01 * tol + 1e-40)
            if weight is None:
                assert g["dweight"] is None
            else:  # a chain of at most rows / 600 + 1 rows, then blocks and warps
                tol = (rows / 600 + 40) * 2.0 ** -24 + ref.stat_tol(width)
                ref.assert_within("dweight", g["dweight"], dw, 1.01 * tol * dw_mag + 1e-40)


def test_backward_is_the_slope():
    # differences of the float64 formula along random directions
    x, _, w = make(5, 48, torch.float32, seed=3)
    dy = make(5, 48, torch.float32, seed=4)[0]
    g = pmha.pmha_rms_norm_backward(x, w, ref.EPS, dy)
    t = torch.Generator().manual_seed(1)
    for _ in range(4):
        vx, vw = (torch.randn(a.shape, generator=t, dtype=torch.float64).to(DEV) for a in (x, w))
        h = 1e-5
        f = [(ref.norm(x.double() + k * vx, w.double() + k * vw)[0] * dy.double()).sum() for k in (h, -h)]
        slope = float((f[0] - f[1]) / (2 * h))
        got = float((g["dx"].double() * vx).sum() + (g["dweight"].double() * vw).sum())
        # differences: h^2 times a third derivative of order 1 a value, and 2^-52 / h; float32 results
        assert abs(got - slope) <= 1e-6 * float((g["dx"].double() * vx).abs().sum() + (g["dweight"].double() * vw).abs().sum())


def test_deterministic_and_rows_zero():
    x, r, w = make(3000, 128, torch.bfloat16)
    a, b = (pmha.pmha_rms_norm_backward(x, w, ref.EPS, r) for _ in range(2))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    e = x[:0]
    out, s = pmha.pmha_rms_norm(e, w, ref.EPS, residual=e)
    assert out.shape == (0, 128) and s.shape == (0, 128)
    g = pmha.pmha_rms_norm_backward(e, w, ref.EPS, e)
    assert g["dx"].shape == (0, 128) and not g["dweight"].any()
    q, scale, _ = pmha.pmha_rms_norm_quantized(e, w, ref.EPS)
    assert q.shape == (0, 128) and scale.shape == (0,)


def test_other_stream_and_captured_graph():
    x, r, w = make(500, 128, torch.bfloat16)
    want, ws = pmha.pmha_rms_norm(x, w, ref.EPS, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, s = pmha.pmha_rms_norm(x, w, ref.EPS, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(s, ws)
    x2 = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, s = pmha.pmha_rms_norm(x2, w, ref.EPS, residual=r)
        g = pmha.pmha_rms_norm_backward(s, w, ref.EPS, out)
    for scale in (1.0, -0.5):
        x2.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        a, b = pmha.pmha_rms_norm(x2, w, ref.EPS, residual=r)
        h = pmha.pmha_rms_norm_backward(b, w, ref.EPS, a)
        assert torch.equal(out, a) and torch.equal(g["dx"], h["dx"]) and torch.equal(g["dweight"], h["dweight"])


def test_refusals():
    x, r, w = make(4, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        pmha.pmha_rms_norm(x.t(), None, ref.EPS)  # not contiguous
    with pytest.raises(ValueError):
        pmha.pmha_rms_norm(x, w.float(), ref.EPS)
    with pytest.raises(ValueError):
        pmha.pmha_rms_norm(x, w, ref.EPS, residual=r[:3])
    with pytest.raises(ValueError):
        pmha.pmha_rms_norm(x.half(), None, ref.EPS)
    for eps in (0.0, float("nan"), float("inf"), -1.0):
        with pytest.raises(pmha.PmhaError):
            pmha.pmha_rms_norm(x, w, eps)
    with pytest.raises(pmha.PmhaError):
        pmha.pmha_rms_norm(x, w, ref.EPS, out=x)  # overlaps its input
    with pytest.raises(pmha.PmhaError):
        pmha.pmha_rms_norm(torch.empty(300, dtype=torch.bfloat16, device=DEV)[1:257].view(4, 64), w, ref.EPS)  # 2-byte aligned

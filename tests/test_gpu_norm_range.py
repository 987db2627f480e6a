"""The norm at the ends of its types: rows whose squares leave float32, up to the
largest finite values, against the formulas in 64 bits."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
# rows that share a warp, one row a warp in one and several pieces, odd ones, one block a row
WIDTHS = [8, 48, 128, 256, 257, 1000, 1023, 1032, 2048, 4099]
# one row each, so that rows of every size stand side by side in a warp; past 2^64 the squares leave float32
SIZES = [1e-18, 1.0, 2.0 ** 60, 2.0 ** 62, 2.0 ** 64, 2.0 ** 65, 1e25, 2.0 ** 96, 1e37, 3e37, 1e38, 3.3e38, 1.0]


def rows_of_every_size(width, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + width)
    s = torch.tensor(SIZES, dtype=torch.float64)[:, None]
    u = 0.3 + 0.7 * torch.rand(len(SIZES), width, generator=g, dtype=torch.float64)
    x = s * u * torch.randn(len(SIZES), width, generator=g).sign()
    w = 1 + 0.2 * torch.randn(width, generator=g)
    return x.to(dtype).to(DEV), w.to(dtype).to(DEV)


@DTYPES
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("eps", [ref.EPS, 1e30])
def test_forward(width, dtype, eps):
    x, w = rows_of_every_size(width, dtype)
    half = x * 0.5  # with itself as the residual the sum is x again
    for weight in (w, None):
        for a, b in ((x, None), (half, half)):
            out, s = pmha.pmha_rms_norm(a, weight, eps, residual=b)
            assert s is None or torch.equal(s, x)
            y, _ = ref.norm(x, weight, eps=float(torch.tensor(eps, dtype=torch.float32)))
            # as for rows of any size; what falls below the normal numbers is off by half of the smallest one at most
            ref.assert_within("out", out, y, 1.01 * (ref.stat_tol(width) + ref.half_ulp(dtype)) * y.abs()
                              + torch.finfo(dtype).smallest_normal)


@DTYPES
@pytest.mark.parametrize("width", WIDTHS)
def test_quantized_is_the_formula_rounded_once(width, dtype):
    x, w = rows_of_every_size(width, dtype)
    x = x[1:].clone()  # the first row's squares are below float32's normal numbers
    q, scale, _ = pmha.pmha_rms_norm_quantized(x, w, ref.EPS)
    y, _ = ref.norm(x, w, eps=float(torch.tensor(ref.EPS, dtype=torch.float32)))
    rq, rscale = ref.quantized(y)
    assert torch.equal(scale, rscale)
    assert torch.equal(q.double(), rq)


@DTYPES
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(width, dtype):
    x, w = rows_of_every_size(width, dtype)
    g = torch.Generator().manual_seed(width)
    # gradients large enough for those of the largest rows, 1e-39 of them, to be normal numbers
    dy, ds = ((s * torch.randn(x.shape, generator=g)).to(dtype).to(DEV) for s in (2.0 ** 30, 2.0 ** -40))
    for dsum in (None, ds):
        got = pmha.pmha_rms_norm_backward(x, w, ref.EPS, dy, dsum=dsum)
        dx, mag, dw, dw_mag = ref.norm_backward(x, w, dy, dsum)
        tol = 4 * ref.stat_tol(width) * mag + ref.half_ulp(dtype) * dx.abs() + torch.finfo(dtype).smallest_normal
        ref.assert_within("dx", got["dx"], dx, 1.01 * tol)
        ref.assert_within("dweight", got["dweight"], dw, 1.01 * (40 * 2.0 ** -24 + ref.stat_tol(width)) * dw_mag)


@DTYPES
@pytest.mark.parametrize("width", WIDTHS)
def test_backward_of_large_rows_and_large_gradients(width, dtype):
    # x = 2^58 and dout = 2^64 are ordinary numbers whose products' sum is not: dx is some 2^6
    g = torch.Generator().manual_seed(width)
    u = 0.5 + 0.5 * torch.rand(5, width, generator=g)
    w = 1 + 0.2 * torch.randn(width, generator=g)
    sizes = torch.tensor([2.0 ** 58, 2.0 ** 62, 1.0, 2.0 ** -20, 2.0 ** 100])[:, None]
    x, w = (sizes * u).to(dtype).to(DEV), w.to(dtype).to(DEV)
    dy = (2.0 ** 64 * (0.5 + 0.5 * torch.rand(5, width, generator=g))).to(dtype).to(DEV)  # of one sign: nothing cancels
    ds = torch.randn(5, width, generator=g).to(dtype).to(DEV)
    for dsum in (None, ds):
        got = pmha.pmha_rms_norm_backward(x, w, ref.EPS, dy, dsum=dsum)
        dx, mag, dw, dw_mag = ref.norm_backward(x, w, dy, dsum)
        tol = 4 * ref.stat_tol(width) * mag + ref.half_ulp(dtype) * dx.abs() + torch.finfo(dtype).smallest_normal
        ref.assert_within("dx", got["dx"], dx, 1.01 * tol)
        ref.assert_within("dweight", got["dweight"], dw, 1.01 * (40 * 2.0 ** -24 + ref.stat_tol(width)) * dw_mag)


@DTYPES
@pytest.mark.parametrize("width", WIDTHS)
def test_quantized_rows_times_large_weights(width, dtype):
    # rows of 2^58 whose squares are float32 numbers, weights of 2^72: their products are not, the norm's values are
    g = torch.Generator().manual_seed(width)
    u = 0.5 + 0.5 * torch.rand(4, width, generator=g)
    x = (torch.tensor([2.0 ** 55, 1.0, 2.0 ** 58, 2.0 ** 100])[:, None] * u).to(dtype).to(DEV)
    w = (2.0 ** 72 * torch.randn(width, generator=g)).to(dtype).to(DEV)
    q, scale, _ = pmha.pmha_rms_norm_quantized(x, w, ref.EPS)
    y, _ = ref.norm(x, w, eps=float(torch.tensor(ref.EPS, dtype=torch.float32)))
    rq, rscale = ref.quantized(y)
    assert torch.equal(scale, rscale)
    assert torch.equal(q.double(), rq)


@DTYPES
@pytest.mark.parametrize("width", [7, 64, 256, 1500])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 40, 2.0 ** 52, 2.0 ** 58, 2.0 ** 62])
def test_quantized_keeps_its_pairs_of_floats(width, dtype, size):
    # the inverse of a large mean square has a second float below the normal numbers: over 20,000 rows some scales show it
    g = torch.Generator(device=DEV).manual_seed(width)
    x = (size * torch.randn(20_000, width, generator=g, device=DEV)).to(dtype)
    w = (1 + 0.2 * torch.randn(width, generator=g, device=DEV)).to(dtype)
    q, scale, _ = pmha.pmha_rms_norm_quantized(x, w, ref.EPS)
    y, _ = ref.norm(x, w, eps=float(torch.tensor(ref.EPS, dtype=torch.float32)))
    rq, rscale = ref.quantized(y)
    assert torch.equal(scale, rscale)
    assert torch.equal(q.double(), rq)

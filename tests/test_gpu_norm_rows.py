"""The norm's gradients over so many rows that every warp and block walks several:
the ring of copies in its steady state, and sums whose error does not grow with the rows."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])

# A column's terms are added in float32 for 128 steps at most, then those of up to 4 lanes and 8 warps; a block's
# sum is added to the others' in pairs of floats.
FOLD = 128


@DTYPES
@pytest.mark.parametrize("rows,width", [(12001, 256), (25001, 128), (40001, 48), (20003, 512), (9001, 600), (9001, 257),
                                        (5003, 1023), (4001, 2048), (3001, 1025)])
def test_backward_in_several_steps(rows, width, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows + width)
    x, dy, ds = (torch.randn(rows, width, generator=g, device=DEV).to(dtype) for _ in range(3))
    w = (1 + 0.2 * torch.randn(width, generator=g, device=DEV)).to(dtype)
    for dsum in (ds, None):
        got = pmha.pmha_rms_norm_backward(x, w, ref.EPS, dy, dsum=dsum)
        dx, mag, dw, dw_mag = ref.norm_backward(x, w, dy, dsum)
        tol = 4 * ref.stat_tol(width) * mag + ref.half_ulp(dtype) * dx.abs()
        ref.assert_within("dx", got["dx"], dx, 1.01 * tol + 1e-40)
        tol = (FOLD + 16) * 2.0 ** -24 + ref.stat_tol(width)
        ref.assert_within("dweight", got["dweight"], dw, 1.01 * tol * dw_mag + 1e-40)
        # most of a sum of either sign cancels: the whole of it is far closer than its terms allow
        assert float((got["dweight"].double() - dw).norm() / dw.norm()) <= 1e-5
        only = pmha.pmha_rms_norm_backward(x, w, ref.EPS, dy, dsum=dsum, input_grad=False)
        assert only["dx"] is None and torch.equal(only["dweight"], got["dweight"])


@DTYPES
@pytest.mark.parametrize("rows,width", [(60_000_000, 8), (2_000_000, 1032)])
def test_weight_gradients_of_one_sign(rows, width, dtype):
    # every row is the same, so that each addition of a chain is off to the same side: n terms by up to n / 2
    # roundings of their sum. A chain of all of a warp's or block's rows would have some 3,000 terms here.
    if dtype == torch.float32 and width > 1024:
        rows //= 2
    g = torch.Generator().manual_seed(width)
    x1 = (0.5 + torch.rand(width, generator=g)).to(dtype).to(DEV)
    dy1 = (0.1 + 0.8 * torch.rand(width, generator=g)).to(dtype).to(DEV)
    x, dy = (t.expand(rows, width).contiguous() for t in (x1, dy1))
    got = pmha.pmha_rms_norm_backward(x, torch.ones_like(x1), ref.EPS, dy, input_grad=False)["dweight"]
    y, _ = ref.norm(x1[None], None)
    want = rows * dy1.double() * y[0]
    ref.assert_within("dweight", got, want, ((FOLD / 2 + 16) * 2.0 ** -24 + ref.stat_tol(width)) * want.abs())


def test_workspace_grows_with_rows_and_holds_nothing_between_calls():
    lib = pmha._lib.load()
    for width in (48, 256, 1025, 4096):
        n = [lib.pmha_rms_norm_backward_workspace_size(1, r, width) for r in (1, 500, 70_000, 80_000, 1_000_000)]
        assert n == sorted(n) and n[0] % 256 == 0

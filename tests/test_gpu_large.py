"""Encoder operators past 2 GiB of hidden rows (which the forward pass then takes in
blocks of rows) and past 2^31 values of a tensor."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as ref
from tests.test_gpu_ffn import BF16, DEV, F32, block, make

pytestmark = pytest.mark.gpu


def check_pieces(y, p, x, residual, b=None, scale=None, step=20_000):
    b = b or block(p)
    for r in range(0, x.shape[0], step):
        part = slice(r, min(x.shape[0], r + step))
        xs = x[part].double() if scale is None else x[part].double() * scale[part].double()[:, None]
        want, bound = b.forward(xs, None if residual is None else residual[part])
        ref.assert_within(f"y from {r}", y[part], want, bound)


# tile by tile, with padded widths, padded and on the chip, float32
@pytest.mark.parametrize("rows,E,F,dtype", [(300_001, 16, 4096, BF16), (320_003, 12, 3500, BF16), (560_001, 12, 2000, BF16),
                                            (140_001, 20, 4096, F32)])
def test_forward_in_blocks_of_rows(rows, E, F, dtype):
    assert rows * F * (2 if dtype == BF16 else 4) > 2 ** 31
    p, x, r = make(rows, E, F, dtype)
    y = pmha.pmha_ffn_forward(p, x, residual=r)
    pmha.pmha_device_status()
    check_pieces(y, p, x, r)


def test_forward_from_8_bits_in_blocks_of_rows():
    rows, E, F = 300_001, 16, 4096
    p, x, r = make(rows, E, F, BF16, act="gelu")
    q = pmha.FfnQuantizedParams.from_params(p)
    x8, xs, _ = pmha.pmha_rms_norm_quantized(x, None, ref.EPS)
    y = pmha.pmha_ffn_forward_quantized(q, x8, xs, residual=r)
    pmha.pmha_device_status()
    b = ref.Block(q.wg.double() * q.wg_scale.double()[:, None], q.wu.double() * q.wu_scale.double()[:, None], p.wd, p.bg,
                  p.bu, p.bd, "gelu")
    check_pieces(y, p, x8, r, b, xs)


# rows of a warp each, and of a block each
@pytest.mark.parametrize("rows,width", [(17_000_003, 128), (1_060_001, 2048)])
def test_norm_of_more_than_2_to_31_values(rows, width):
    assert rows * width > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(width)
    few = torch.randn(1000, width, generator=g, device=DEV).to(BF16)
    x = few.repeat(rows // 1000 + 1, 1)[:rows]
    w = (1 + 0.2 * torch.randn(width, generator=g, device=DEV)).to(BF16)
    out, s = pmha.pmha_rms_norm(x, w, ref.EPS, residual=x)
    want, ws = pmha.pmha_rms_norm(few, w, ref.EPS, residual=few)
    ends = [(slice(0, 1000), slice(0, 1000)), (slice(rows - rows % 1000, rows), slice(0, rows % 1000))]
    middle = (2 ** 31 // width - 500) // 1000 * 1000
    ends.append((slice(middle, middle + 1000), slice(0, 1000)))
    for a, b in ends:
        assert torch.equal(out[a], want[b]) and torch.equal(s[a], ws[b])
    q, scale, _ = pmha.pmha_rms_norm_quantized(x, w, ref.EPS)
    wq, wscale, _ = pmha.pmha_rms_norm_quantized(few, w, ref.EPS)
    for a, b in ends:
        assert torch.equal(q[a].view(torch.uint8), wq[b].view(torch.uint8)) and torch.equal(scale[a], wscale[b])
    del q, out
    got = pmha.pmha_rms_norm_backward(x, w, ref.EPS, s)
    few_got = pmha.pmha_rms_norm_backward(few, w, ref.EPS, ws)
    for a, b in ends:
        assert torch.equal(got["dx"][a], few_got["dx"][b])
    _, _, dw, mag = ref.norm_backward(few, w, ws, None)
    _, _, tail, tail_mag = ref.norm_backward(few[:rows % 1000], w, ws[:rows % 1000], None)
    k = rows // 1000
    tol = (128 + 16) * 2.0 ** -24 + ref.stat_tol(width)
    ref.assert_within("dweight", got["dweight"], k * dw + tail, tol * (k * mag + tail_mag))


def test_block_of_more_than_2_to_31_values():
    rows, E, F = 17_000_003, 128, 64
    p, few, _ = make(1000, E, F, BF16)
    x = few.repeat(rows // 1000 + 1, 1)[:rows]
    y = pmha.pmha_ffn_forward(p, x, residual=x)
    pmha.pmha_device_status()
    want, bound = block(p).forward(few, few)
    n = rows % 1000
    ref.assert_within("first", y[:1000], want, bound)
    ref.assert_within("last", y[rows - n:], want[:n], bound[:n])
    middle = 2 ** 31 // E // 1000 * 1000
    ref.assert_within("middle", y[middle:middle + 1000], want, bound)
    del y
    got = pmha.pmha_ffn_backward(p, x, x)
    pmha.pmha_device_status()
    grads = block(p).backward(few, few)
    ref.assert_within("dx first", got["dx"][:1000], *grads["dx"])
    ref.assert_within("dx last", got["dx"][rows - n:], grads["dx"][0][:n], grads["dx"][1][:n])
    tail = block(p).backward(few[:n], few[:n])
    for name in ("dwg", "dwu", "dwd", "dbg", "dbu", "dbd"):
        total = rows // 1000 * grads[name][0] + tail[name][0]
        # rounding errors of the same 1,000 rows add up: 2^-9 of h, dg and du and of the result, sums in float32
        assert float((got[name].double() - total).norm() / total.norm()) <= 3 * 2.0 ** -9, name

"""Gradients of the gated block and of the encoder layer as a whole: next to the
bounds a value (which grow with the rows, as sums of worst cases do) their
distance from the 64-bit formulas in norm, which a lost row shows in."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import test_gpu_encoder as layers
from tests import test_gpu_ffn as plain
from tests.test_gpu_ffn import BF16, DEV, F32, block, make

pytestmark = pytest.mark.gpu
WEIGHTS = ("dwg", "dwu", "dwd", "dx")

# bf16: h, dg and du, and then the result, are off by 2^-9 of a value at most; as independent errors of terms of either
# sign they add up to less than 2 x 2^-9 of the norm. float32: chains of 256 to 450 terms, whose running sums are
# off by 2.4e-8 (rms) an addition, leave 4e-7, those of the factors' sums of E terms as much again in each.
BAR = {BF16: 3 * 2.0 ** -9, F32: 2e-6}


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def reference(p, x, dy, step=20_000):
    """{name: gradient} in 64 bits, by pieces of the rows."""
    out = {}
    for r in range(0, x.shape[0], step):
        for n, (v, _) in block(p).backward(x[r:r + step], dy[r:r + step]).items():
            if n == "dx":
                out.setdefault(n, []).append(v)
            else:
                out[n] = out[n] + v if n in out else v
    out["dx"] = torch.cat(out["dx"])
    return out


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,E,F,dtype", [(*s, BF16) for s in plain.LONG + plain.BIG] + [(*s, F32) for s in plain.F32_LONG])
def test_gradients_in_norm(rows, E, F, dtype, act):
    p, x, dy = make(rows, E, F, dtype, act=act)
    got = pmha.pmha_ffn_backward(p, x, dy)
    pmha.pmha_device_status()
    want = reference(p, x, dy)
    for n in WEIGHTS:
        assert rel(got[n], want[n]) <= BAR[dtype], n
    # the bar sees a lost block of 64 rows, wherever it is
    for r in (0, rows // 2 // 64 * 64, (rows - 1) // 64 * 64 - 64):
        cut = block(p).backward(x[r:r + 64], dy[r:r + 64])
        for n in ("dwg", "dwu", "dwd"):
            assert rel(got[n], want[n] - cut[n][0]) > 2 * BAR[dtype], n


@pytest.mark.parametrize("rows,E,F,dtype", [(2300, 8, 72, BF16), (2500, 128, 512, BF16), (3001, 192, 264, BF16),
                                            (2200, 72, 4096, BF16), (9001, 320, 72, BF16), (3000, 328, 1032, BF16),
                                            (20011, 100, 171, BF16), (5000, 130, 260, F32), (300, 24, 40, BF16)])
def test_one_row_alone(rows, E, F, dtype):
    # dout is zero but in one row: at the ends of tiles, of blocks of K, of splits, and of the rows
    p, x, full = make(rows, E, F, dtype)
    names = ("dwg", "dwu", "dwd", "dbg", "dbu", "dbd")
    for r in sorted({0, 63, 64, 127, 128, 255, 256, rows // 2, (rows - 1) // 256 * 256, (rows - 1) // 64 * 64 - 1, rows - 2, rows - 1}):
        dy = torch.zeros_like(full)
        dy[r] = full[r]
        got = pmha.pmha_ffn_backward(p, x, dy)
        want = block(p).backward(x[r:r + 1], dy[r:r + 1])
        for n in names:
            assert rel(got[n], want[n][0]) <= BAR[dtype], (n, r)
        assert rel(got["dx"][r:r + 1], want["dx"][0]) <= BAR[dtype], r
        got["dx"][r] = 0
        assert not got["dx"].any(), r
    pmha.pmha_device_status()


# hidden rows of more than 2 GiB, which are taken in blocks of rows
@pytest.mark.parametrize("rows,E,F,dtype", [(100_001, 16, 4096, BF16), (190_000, 128, 2048, BF16),
                                            (180_001, 200, 2048, BF16), (120_000, 12, 3500, BF16), (50_001, 20, 4096, F32)])
def test_rows_here_and_there(rows, E, F, dtype):
    # every 61st row and the last: one in every block of 64, so that a lost one of them takes one of 1,600 with it
    p, x, full = make(rows, E, F, dtype)
    at = torch.cat([torch.arange(0, rows, 61), torch.tensor([rows - 1])]).unique().to(DEV)
    dy = torch.zeros_like(full)
    dy[at] = full[at]
    got = pmha.pmha_ffn_backward(p, x, dy)
    pmha.pmha_device_status()
    want = reference(p, x[at], dy[at])
    for n in ("dwg", "dwu", "dwd", "dbg", "dbu", "dbd"):
        assert rel(got[n], want[n]) <= BAR[dtype], n
    assert rel(got["dx"][at], want["dx"]) <= BAR[dtype]
    got["dx"][at] = 0
    assert not got["dx"].any()
    one = block(p).backward(x[at[-1:]], dy[at[-1:]])  # the bar sees the last row
    for n in ("dwg", "dwu", "dwd"):
        assert rel(got[n], want[n] - one[n][0]) > 2 * BAR[dtype], n


@pytest.mark.parametrize("n,nnz,B,E,H,F,dt", [(64, 256, 2, 32, 4, 88, "f32"), (300, 3000, 2, 128, 8, 344, "bf16"),
                                              (130, 900, 1, 256, 8, 512, "bf16"), (700, 9000, 3, 64, 4, 171, "bf16")])
def test_layer_gradients_in_norm(n, nnz, B, E, H, F, dt):
    # The longest way to a gradient goes through some 16 results rounded to 16 bits (norms, sums, projections, h, dg,
    # du, the gradients of each), 2^-9 at most each and independent: 2^-7 of the norm; the softmax's differences
    # and the norms' projections, which take a part of the gradient out, leave four times that at most. float32: the
    # same count at 2^-22 (a sum's some 4 roundings of 2^-24) is 2^-18.
    layer, x, dy, spec = layers.make(n, nnz, B, E, H, F, dt, seed=11)
    y, grads = layer(x), layer.backward(x, dy)
    pmha.pmha_device_status()
    want, leaf = layers.plain(layer, x, spec)
    want.backward(dy.double())
    bar = 2.0 ** -5 if dt == "bf16" else 2.0 ** -18
    assert rel(y, want.detach()) <= bar
    for name, v in leaf.items():
        if name != "bk":  # zero in exact arithmetic
            assert rel(grads["dx" if name == "x" else "d" + name], v.grad) <= bar, name


def test_weight_gradients_of_one_sign():
    # Sums over many rows of a narrow block, all terms positive: cut at each of 4,096 additions by up to 2^-22 of the
    # running sum (two bits below float32's) they are off by 2^-11 at most, to one side. The gradients of a row of the
    # weights are all alike here, so that their roundings to bf16 may go one way too: 2^-9.
    rows, E, F = 20_000_000, 64, 16
    g = torch.Generator(device=DEV).manual_seed(4)

    def r(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    p = pmha.FfnParams(*((t / E * 2).to(BF16) for t in (r(F, E), r(F, E))), (r(E, F) / F).to(BF16))
    x, dy = (0.5 + r(rows, E)).to(BF16), (0.5 + r(rows, E)).to(BF16)
    got = pmha.pmha_ffn_backward(p, x, dy, input_grads=False)
    pmha.pmha_device_status()
    want = {}
    for at in range(0, rows, 200_000):
        for n, (v, _) in block(p).backward(x[at:at + 200_000], dy[at:at + 200_000]).items():
            if n in ("dwg", "dwu", "dwd"):
                want[n] = want.get(n, 0) + v
    for n, v in want.items():
        assert bool((v > 0).all())
        off = float((got[n].double() / v - 1).mean())
        assert abs(off) <= 2.0 ** -11 + 2.0 ** -9, (n, off)

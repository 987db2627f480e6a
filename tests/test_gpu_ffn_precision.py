"""What the gated block's sums keep: bias gradients rounded once, long float32
sums folded, columns that do not touch one another, and workspaces of a larger batch."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as ref
from tests import test_gpu_ffn as plain
from tests.test_gpu_ffn import BF16, DEV, F32, block, make

pytestmark = pytest.mark.gpu


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


# both kernels that form the hidden gradients: one that keeps the tokens on the chip, one tile by tile
@pytest.mark.parametrize("rows,E,F", [(5000, 64, 520), (6001, 200, 264), (20000, 24, 2048), (4000, 320, 1000)])
def test_bias_gradients_are_rounded_once(rows, E, F):
    # float32 sums of float32 terms: next to the one rounding to bf16 (2^-9 / sqrt(3) of a value, rms) they add some
    # sqrt(rows) 2^-24, a few percent at most. Sums of terms rounded to bf16 are off by as much again: 1.41 times.
    p, x, dy = make(rows, E, F, BF16)
    got = pmha.pmha_ffn_backward(p, x, dy)
    pmha.pmha_device_status()
    want = block(p).backward(x, dy)
    for n in ("dbg", "dbu", "dbd"):
        v = want[n][0]
        assert rel(got[n], v) <= 1.2 * rel(v.to(BF16), v)


@pytest.mark.parametrize("rows,E,F", [(97, 928, 2976), (7, 1008, 1928), (2, 656, 1536)])
def test_long_float32_sums(rows, E, F):
    # A sum of K terms of either sign in ascending order has a running value of sqrt(k) terms, each addition off by
    # 2.4e-8 of it (rms of a rounding to 24 bits): sqrt(K / 2) 2.4e-8 of the result, 2.7e-7 for pieces of 256 and
    # 8e-8 for some 20 of them; its factors, sums of E terms, bring 2.7e-7 (in two products) each: 6e-7 in all. In
    # one piece of 2 F the sum alone is off by 1.3e-6 and more at these widths.
    p, x, dy = make(rows, E, F, F32)
    got = pmha.pmha_ffn_backward(p, x, dy)
    want = block(p).backward(x, dy)
    assert rel(got["dx"], want["dx"][0]) <= 9e-7
    y = pmha.pmha_ffn_forward(p, x)
    assert rel(y, block(p).forward(x, None)[0]) <= 9e-7


@pytest.mark.parametrize("rows,E,F", [(5000, 64, 520), (4000, 320, 264), (40, 24, 40)])
def test_an_infinite_column_stays_one_column(rows, E, F):
    p, x, dy = make(rows, E, F, BF16)
    clean = pmha.pmha_ffn_backward(p, x, dy)
    p.wd[:, 17] = float("inf")
    got = pmha.pmha_ffn_backward(p, x, dy)
    pmha.pmha_device_status()
    for n in ("dbg", "dbu", "dwg", "dwu"):
        assert not torch.isfinite(got[n][17]).any()
        for part in (slice(0, 17), slice(18, F)):
            assert torch.equal(got[n][part], clean[n][part])
    assert torch.equal(got["dbd"], clean["dbd"]) and torch.equal(got["dwd"], clean["dwd"])


@pytest.mark.parametrize("rows,E,F", [(3000, 64, 64), (3000, 128, 200), (600, 320, 72), (9, 64, 64)])
def test_gate_far_below_zero_times_a_large_up(rows, E, F):
    # silu(g) u with g = -2^66, u = 2^66: the gate's factor is 0, also where g u leaves float32
    p, x, r = make(rows, E, F, BF16, bias=False)
    x = torch.zeros_like(x)
    x[:, 0] = 2.0 ** 40
    p.wg[:], p.wu[:] = 0, 0
    p.wg[:, 0], p.wu[:, 0] = -(2.0 ** 26), 2.0 ** 26
    y = pmha.pmha_ffn_forward(p, x, residual=r)
    pmha.pmha_device_status()
    assert torch.equal(y, r)


@pytest.mark.parametrize("E,F", [(64, 72), (100, 33), (256, 1024), (320, 264)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_workspace_for_many_rows_runs_fewer(E, F, dtype):
    p, x, dy = make(4000, E, F, dtype)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in
          (pmha.pmha_ffn_forward_workspace_size(p, 4000), pmha.pmha_ffn_backward_workspace_size(p, 4000))]
    for rows in (1, 17, 64, 65, 700, 2047, 2048, 4000):
        a, b = x[:rows].clone(), dy[:rows].clone()
        for t in ws:
            t.fill_(255)  # NaN wherever a value is read before it is written
        y = pmha.pmha_ffn_forward(p, a, residual=b, workspace=ws[0])
        want, bound = block(p).forward(a, b)
        ref.assert_within(f"y {rows}", y, want, bound)
        g = pmha.pmha_ffn_backward(p, a, b, workspace=ws[1])
        pmha.pmha_device_status()
        for n, (v, e) in block(p).backward(a, b).items():
            ref.assert_within(f"{n} {rows}", g[n], v, e)


def test_two_streams_at_once():
    # calls that overlap on the device, each with its own workspace: the same results as alone
    cases = [make(3000, 128, 512, BF16), make(700, 320, 264, BF16, act="gelu"), make(5, 256, 1024, BF16)]
    alone = [(pmha.pmha_ffn_forward(p, x, residual=dy), pmha.pmha_ffn_backward(p, x, dy)) for p, x, dy in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        both = [(pmha.pmha_ffn_forward(p, x, residual=dy, stream=s), pmha.pmha_ffn_backward(p, x, dy, stream=s))
                for (p, x, dy), s in zip(cases, streams)]
        torch.cuda.synchronize()
        pmha.pmha_device_status()
        for (y, g), (y1, g1) in zip(both, alone):
            assert torch.equal(y, y1) and all(torch.equal(g[n], g1[n]) for n in g)


# hidden rows of more than 2 GiB: tile by tile, kept on the chip with and without dx, padded widths, float32
@pytest.mark.parametrize("rows,E,F,dtype", [(100_001, 16, 4096, BF16), (190_000, 128, 2048, BF16),
                                            (180_001, 200, 2048, BF16), (120_000, 12, 3500, BF16), (50_001, 20, 4096, F32)])
def test_several_blocks_of_rows(rows, E, F, dtype):
    p, x, dy = make(rows, E, F, dtype)
    got = pmha.pmha_ffn_backward(p, x, dy)
    y = pmha.pmha_ffn_forward(p, x, residual=dy)
    pmha.pmha_device_status()
    b, sums = block(p), {}
    step = 20_000
    for r in range(0, rows, step):
        part = slice(r, min(rows, r + step))
        want, bound = b.forward(x[part], dy[part])
        ref.assert_within(f"y from {r}", y[part], want, bound)
        for n, (v, e) in b.backward(x[part], dy[part]).items():
            if n == "dx":
                ref.assert_within(f"dx from {r}", got["dx"][part], v, e)
            else:
                sums[n] = [a + c for a, c in zip(sums[n], (v, e))] if n in sums else [v, e]
    for n, (v, e) in sums.items():
        ref.assert_within(n, got[n], v, e)


@pytest.mark.parametrize("rows,E,F", [(3000, 128, 512), (40, 256, 1024), (700, 320, 264)])
def test_captured_and_replayed(rows, E, F):
    # one graph of the forward and backward pass: replays on new inputs give what the calls give
    p, x, dy = make(rows, E, F, BF16)
    x_in, dy_in = x.clone(), dy.clone()
    pmha.pmha_ffn_forward(p, x_in, residual=dy_in), pmha.pmha_ffn_backward(p, x_in, dy_in)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = pmha.pmha_ffn_forward(p, x_in, residual=dy_in)
        g = pmha.pmha_ffn_backward(p, x_in, dy_in)
    for k in range(3):
        x_in.copy_(x.roll(k, 0)), dy_in.copy_(dy.roll(2 * k, 0))
        graph.replay()
        torch.cuda.synchronize()
        a, b = x.roll(k, 0), dy.roll(2 * k, 0)
        assert torch.equal(y, pmha.pmha_ffn_forward(p, a, residual=b))
        w = pmha.pmha_ffn_backward(p, a, b)
        assert all(torch.equal(g[n], w[n]) for n in w)
    pmha.pmha_device_status()


# the kernel that keeps the hidden rows on the chip, at every embed_dim it has, with ragged ends and short and long
# hidden widths (it runs from some rows on: fewer for narrow blocks), each with a second round of row blocks
CHIP = [(70, 64, 128), (300, 40, 264), (5000, 128, 264), (16500, 72, 2048), (41000, 128, 136), (4000, 192, 264),
        (20001, 136, 1032), (4100, 256, 320), (16400, 256, 2048), (25000, 200, 72)]


@pytest.mark.parametrize("rows,E,F", CHIP)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward_on_the_chip(rows, E, F, act):
    plain.check_forward(rows, E, F, BF16, bias=True, act=act, residual=rows % 2 == 0)
    plain.check_forward(rows, E, F, BF16, bias=False, act=act, residual=rows % 2 == 1)


@pytest.mark.parametrize("rows,E,F", [(70, 64, 128), (5000, 128, 264), (16500, 80, 2048), (4000, 192, 264),
                                      (20001, 144, 1032), (41000, 256, 72)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_quantized_on_the_chip(rows, E, F, act):
    plain.test_forward_quantized(rows, E, F, act)

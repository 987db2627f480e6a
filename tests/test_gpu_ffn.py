"""The gated feed-forward block, forward, from 8-bit tokens and backward, against
its formulas in 64 bits with counted error bounds."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def make(rows, E, F, dtype, bias=True, act="silu", seed=0):
    g = torch.Generator().manual_seed(seed + rows + 7 * E + 13 * F)

    def n(*shape, s=1.0):
        return (torch.randn(*shape, generator=g) * s).to(dtype).to(DEV)

    b = (n(F, s=0.3), n(F, s=0.3), n(E, s=0.3)) if bias else (None, None, None)
    p = pmha.FfnParams(n(F, E, s=E ** -0.5), n(F, E, s=E ** -0.5), n(E, F, s=F ** -0.5), *b, act=act)
    return p, n(rows, E), n(rows, E)


def block(p):
    return ref.Block(p.wg, p.wu, p.wd, p.bg, p.bu, p.bd, p.act)


def check_forward(rows, E, F, dtype, bias=True, act="silu", residual=True):
    p, x, r = make(rows, E, F, dtype, bias, act)
    y = pmha.pmha_ffn_forward(p, x, residual=r if residual else None)
    pmha.pmha_device_status()
    want, bound = block(p).forward(x, r if residual else None)
    ref.assert_within(f"y {rows} {E} {F}", y, want, bound)


def check_backward(rows, E, F, dtype, bias=True, act="silu"):
    p, x, dy = make(rows, E, F, dtype, bias, act)
    got = pmha.pmha_ffn_backward(p, x, dy)
    pmha.pmha_device_status()
    want = block(p).backward(x, dy)
    for n, (v, e) in want.items():
        if n.startswith("db") and not bias:
            assert got[n] is None
            continue
        ref.assert_within(f"{n} {rows} {E} {F}", got[n], v, e)


# one tile, ragged tiles, several tiles, both column-tile widths, K past one block, padded widths
SHAPES = [(256, 128, 128), (1, 64, 64), (128, 64, 128), (129, 64, 64), (255, 8, 8), (257, 72, 200), (300, 256, 136),
          (1000, 128, 512), (513, 320, 264), (700, 576, 128), (1, 256, 1024), (33, 512, 2048), (2, 1024, 96)]
# rows enough for the kernel that keeps the hidden rows on the chip, every width it has, ragged ends
LONG = [(2048, 64, 64), (2300, 8, 72), (2500, 128, 512), (3001, 192, 264), (2049, 256, 1024), (40000, 128, 136),
        (2200, 72, 4096), (2600, 248, 8)]
# a few tokens: the kernels that read each weight once on the CUDA cores
FEW = [(1, 8, 8), (1, 128, 512), (3, 256, 1000), (4, 100, 171), (5, 64, 72), (16, 512, 2048), (16, 33, 65), (2, 4096, 264),
       (7, 1024, 4097), (40, 72, 520), (64, 129, 264)]
ODD = [(5, 1, 1), (3, 7, 9), (130, 33, 65), (257, 100, 171), (64, 130, 514)]


@pytest.mark.parametrize("rows,E,F", SHAPES + LONG + FEW + ODD + [(2055, 100, 171)])
def test_forward_bf16(rows, E, F):
    check_forward(rows, E, F, BF16, bias=(rows + E) % 2 == 0, residual=F % 16 != 0 or rows % 2 == 1)
    check_forward(rows, E, F, BF16, bias=True, act="gelu", residual=True)


F32_LONG = [(5000, 130, 260), (20000, 33, 65)]


@pytest.mark.parametrize("rows,E,F", SHAPES[:9] + ODD + F32_LONG)
def test_forward_f32(rows, E, F):
    check_forward(rows, E, F, F32, bias=(rows + E) % 2 == 0, residual=rows % 2 == 1)
    check_forward(rows, E, F, F32, act="gelu")


# past the small problems that run in float32: fused or not, padded widths, K tails
BIG = [(40000, 64, 64), (30000, 136, 264), (9000, 320, 72), (5000, 192, 520), (12001, 256, 600), (20011, 100, 171),
       (3000, 328, 1032)]


@pytest.mark.parametrize("rows,E,F", SHAPES + LONG + BIG + ODD)
def test_backward_bf16(rows, E, F):
    check_backward(rows, E, F, BF16)
    check_backward(rows, E, F, BF16, bias=False, act="gelu")


@pytest.mark.parametrize("rows,E,F", SHAPES[:9] + ODD + F32_LONG)
def test_backward_f32(rows, E, F):
    check_backward(rows, E, F, F32)
    check_backward(rows, E, F, F32, bias=False, act="gelu")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_more_rows_than_a_block(dtype):
    # many rows of a wide block (test_gpu_ffn_precision.py has those of several blocks of rows)
    check_forward(9000 if dtype == BF16 else 5000, 32, 4096, dtype)
    check_backward(4500, 32, 4096, dtype)


@pytest.mark.parametrize("rows,E,F", [(256, 128, 128), (1, 16, 8), (100, 48, 72), (300, 256, 264), (1000, 512, 1024),
                                      (4, 128, 512), (16, 80, 136), (2048, 128, 512), (2111, 48, 72), (2300, 192, 200), (2500, 256, 4096)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward_quantized(rows, E, F, act):
    p, x, r = make(rows, E, F, BF16, act=act)
    q = pmha.FfnQuantizedParams.from_params(p)
    x8, xs, _ = pmha.pmha_rms_norm_quantized(x, None, ref.EPS)
    for residual in (r, None):
        y = pmha.pmha_ffn_forward_quantized(q, x8, xs, residual=residual)
        pmha.pmha_device_status()
        b = ref.Block(q.wg.double() * q.wg_scale.double()[:, None], q.wu.double() * q.wu_scale.double()[:, None],
                      p.wd, p.bg, p.bu, p.bd, act)
        want, bound = b.forward(x8.double() * xs.double()[:, None], residual)
        ref.assert_within("y", y, want, bound)


def test_gradient_is_the_slope():
    p, x, dy = make(9, 24, 40, F32, act="gelu")
    got = pmha.pmha_ffn_backward(p, x, dy)
    t = torch.Generator().manual_seed(2)
    names = ("wg", "wu", "wd", "bg", "bu", "bd")
    for _ in range(3):
        v = {n: torch.randn(getattr(p, n).shape, generator=t, dtype=torch.float64).to(DEV) for n in names}
        vx = torch.randn(x.shape, generator=t, dtype=torch.float64).to(DEV)
        f = []
        for h in (1e-5, -1e-5):
            b = block(p)
            b.w = [getattr(p, n).double() + h * v[n] for n in names[:3]]
            b.b = [getattr(p, n).double() + h * v[n] for n in names[3:]]
            f.append(float((b.forward(x.double() + h * vx, None)[0] * dy.double()).sum()))
        terms = [(got["d" + n].double() * v[n]) for n in names] + [got["dx"].double() * vx]
        # float32 gradients (some 2^-20 of the terms) and differences (1e-10 of a third derivative)
        mag = sum(float(t_.abs().sum()) for t_ in terms)
        assert abs(sum(float(t_.sum()) for t_ in terms) - (f[0] - f[1]) / 2e-5) <= 1e-5 * mag


def test_values_far_out():
    # gates far in both tails, hidden values large: bf16 holds them
    p, x, r = make(64, 64, 64, BF16)
    x = x * 200
    y = pmha.pmha_ffn_forward(p, x, residual=r)
    want, bound = block(p).forward(x, r)
    ref.assert_within("y", y, want, bound)
    assert y.isfinite().all()


def test_deterministic_stream_graph_and_shared_workspace():
    p, x, dy = make(4000, 128, 344, BF16)
    want, g0 = pmha.pmha_ffn_forward(p, x, residual=dy), pmha.pmha_ffn_backward(p, x, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = pmha.pmha_ffn_forward(p, x, residual=dy, stream=side)
    g1 = pmha.pmha_ffn_backward(p, x, dy, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and all(torch.equal(g0[n], g1[n]) for n in g0)
    # two graphs that share one workspace, replayed one after the other
    need = max(pmha.pmha_ffn_forward_workspace_size(p, 4000), pmha.pmha_ffn_backward_workspace_size(p, 4000))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for run in (lambda: pmha.pmha_ffn_forward(p, x, residual=dy, workspace=ws),
                lambda: pmha.pmha_ffn_backward(p, x, dy, workspace=ws)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run())
        graphs.append(graph)
    for k in (1, 0, 1, 0):
        ws.fill_(0xff)  # NaN everywhere
        graphs[k].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and all(torch.equal(g0[n], outs[1][n]) for n in g0)


def test_rows_zero_and_parts():
    p, x, dy = make(40, 64, 72, BF16)
    assert pmha.pmha_ffn_forward(p, x[:0]).shape == (0, 64)
    g = pmha.pmha_ffn_backward(p, x[:0], dy[:0])
    assert all(not g[n].any() for n in g) and g["dx"].shape == (0, 64)
    full = pmha.pmha_ffn_backward(p, x, dy)
    only = pmha.pmha_ffn_backward(p, x, dy, param_grads=False)
    assert set(only) == {"dx"} and torch.equal(only["dx"], full["dx"])
    rest = pmha.pmha_ffn_backward(p, x, dy, input_grads=False)
    assert "dx" not in rest and all(torch.equal(rest[n], full[n]) for n in rest)
    y = pmha.pmha_ffn_forward(p, x.view(5, 8, 64))
    assert torch.equal(y.view(40, 64), pmha.pmha_ffn_forward(p, x))


def test_rows_do_not_touch_one_another():
    # a row of NaN stays a row of NaN; rows behind the last one stay as they were
    p, x, _ = make(200, 64, 128, BF16)
    want = pmha.pmha_ffn_forward(p, x)
    x2 = x.clone()
    x2[77] = float("nan")
    buf = torch.full((300, 64), 3.0, dtype=BF16, device=DEV)
    pmha.pmha_ffn_forward(p, x2, out=buf[:200])
    keep = torch.arange(200, device=DEV) != 77
    assert torch.equal(buf[:200][keep], want[keep]) and buf[77].isnan().all() and bool((buf[200:] == 3.0).all())


def test_refusals():
    p, x, r = make(16, 64, 72, BF16)
    with pytest.raises(ValueError):
        pmha.pmha_ffn_forward(p, x.float())
    with pytest.raises(ValueError):
        pmha.pmha_ffn_forward(p, x[:, :32].contiguous())
    with pytest.raises(ValueError):
        pmha.pmha_ffn_forward(p, x, residual=r[:8])
    with pytest.raises(ValueError):
        pmha.pmha_ffn_forward(p, x, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        pmha.pmha_ffn_forward(pmha.FfnParams(p.wg, p.wu, p.wd, act="relu"), x)
    with pytest.raises(ValueError):
        pmha.pmha_ffn_forward(pmha.FfnParams(p.wg[:8], p.wu, p.wd), x)
    with pytest.raises(pmha.PmhaError):
        pmha.pmha_ffn_forward(p, x, out=x)
    q = pmha.FfnQuantizedParams.from_params(make(1, 24, 72, BF16)[0])
    x8, xs = pmha.quantize_rows(torch.ones(4, 24, device=DEV))
    with pytest.raises(pmha.PmhaError):
        pmha.pmha_ffn_forward_quantized(q, x8, xs)  # 24 is no multiple of 16

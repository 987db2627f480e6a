"""Microscaled 4-bit floating point: quantisation, the linear product and the gated block, against 64-bit forms."""
import copy
import pickle

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as enc
from tests import _mx_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def normal(seed, *shape, s=1.0, dtype=BF16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (s * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def tokens(seed, rows, width, dtype=BF16):
    """Rows and channels of very different sizes."""
    x = normal(seed, rows, width, dtype=torch.float32)
    x = x * torch.exp(normal(seed + 1, width, s=1.5, dtype=torch.float32)) * torch.exp(normal(seed + 2, rows, 1, s=2.0,
                                                                                              dtype=torch.float32))
    return x.to(dtype)


# ---------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 32), (2, 31), (3, 33), (5, 40), (127, 64), (128, 128), (129, 129), (7, 171),
                                        (300, 256), (33, 1000), (2, 4100), (257, 18)])
def test_codes_are_those_of_exact_arithmetic(rows, width, dtype):
    x = tokens(1, rows, width, dtype)
    q = pmha.pmha_mx_quantize(x)
    codes, scale = ref.packed(x)
    assert torch.equal(q.scale, scale) and torch.equal(q.codes, codes)
    assert torch.equal(q.values(), ref.values(x))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_borders_ties_and_extremes(dtype):
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    rows = []
    for e in (-130, -127, -126, -120, -3, 0, 5, 100, 124, 125):
        p = 2.0 ** e
        rows.append([6 * p] + [m * p for m in mids] + [-m * p for m in mids] + [m * p * (1 + 2.0 ** -7) for m in mids]
                    + [m * p * (1 - 2.0 ** -8) for m in mids] + [0.0, -0.0, p])
        rows.append([6 * p * (1 + 2.0 ** -7)] + [p] * 31)  # just above: the next power
        rows.append([3 * p] + [p * k / 7 for k in range(31)])
    rows.append([0.0] * 32)
    rows.append([torch.finfo(dtype).max] * 16 + [1.0] * 16)
    rows.append([2.0 ** -133] * 32)
    x = torch.tensor(rows, dtype=torch.float64, device=DEV).clamp(-3.3e38, 3.3e38).to(dtype)
    q = pmha.pmha_mx_quantize(x)
    codes, scale = ref.packed(x)
    assert torch.equal(q.scale, scale)
    assert torch.equal(q.values(), ref.values(x)) and torch.equal(q.codes, codes)


def test_values_of_a_matrix_by_hand():
    codes = torch.zeros(1, 16, dtype=torch.uint8, device=DEV)
    codes[0, :4] = torch.tensor([0x21, 0x43, 0x65, 0x8F], dtype=torch.uint8)
    scale = torch.zeros(1, 1, 512, dtype=torch.uint8, device=DEV)
    scale[0, 0, 0] = 128
    v = pmha.MxTensor(codes, scale, (1, 8)).values()
    assert v.tolist() == [[1.0, 2.0, 3.0, 4.0, 6.0, 8.0, -12.0, 0.0]]


def test_blocks_that_are_not_finite():
    x = normal(5, 130, 96)
    x[3, 40], x[129, 0], x[64, 95] = float("nan"), float("inf"), float("-inf")
    q = pmha.pmha_mx_quantize(x)
    bad = q.values().isnan().view(130, 3, 32)
    want = torch.zeros(130, 3, dtype=torch.bool, device=DEV)
    want[3, 1] = want[129, 0] = want[64, 2] = True
    assert torch.equal(bad.all(-1), want) and torch.equal(bad.any(-1), want)
    w = pmha.pmha_mx_quantize(normal(6, 24, 96))
    y = pmha.pmha_mx_linear(q, w)
    assert torch.equal(y.isnan().all(-1), want.any(-1)) and torch.equal(y.isnan().any(-1), want.any(-1))
    few = pmha.pmha_mx_linear(pmha.pmha_mx_quantize(x[:4].contiguous()), w)
    assert torch.equal(few.isnan().all(-1), want[:4].any(-1))


# ---------------------------------------------------------------- the product
def check_linear(x, w, bias, residual, got):
    """x, w: float64 values of the operands."""
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    for t in (bias, residual):
        if t is not None:
            y, mag = y + t.double(), mag + t.double().abs()
    # a float32 sum of K products by adders that may cut
    bound = (x.shape[1] + 4) * 2.0 ** -22 * mag + enc.half_ulp(BF16) * y.abs()
    enc.assert_within("y", got, y, 1.01 * bound + 1e-30)


@pytest.mark.parametrize("rows,width,outputs", [
    (1, 1, 1), (1, 32, 8), (1, 256, 1024), (1, 512, 2048), (1, 4096, 100), (2, 33, 17), (3, 171, 40), (4, 1000, 96), (8, 64, 24),
    (8, 2400, 64), (5, 4096, 72), (9, 32, 8), (9, 64, 16), (16, 128, 128), (100, 256, 256), (128, 200, 264), (129, 300, 7),
    (200, 100, 513), (256, 512, 512), (300, 257, 384), (511, 1025, 130), (1000, 2048, 1000), (77, 40, 1), (2000, 128, 24),
    (20_000, 256, 300), (20_000, 64, 301), (6, 1024, 4096), (7, 1024, 4096), (8000, 1100, 511), (9000, 1030, 1280),
    (9000, 1030, 1281)])
@pytest.mark.parametrize("extra", [False, True])
def test_linear(rows, width, outputs, extra):
    x, w = tokens(10, rows, width), normal(20, outputs, width, s=width ** -0.5)
    bias = normal(30, outputs) if extra else None
    residual = normal(31, rows, outputs, s=4.0) if extra else None
    qx, qw = pmha.pmha_mx_quantize(x), pmha.pmha_mx_quantize(w)
    got = pmha.pmha_mx_linear(qx, qw, bias=bias, residual=residual)
    pmha.pmha_device_status()
    check_linear(ref.values(x), ref.values(w), bias, residual, got)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("ex,ew", [(119, -119), (-119, 119), (60, 50), (-60, -50), (124, -20)])
def test_linear_of_far_scales(rows, ex, ew):
    """Scales near the ends of their range whose products are ordinary numbers."""
    width, outputs = 96, 40
    x = (normal(10, rows, width, dtype=torch.float32).clamp(-3, 3).double() * 2.0 ** ex).float()
    w = (normal(20, outputs, width, dtype=torch.float32).clamp(-3, 3).double() * 2.0 ** ew).float()
    got = pmha.pmha_mx_linear(pmha.pmha_mx_quantize(x), pmha.pmha_mx_quantize(w))
    check_linear(ref.values(x), ref.values(w), None, None, got)


def test_linear_places_every_row_column_and_scale():
    """Integers small enough for exact sums, scales of every block their own: the result is exact."""
    rows, width, outputs = 391, 800, 520
    g = torch.Generator(device=DEV).manual_seed(3)
    grid = torch.tensor(ref.GRID + tuple(-v for v in ref.GRID), device=DEV)

    def matrix(n):
        v = grid[torch.randint(0, 16, (n, width), generator=g, device=DEV)]
        v[:, ::32] = 6.0  # every block's largest: its scale is then the power below
        e = torch.randint(-2, 3, (n, width // 32), generator=g, device=DEV)
        return (v * torch.exp2(e.float()).repeat_interleave(32, 1)).to(BF16)

    x, w = matrix(rows), matrix(outputs)
    qx, qw = pmha.pmha_mx_quantize(x), pmha.pmha_mx_quantize(w)
    assert torch.equal(qx.values(), x.double()) and torch.equal(qw.values(), w.double())
    # sums of multiples of 2^-6 up to 800 * 576 = 2^18.8: 25 bits; the adders may cut one
    got = pmha.pmha_mx_linear(qx, qw)
    want = x.double() @ w.double().t()
    assert bool(((got.double() - want).abs() <= enc.half_ulp(BF16) * want.abs() * 1.01 + 2.0 ** -4).all())
    few = pmha.pmha_mx_linear(pmha.pmha_mx_quantize(x[:5].contiguous()), qw)
    assert torch.equal(few, want[:5].to(BF16))


# ---------------------------------------------------------------- the gated block
def plain_block(x, p, act, biases, residual):
    """y of the block in float64 with the hidden rows rounded to 4 bits, and what a rounding of them to the next value on the
    grid can do to it: values next to a border of the grid fall on either side by the last bits of float32."""
    wg, wu, wd = p
    bg, bu, bd = biases
    z = torch.zeros((), dtype=torch.float64, device=x.device)
    g = x @ wg.t() + (z if bg is None else bg.double())
    u = x @ wu.t() + (z if bu is None else bu.double())
    k = (x.shape[1] + 4) * 2.0 ** -22
    eg = k * (x.abs() @ wg.abs().t() + (z if bg is None else bg.double().abs()))
    eu = k * (x.abs() @ wu.abs().t() + (z if bu is None else bu.double().abs()))
    a, slope = enc.act(act, g)
    h = a * u
    eh = 1.01 * ((slope.abs() + 0.5 * eg) * eg * u.abs() + a.abs() * eu + 2.0 ** -19 * (a.abs() + 2.0 ** -20) * u.abs())
    q = ref.values(h)
    lo, hi = ref.values(h - eh), ref.values(h + eh)
    # where the whole block takes another scale, its values may move by a step of the larger one
    other = ref.quantize(h - eh)[1].maximum(ref.quantize(h + eh)[1])
    top = ref.blocks_of(h.abs() + eh).amax(-1)
    low = ref.blocks_of((h.abs() - eh).clamp_min(0)).amax(-1)
    flips = ref.quantize(top[..., None].expand(-1, -1, 32).flatten(1))[1] != ref.quantize(
        low[..., None].expand(-1, -1, 32).flatten(1))[1]
    step = torch.where(flips, 2 * ref.power(other.maximum(ref.quantize(h)[1]) + 1), z)
    move = torch.maximum((lo - q).abs(), (hi - q).abs()) + step.repeat_interleave(32, 1)[:, :h.shape[1]]
    y, mag = q @ wd.t(), q.abs() @ wd.abs().t()
    for t in (bd, residual):
        if t is not None:
            y, mag = y + t.double(), mag + t.double().abs()
    bound = move @ wd.abs().t() + (h.shape[1] + 4) * 2.0 ** -22 * mag + enc.half_ulp(BF16) * y.abs()
    return y, 1.01 * bound + 1e-30


@pytest.mark.parametrize("rows,E,F,act,extra", [
    (1, 32, 32, "silu", True), (1, 256, 1024, "silu", True), (3, 40, 100, "gelu", True), (8, 128, 512, "silu", False),
    (5, 33, 71, "gelu", False), (2, 1024, 4096, "silu", True), (16, 128, 512, "silu", True), (130, 64, 40, "gelu", True),
    (300, 171, 344, "silu", True), (257, 512, 2048, "gelu", True), (1000, 256, 688, "silu", False), (700, 7, 9, "gelu", True),
    (4096, 128, 512, "silu", True)])
def test_block(rows, E, F, act, extra):
    x = normal(10, rows, E)
    w = [normal(20, F, E, s=E ** -0.5), normal(21, F, E, s=E ** -0.5), normal(22, E, F, s=F ** -0.5)]
    biases = [normal(30, F, s=0.1), normal(31, F, s=0.1), normal(32, E, s=0.1)] if extra else [None] * 3
    residual = normal(33, rows, E) if extra else None
    params = pmha.FfnMxParams.from_params(pmha.FfnParams(*w, *biases, act=act))
    got = pmha.pmha_ffn_forward_mx(params, pmha.pmha_mx_quantize(x), residual=residual)
    pmha.pmha_device_status()
    y, bound = plain_block(ref.values(x), [ref.values(t) for t in w], act, biases, residual)
    enc.assert_within("y", got, y, bound)
    # typical values are far nearer than the bound, which allows every border its worst
    assert float((got.double() - y).norm() / y.norm()) < 1e-2


def test_block_of_zero_and_far_hidden_rows():
    """Gates far below zero leave hidden blocks of zeros; one token's block of large values next to them."""
    E, F, rows = 64, 256, 40
    x = normal(10, rows, E)
    x[7] = 0
    wg, wu, wd = normal(20, F, E, s=0.1), normal(21, F, E, s=0.1), normal(22, E, F, s=0.1)
    bg = torch.full((F,), -400.0, dtype=BF16, device=DEV)
    bg[32:64] = 100.0
    params = pmha.FfnMxParams.from_params(pmha.FfnParams(wg, wu, wd, bg, None, None))
    got = pmha.pmha_ffn_forward_mx(params, pmha.pmha_mx_quantize(x))
    y, bound = plain_block(ref.values(x), [ref.values(t) for t in (wg, wu, wd)], "silu", [bg, None, None], None)
    enc.assert_within("y", got, y, bound)
    assert bool((got[7] == 0).all())


# ---------------------------------------------------------------- as used
def test_batches_capture_streams_and_workspace():
    E, F = 128, 512
    block = pmha.FfnParams(normal(20, F, E, s=E ** -0.5), normal(21, F, E, s=E ** -0.5), normal(22, E, F, s=F ** -0.5))
    params = pmha.FfnMxParams.from_params(block)
    x = normal(10, 3, 100, E)

    def step():
        q = pmha.pmha_mx_quantize(x)
        y = pmha.pmha_ffn_forward_mx(params, q, residual=x)
        return [q.codes, q.scale, y, pmha.pmha_mx_linear(pmha.pmha_mx_quantize(y), params.wg)]

    want = step()
    assert want[2].shape == x.shape and want[3].shape == (3, 100, F)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = pmha.pmha_mx_quantize(x, stream=side)
    ws = torch.empty(pmha.pmha_ffn_forward_mx_workspace_size(params, 300), dtype=torch.uint8, device=DEV)
    y = pmha.pmha_ffn_forward_mx(params, q, residual=x, workspace=ws, out=torch.empty_like(x), stream=side)
    side.synchronize()
    assert torch.equal(y, want[2])
    # a workspace of the largest batch serves every smaller one
    sizes = [pmha.pmha_ffn_forward_mx_workspace_size(params, r) for r in range(0, 400)]
    assert sizes == sorted(sizes)
    small = pmha.pmha_ffn_forward_mx(params, pmha.pmha_mx_quantize(x[0, :1].contiguous()), workspace=ws)
    assert small.shape == (1, E)
    with pytest.raises(ValueError, match="workspace"):
        pmha.pmha_ffn_forward_mx(params, q, workspace=ws[:64])
    none = pmha.pmha_mx_quantize(x[:0])
    assert pmha.pmha_ffn_forward_mx(params, none).shape == (0, 100, E)


def test_calls_at_once():
    """Products, blocks and joins on three streams at the same time, some of them captured: the results of each alone."""
    E, F = 256, 1024
    block = pmha.FfnParams(normal(20, F, E, s=E ** -0.5), normal(21, F, E, s=E ** -0.5), normal(22, E, F, s=F ** -0.5))
    params = pmha.FfnMxParams.from_params(block)
    w = pmha.pmha_mx_quantize(normal(23, 1280, 1030, s=0.03))
    join = pmha.JoinParams(pre=normal(1, E), post=normal(2, E), gate=normal(3, 8, E))
    x, y = normal(10, 4000, E), normal(11, 6000, 1030)

    def step():
        s, n, kept, _ = pmha.pmha_join_checkpointed(join, x, x, keep_residual=False)
        g = pmha.pmha_join_backward(join, kept, s, n, x)
        f = pmha.pmha_ffn_forward_mx(params, pmha.pmha_mx_quantize(n), residual=s)
        return [f, g["dbranch"], g["dgate"], g["dpost"], pmha.pmha_mx_linear(pmha.pmha_mx_quantize(y), w)]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        graph.replay()
        for st in streams:
            with torch.cuda.stream(st):
                got.append(step())
    torch.cuda.synchronize()
    pmha.pmha_device_status()
    for out in (captured, *got):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_weights_written_by_the_launch_before():
    """Quantisation of the weights right in front of the products that read them, many times over: no product starts early."""
    E, F = 256, 1024
    x = pmha.pmha_mx_quantize(normal(10, 1, E))
    sets = [[normal(100 * i + j, *s, s=0.05) for j, s in enumerate(((F, E), (F, E), (E, F)))] for i in range(2)]
    want = []
    for w in sets:
        p = pmha.FfnMxParams.from_params(pmha.FfnParams(*w))
        torch.cuda.synchronize()
        want.append((pmha.pmha_ffn_forward_mx(p, x), pmha.pmha_mx_linear(x, p.wg)))
    torch.cuda.synchronize()
    for i in range(40):
        p = pmha.FfnMxParams.from_params(pmha.FfnParams(*sets[i % 2]))
        y = pmha.pmha_ffn_forward_mx(p, x)
        z = pmha.pmha_mx_linear(x, pmha.pmha_mx_quantize(sets[i % 2][0]))
        assert torch.equal(y, want[i % 2][0]) and torch.equal(z, want[i % 2][1]), i


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_copies_stand_for_the_same_values(how):
    """A copy has arrays of its own (copy: the same ones), which the calls read after the original is gone."""
    make = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda t: pickle.loads(pickle.dumps(t))}[how]
    x, w = normal(1, 40, 96), normal(2, 24, 96)
    q, k = pmha.pmha_mx_quantize(w), pmha.pmha_checkpoint(x)
    want = pmha.pmha_mx_linear(pmha.pmha_mx_quantize(x), q), pmha.pmha_checkpoint_restore(k)
    block = make(pmha.FfnMxParams(q, q, pmha.pmha_mx_quantize(normal(3, 96, 24))))
    assert torch.equal(block.wg.values(), q.values())
    q2, k2 = make(q), make(k)
    if how != "copy":
        q.codes.fill_(0x11), k.codes.zero_()
    del q, k
    assert q2.shape == w.shape and k2.dtype == BF16
    got = pmha.pmha_mx_linear(pmha.pmha_mx_quantize(x), q2), pmha.pmha_checkpoint_restore(k2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if how != "copy":
        pmha.pmha_device_status()
        assert torch.equal(block.wg.values(), q2.values())


def test_refusals():
    x = normal(1, 4, 64)
    q, w = pmha.pmha_mx_quantize(x), pmha.pmha_mx_quantize(normal(2, 32, 64))
    with pytest.raises(ValueError, match="weight"):
        pmha.pmha_mx_linear(q, pmha.pmha_mx_quantize(normal(2, 32, 96)))
    with pytest.raises(TypeError, match="MxTensor"):
        pmha.pmha_mx_linear(x, w)
    with pytest.raises(ValueError, match="codes"):
        pmha.MxTensor(q.codes, q.scale, (5, 64))
    with pytest.raises(ValueError, match="scale"):
        pmha.MxTensor(q.codes, q.scale[:, :, :256], (4, 64))
    with pytest.raises(AttributeError):
        q.codes = w.codes
    with pytest.raises(ValueError, match="bias"):
        pmha.pmha_mx_linear(q, w, bias=normal(3, 32, dtype=torch.float32))
    with pytest.raises(ValueError, match="beside"):
        pmha.pmha_ffn_forward_mx(pmha.FfnMxParams(w, w, w), q)
    with pytest.raises(ValueError):
        pmha.pmha_mx_quantize(x.half())
    with pytest.raises(pmha.PmhaError, match="overlap"):
        both = torch.empty(4, 64, dtype=BF16, device=DEV)
        pmha.pmha_mx_linear(q, pmha.pmha_mx_quantize(normal(2, 64, 64)), residual=both, out=both)

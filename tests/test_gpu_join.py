"""The join with the residual stream, forward and backward, and tensors kept in 8 bits, against 64-bit forms."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests import _encoder_ref as enc
from tests import _stream_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def normal(seed, *shape, s=1.0, off=0.0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (off + s * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def params(width, dtype, post=True, gates=1, pre=True, alpha=1.0, eps=EPS):
    gate = None if gates == 0 else normal(3, width, s=0.7, dtype=dtype) if gates == 1 else \
        normal(3, gates, width, s=0.7, dtype=dtype)
    return pmha.JoinParams(pre=normal(1, width, s=0.1, off=1.0, dtype=dtype) if pre else None,
                           post=normal(2, width, s=0.1, off=1.0, dtype=dtype) if post else None, gate=gate,
                           residual_scale=alpha, eps=eps)


def check_forward(p, branch, residual, s, n, b64=None, r64=None):
    """s against the formula, n against the norm of s as it came."""
    dtype = s.dtype
    b64 = (None if branch is None else branch.double()) if b64 is None else b64
    want, bound = ref.join_sum(b64, residual.double() if r64 is None else r64, p.post, p.gate, p.residual_scale, p.eps)
    enc.assert_within("sum", s, *ref.with_rounding(want, bound, dtype))
    if p.pre is None:
        assert n is None
        return
    y, _ = enc.norm(s, p.pre, p.eps)
    enc.assert_within("out", n, *ref.with_rounding(y, ref.tol(s.shape[-1]) * y.abs(), dtype))


def check_backward(p, got, branch, s, dout, dsum):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    want = ref.backward(d(branch), d(s), d(dout), d(dsum), p.post, p.gate, p.pre, p.residual_scale, p.eps)
    dtype = (dsum if dout is None else dout).dtype
    for name in ("dbranch", "dresidual", "dpre", "dpost", "dgate"):
        assert (got[name] is None) == (name not in want), name
        if name in want:
            t = dtype if name in ("dbranch", "dresidual") else torch.float32
            assert got[name].dtype == t
            enc.assert_within(name, got[name], *ref.with_rounding(*want[name], t))


WIDTHS = [1, 2, 7, 16, 31, 32, 33, 64, 100, 120, 128, 171, 256, 257, 258, 264, 512, 520, 1000, 1024, 1025, 2048, 2049, 2056, 4100]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dt):
    dtype = TYPES[dt]
    rows = 37
    branch, residual = normal(10, rows, width, s=0.5, dtype=dtype), normal(11, rows, width, s=2.0, dtype=dtype)
    p = params(width, dtype, alpha=1.25)
    s, n = pmha.pmha_join(p, branch, residual)
    check_forward(p, branch, residual, s, n)
    dout, dsum = normal(12, rows, width, dtype=dtype), normal(13, rows, width, dtype=dtype)
    check_backward(p, pmha.pmha_join_backward(p, branch, s, dout, dsum), branch, s, dout, dsum)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("width", [24, 128, 344, 1536, 2500])
@pytest.mark.parametrize("rows,gates,post,pre,with_dsum,alpha", [
    (1, 0, False, True, True, 1.0), (1, 1, True, True, False, 1.0), (6, 3, True, True, True, 0.5), (6, 6, True, True, True, 1.0),
    (35, 7, False, True, True, 1.0), (64, 2, False, False, True, -1.5), (64, 0, True, False, True, 1.0),
    (50, 0, False, False, True, 2.0), (999, 1, False, True, False, 1.0), (1000, 4, True, True, True, 1.0)])
def test_forms(width, dt, rows, gates, post, pre, with_dsum, alpha):
    dtype = TYPES[dt]
    branch, residual = normal(10, rows, width, s=0.5, dtype=dtype), normal(11, rows, width, s=2.0, dtype=dtype)
    p = params(width, dtype, post, gates, pre, alpha)
    s, n = pmha.pmha_join(p, branch, residual)
    check_forward(p, branch, residual, s, n)
    dout = normal(12, rows, width, dtype=dtype) if pre else None
    dsum = normal(13, rows, width, dtype=dtype) if with_dsum else None
    got = pmha.pmha_join_backward(p, branch, s, dout, dsum)
    check_backward(p, got, branch, s, dout, dsum)
    # single parts of it give the same bits
    only = pmha.pmha_join_backward(p, branch, s, dout, dsum, param_grads=False)
    assert torch.equal(only["dbranch"], got["dbranch"]) and torch.equal(only["dresidual"], got["dresidual"])
    only = pmha.pmha_join_backward(p, branch, s, dout, dsum, input_grads=False)
    assert all(only[k] is None if got[k] is None else torch.equal(only[k], got[k]) for k in ("dpre", "dpost", "dgate"))


def test_many_rows_of_one_gate():
    """More rows than a block takes steps: the sums over rows come from many partial rows."""
    rows, width, dtype = 300_000, 64, torch.bfloat16
    branch, residual = normal(10, rows, width, s=0.5, dtype=dtype), normal(11, rows, width, s=2.0, dtype=dtype)
    p = params(width, dtype)
    s, n = pmha.pmha_join(p, branch, residual)
    dout, dsum = normal(12, rows, width, dtype=dtype), normal(13, rows, width, dtype=dtype)
    got = pmha.pmha_join_backward(p, branch, s, dout, dsum)
    check_forward(p, branch, residual, s, n)
    check_backward(p, got, branch, s, dout, dsum)
    again = pmha.pmha_join_backward(p, branch, s, dout, dsum)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("width", [40, 129, 700, 2048, 2304])
def test_large_and_zero_rows(width, dt):
    """Rows whose squares leave float32, rows of zeros, a row with a NaN and one with an infinity beside ordinary ones."""
    dtype = TYPES[dt]
    big = torch.finfo(dtype).max / 4
    branch, residual = normal(10, 9, width, dtype=dtype), normal(11, 9, width, dtype=dtype)
    branch[2] = torch.where(branch[2] > 0, big, -big).to(dtype)
    branch[4] = 0
    residual[5] = torch.where(residual[5] > 0, big, -big).to(dtype)
    branch[5] = 0
    branch[6] = 0
    residual[6] = 0
    branch[7, width // 2] = float("nan")
    residual[8, width - 1] = float("inf")
    p = params(width, dtype)
    s, n = pmha.pmha_join(p, branch, residual)
    fine = [0, 1, 2, 3, 4, 5, 6]
    check_forward(p, branch[fine], residual[fine], s[fine], n[fine])
    assert bool(n[7].isnan().all()) and bool(s[8, -1].isinf())
    dout, dsum = normal(12, 9, width, dtype=dtype), normal(13, 9, width, dtype=dtype)
    b, h, dy, ds = (t[fine].contiguous() for t in (branch, s, dout, dsum))
    check_backward(p, pmha.pmha_join_backward(p, b, h, dy, ds), b, h, dy, ds)


# ---------------------------------------------------------------- 8 bits
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 2), (5, 31), (4, 32), (7, 33), (9, 40), (33, 128), (2, 171), (11, 1000),
                                        (3, 2049), (1, 70_000), (5000, 24), (4001, 171), (1001, 7), (300, 33), (600, 6), (100, 3),
                                        (64, 48)])
def test_checkpoint_codes_are_those_of_exact_arithmetic(rows, width, dt):
    x = normal(20, rows, width, s=3.0, dtype=TYPES[dt])
    x = x * torch.exp2(torch.randint(-8, 9, (rows, 1), device=DEV)).to(x.dtype)
    k = pmha.pmha_checkpoint(x)
    codes, scale = ref.kept(x)
    assert torch.equal(k.scale.double(), scale) and torch.equal(k.codes.double(), codes)
    back = pmha.pmha_checkpoint_restore(k)
    assert back.dtype == x.dtype and torch.equal(back, (codes * scale.repeat_interleave(32, -1)[:, :width]).to(x.dtype))
    # within half a scale, and half a step of the type
    off = (back.double() - x.double()).abs()
    assert bool((off <= 0.5 * scale.repeat_interleave(32, -1)[:, :width] + enc.half_ulp(x.dtype) * x.double().abs()
                 + 2.0 ** -100).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_checkpoint_of_ties_borders_and_extremes(dt):
    """Values halfway between codes, the group's largest at every mantissa, zeros, the type's largest and least, NaN."""
    dtype = TYPES[dt]
    rows = []
    for m in range(128):
        scale = 2.0 ** ((m % 9) - 4) * (1 + m / 128)
        most = 127 * scale  # exact in float32; in bfloat16 rounded, the ties then lie elsewhere
        rows.append([most] + [scale * (k + 0.5) for k in range(-15, 16)])
    big = torch.finfo(dtype).max
    rows += [[0.0] * 32, [big] + [big / 3] * 31, [1e-38] * 32, [2.0 ** -90] + [0.0] * 31, [-0.0] * 32,
             [2.0 ** -133] * 32, [1.0] + [0.5] * 31, [128.0] + [64.0] * 31]
    x = torch.tensor(rows, dtype=torch.float64, device=DEV).to(dtype)
    codes, scale = ref.kept(x)
    k = pmha.pmha_checkpoint(x)
    assert torch.equal(k.scale.double(), scale) and torch.equal(k.codes.double(), codes)
    y = torch.ones(3, 64, dtype=dtype, device=DEV)
    y[0, 3], y[1, 40], y[2, 63] = float("nan"), float("inf"), float("-inf")
    back = pmha.pmha_checkpoint_restore(pmha.pmha_checkpoint(y))
    bad = back.isnan().view(3, 2, 32)
    assert bool((bad.all(-1) == torch.tensor([[True, False], [False, True], [False, True]], device=DEV)).all())
    assert bool((back[~back.isnan()] - 1).abs().max() <= 2.0 ** -7)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("width", [24, 33, 66, 128, 512, 1000, 1030, 2048, 2052, 3001])
def test_kept_forms(width, dt):
    """What the join keeps is what pmha_checkpoint keeps; join and gradients from it are those of the restored values."""
    dtype = TYPES[dt]
    rows = 30
    branch, residual = normal(10, rows, width, s=0.5, dtype=dtype), normal(11, rows, width, s=2.0, dtype=dtype)
    p = params(width, dtype, gates=5, alpha=0.75)
    s, n, kb, kr = pmha.pmha_join_checkpointed(p, branch, residual)
    s0, n0 = pmha.pmha_join(p, branch, residual)
    assert torch.equal(s, s0) and torch.equal(n, n0)
    for k, x in ((kb, branch), (kr, residual)):
        alone = pmha.pmha_checkpoint(x)
        assert torch.equal(k.codes, alone.codes) and torch.equal(k.scale, alone.scale)
    b64, r64 = ref.restored(branch), ref.restored(residual)
    for b, r, bd, rd in ((kb, kr, b64, r64), (branch, kr, branch.double(), r64), (kb, residual, b64, residual.double())):
        s2, n2 = pmha.pmha_join(p, b, r)
        check_forward(p, branch, residual, s2, n2, bd, rd)
    dout, dsum = normal(12, rows, width, dtype=dtype), normal(13, rows, width, dtype=dtype)
    got = pmha.pmha_join_backward(p, kb, s, dout, dsum)
    check_backward(p, got, b64, s, dout, dsum)
    # one of the two kept, and a norm alone from a kept tensor
    s3, n3, kb3, none = pmha.pmha_join_checkpointed(p, branch, kr, keep_residual=False)
    assert none is None and torch.equal(kb3.codes, kb.codes) and torch.equal(kb3.scale, kb.scale)
    q = pmha.JoinParams(pre=p.pre, eps=EPS)
    s4, n4 = pmha.pmha_join(q, None, kr)
    assert torch.equal(s4, pmha.pmha_checkpoint_restore(kr))
    check_forward(q, None, residual, s4, n4, None, r64)


# ---------------------------------------------------------------- gradients against differences, runs as used
def test_gradients_are_those_of_differences():
    rows, width = 6, 48
    p = params(width, torch.float32, gates=3, alpha=0.8)
    branch, residual = normal(10, rows, width), normal(11, rows, width)
    dout, dsum = normal(12, rows, width), normal(13, rows, width)
    s, _ = pmha.pmha_join(p, branch, residual)
    got = pmha.pmha_join_backward(p, branch, s, dout, dsum)

    def loss(b, r, pre, post, gate):
        h, _ = ref.join_sum(b, r, post, gate, p.residual_scale, EPS)
        return float((enc.norm(h, pre)[0] * dout.double()).sum() + (h * dsum.double()).sum())

    at = [t.double() for t in (branch, residual, p.pre, p.post, p.gate)]
    for i, name in enumerate(("dbranch", "dresidual", "dpre", "dpost", "dgate")):
        way = normal(30 + i, *at[i].shape).double()
        h = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * way, at[i] - h * way
        diff = (loss(*up) - loss(*down)) / (2 * h)
        along = float((got[name].double() * way).sum())
        # float32 values in the analytic side, 1e-10 of the losses over 2e-5 in the other
        assert abs(along - diff) <= 1e-4 * (abs(diff) + float((got[name].double() * way).abs().sum()) * 1e-2 + 1e-3), name


def test_stream_capture_workspace_and_strides():
    rows, width, dtype = 4000, 128, torch.bfloat16
    branch, residual = normal(10, rows, width, s=0.5, dtype=dtype), normal(11, rows, width, s=2.0, dtype=dtype)
    dout, dsum = normal(12, rows, width, dtype=dtype), normal(13, rows, width, dtype=dtype)
    p = params(width, dtype, gates=8)

    def step():
        s, n, kb, kr = pmha.pmha_join_checkpointed(p, branch, residual)
        return [s, n, kb.codes, kb.scale, kr.codes, kr.scale, *pmha.pmha_join_backward(p, kb, s, dout, dsum).values()]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s, n = pmha.pmha_join(p, branch, residual, stream=side)
    ws = torch.empty(pmha.pmha_join_backward_workspace_size(p, dout), dtype=torch.uint8, device=DEV)
    got = pmha.pmha_join_backward(p, branch, s, dout, dsum, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(s, want[0]) and got["dgate"].shape == (8, width)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    with pytest.raises(ValueError, match="contiguous"):
        pmha.pmha_join(p, branch, residual.t().contiguous().t())
    with pytest.raises(ValueError):
        pmha.pmha_join(p, branch[:, :64], residual)
    with pytest.raises(ValueError, match="workspace"):
        pmha.pmha_join_backward(p, branch, s, dout, dsum, workspace=ws[:256])


def test_batches_and_no_rows():
    p = params(64, torch.float32, gates=0)
    branch, residual = normal(10, 3, 5, 64), normal(11, 3, 5, 64)
    s, n = pmha.pmha_join(p, branch, residual)
    flat = pmha.pmha_join(p, branch.view(15, 64), residual.view(15, 64))
    assert s.shape == (3, 5, 64) and torch.equal(s.view(15, 64), flat[0]) and torch.equal(n.view(15, 64), flat[1])
    k = pmha.pmha_checkpoint(branch)
    assert k.shape == (3, 5, 64) and k.scale.shape == (3, 5, 2) and k.nbytes == 15 * (64 + 4)
    none = torch.empty(0, 64, device=DEV)
    s, n, kb, kr = pmha.pmha_join_checkpointed(p, none, none)
    got = pmha.pmha_join_backward(p, kb, s, none, none)
    assert s.shape == (0, 64) and bool((got["dpre"] == 0).all()) and bool((got["dpost"] == 0).all())
    assert pmha.pmha_checkpoint_restore(pmha.pmha_checkpoint(none)).shape == (0, 64)

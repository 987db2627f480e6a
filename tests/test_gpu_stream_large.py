"""The residual stream's operators and 4-bit products on tensors past 2^31 values: the last rows are those of a call on them
alone, bit for bit."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"
BF16 = torch.bfloat16


def big(seed, rows, width, s=1.0):
    """Few distinct rows, over and over, and its own last ones."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    base = (s * torch.randn(4099, width, generator=g, device=DEV)).to(BF16)
    x = torch.empty(rows, width, dtype=BF16, device=DEV)
    for at in range(0, rows, 4099):
        n = min(4099, rows - at)
        x[at:at + n] = base[:n]
    x[-1000:] = (s * torch.randn(1000, width, generator=g, device=DEV)).to(BF16)
    return x


@pytest.mark.parametrize("rows,width", [(18_000_000, 120), (1_050_000, 2056)])
def test_join_and_checkpoints(rows, width):
    assert rows * width > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(9)
    pre, post, gate = ((1 + 0.1 * torch.randn(width, generator=g, device=DEV)).to(BF16) for _ in range(3))
    p = pmha.JoinParams(pre=pre, post=post, gate=gate)
    branch, residual = big(1, rows, width), big(2, rows, width, 2.0)
    tail = [t[-1000:].contiguous() for t in (branch, residual)]
    s, n, kept, _ = pmha.pmha_join_checkpointed(p, branch, residual, keep_residual=False)
    s1, n1, kept1, _ = pmha.pmha_join_checkpointed(p, *tail, keep_residual=False)
    assert torch.equal(s[-1000:], s1) and torch.equal(n[-1000:], n1)
    assert torch.equal(kept.codes[-1000:], kept1.codes) and torch.equal(kept.scale[-1000:], kept1.scale)
    got = pmha.pmha_join_backward(p, kept, s, n, residual)
    one = pmha.pmha_join_backward(p, kept1, s1, n1, tail[1])
    for k in ("dbranch", "dresidual"):
        assert torch.equal(got[k][-1000:], one[k]), k
    del got, branch, n
    back = pmha.pmha_checkpoint_restore(kept)
    assert torch.equal(back[-1000:], pmha.pmha_checkpoint_restore(kept1))


def test_gates_of_every_row():
    """More than 2^31 gate values: dpost sums over all of them."""
    rows, width = 16_800_000, 128
    assert rows * width > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(9)
    post = (1 + 0.1 * torch.randn(width, generator=g, device=DEV)).to(BF16)
    gate, branch, ds = big(1, rows, width), big(2, rows, width), big(3, rows, width)
    gate[-1000:] *= 8  # their part is no small one
    got = pmha.pmha_join_backward(pmha.JoinParams(post=post, gate=gate), branch, None, None, ds, input_grads=False)
    want, mag = (torch.zeros(width, dtype=torch.float64, device=DEV) for _ in range(2))
    for at in range(0, rows, 400_000):
        b = branch[at:at + 400_000].double()
        t = gate[at:at + 400_000].double() * ds[at:at + 400_000].double() * b * (b.square().mean(-1, True) + 1e-6).rsqrt()
        want += t.sum(0)
        mag += t.abs().sum(0)
    # a root within 2^-21 and two products, each rounded, a row; sums as pairs
    assert bool(((got["dpost"].double() - want).abs() <= 2.0 ** -20 * mag + 2.0 ** -23 * want.abs()).all())
    b = branch[-5:].double()
    r = ds[-5:].double() * b * (b.square().mean(-1, True) + 1e-6).rsqrt() * post.double()
    assert bool(((got["dgate"][-5:].double() - r).abs() <= 2.0 ** -20 * r.abs()).all())


def test_quantize_linear_and_block():
    rows, width, outputs = 34_000_000, 64, 72
    assert rows * width > 2 ** 31 and rows * outputs > 2 ** 31
    x = big(3, rows, width)
    g = torch.Generator(device=DEV).manual_seed(9)
    w = pmha.pmha_mx_quantize((torch.randn(outputs, width, generator=g, device=DEV) / 8).to(BF16))
    wd = pmha.pmha_mx_quantize((torch.randn(width, outputs, generator=g, device=DEV) / 8).to(BF16))
    q = pmha.pmha_mx_quantize(x)
    tail = x[-1000:].contiguous()
    q1 = pmha.pmha_mx_quantize(tail)
    assert torch.equal(q.codes[-1000:], q1.codes)
    y = pmha.pmha_mx_linear(q, w)
    assert torch.equal(y[-1000:], pmha.pmha_mx_linear(q1, w))
    del y
    params = pmha.FfnMxParams(w, w, wd)
    y = pmha.pmha_ffn_forward_mx(params, q, residual=x)
    assert torch.equal(y[-1000:], pmha.pmha_ffn_forward_mx(params, q1, residual=tail))
    pmha.pmha_device_status()

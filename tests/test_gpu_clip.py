"""Clipping by the global gradient norm against the formula in 64 bits."""
import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests._encoder_ref import half_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def reference(grads, max_norm):
    norm = torch.stack([(g.double() ** 2).sum() for g in grads]).sum().sqrt()
    return float(norm), float((max_norm / (norm + 1e-6)).clamp_max(1.0))


def check(grads, max_norm, out=None):
    before = [g.clone() for g in grads]
    want, coef = reference(before, max_norm)
    norm = pmha.pmha_clip_grad_norm(grads, max_norm, out=out)
    torch.cuda.synchronize()
    # squares and chains of a few thousand adds in float32 a thread, all positive; the rest in double
    assert abs(float(norm) - want) <= 2.0 ** -18 * want + 1e-45
    for g, o, b in zip(grads, grads if out is None else out, before):
        if out is not None:
            assert torch.equal(g, b)
        # the factor is off by as much as the norm, then rounded; product and result round once each
        tol = (2.0 ** -18 + 2.0 ** -23 + half_ulp(o.dtype)) * (b.double() * coef).abs() + 1e-45
        assert bool(((o.double() - b.double() * coef).abs() <= tol).all())
    return norm


def make(sizes, dtype=torch.float32, scale=0.02, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(n, generator=g, device=DEV) * scale).to(dtype) for n in sizes]


SIZES = [1, 2, 3, 5, 127, 128, 16383, 16384, 16385, 100001]


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
@pytest.mark.parametrize("separate", [False, True])
def test_mixed_types_and_sizes(max_norm, separate):
    grads = make(SIZES) + make(SIZES, torch.bfloat16, seed=1)
    out = [torch.full_like(g, 7.0) for g in grads] if separate else None
    check(grads, max_norm, out)


def test_many_tensors_take_several_launches():
    grads = make([17 + i % 5 for i in range(1300)], seed=2)
    before = pmha.pmha_launch_count()
    check(grads, 0.1)
    assert pmha.pmha_launch_count() - before == 6


def test_views_off_the_16_byte_boundary_leave_their_neighbours():
    flat = make([5000])[0]
    keep = flat.clone()
    grads = [flat[1:1000], flat[1003:4001]]
    out = torch.zeros(5000, device=DEV)
    check(grads, 0.1, [out[2:1001], out[1500:4498]])
    assert not out[:2].any() and not out[1001:1500].any() and not out[4498:].any()
    check(grads, 0.1)
    assert torch.equal(flat[0], keep[0]) and torch.equal(flat[1000:1003], keep[1000:1003])
    assert torch.equal(flat[4001:], keep[4001:])


@pytest.mark.parametrize("scale", [1e-30, 1e-14, 1e14, 1e30])
def test_squares_outside_float32(scale):
    grads = make([1000, 20000], scale=scale)
    grads[0][:10] = 0.0
    check(grads, 1.0)


def test_small_beside_large():
    grads = [torch.full((4096,), 3e-20, device=DEV), torch.tensor([1e-18], device=DEV)]
    check(grads, 1.0)
    check([torch.full((64,), 2.0 ** 41, device=DEV), torch.full((64,), 1.0, device=DEV)], 1.0)


def test_not_finite():
    grads = make([100, 100])
    grads[1][7] = float("inf")
    norm = pmha.pmha_clip_grad_norm(grads, 1.0)
    assert norm.isinf() and grads[1][7].isnan() and not grads[0].any() and int(grads[1].isnan().sum()) == 1
    grads = make([100, 100])
    grads[0][3] = float("nan")
    norm = pmha.pmha_clip_grad_norm(grads, 1.0)
    assert norm.isnan() and all(g.isnan().all() for g in grads)


def test_zero_norm_empty_tensors_and_none():
    z = [torch.zeros(10, device=DEV), torch.zeros(0, device=DEV), None]
    assert float(pmha.pmha_clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    assert float(pmha.pmha_clip_grad_norm([torch.zeros(0, device=DEV)], 1.0)) == 0.0


def test_deterministic_stream_and_graph():
    grads = make(SIZES, seed=3)
    out = [torch.empty_like(g) for g in grads]
    a = pmha.pmha_clip_grad_norm(grads, 0.3, out=out)
    first = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = pmha.pmha_clip_grad_norm(grads, 0.3, out=out, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and all(torch.equal(o, f) for o, f in zip(out, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = pmha.pmha_clip_grad_norm(grads, 0.3, out=out)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c) and all(torch.equal(o, f) for o, f in zip(out, first))


def test_refusals():
    a, b = make([64, 64])
    for bad in ([a, a], [a, a[3:9]], [a.half()], [a.view(8, 8).t()], [a.cpu()], []):
        with pytest.raises((ValueError, TypeError, pmha.PmhaError)):
            pmha.pmha_clip_grad_norm(bad, 1.0)
    for m in (-1.0, float("nan"), float("inf")):
        with pytest.raises(pmha.PmhaError):
            pmha.pmha_clip_grad_norm([a], m)
    with pytest.raises(ValueError):
        pmha.pmha_clip_grad_norm([a, b], 1.0, out=[a])
    with pytest.raises(pmha.PmhaError):
        pmha.pmha_clip_grad_norm([a, b], 1.0, out=[b, a])  # an output over another gradient
    with pytest.raises(ValueError):
        pmha.pmha_clip_grad_norm([a], 1.0, out=[torch.empty(63, device=DEV)])

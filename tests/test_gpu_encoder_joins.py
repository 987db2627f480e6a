"""The encoder layer with norms after its blocks, gates and a scaled residual stream; its training step from 8-bit
checkpoints; and serving it with blocks of 8 and 4 bits."""
import math

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests.test_gpu_encoder import BARS, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def joined(layer, seed, post=True, gates=1, scale=1.0):
    """The layer of the same tensors with joins."""
    dtype, E = layer.attention.dtype, layer.attention.embed_dim
    g = torch.Generator(device=DEV).manual_seed(seed)

    def t(*shape, s=0.1, off=1.0):
        return (off + s * torch.randn(*shape, generator=g, device=DEV)).to(dtype)

    kw = {}
    for i in (1, 2):
        kw[f"post{i}"] = t(E) if post else None
        kw[f"gate{i}"] = t(E, s=0.3) if gates == 1 else t(gates, E, s=0.3) if gates else None
    return pmha.PackedEncoderLayer(layer.graph, layer.attention, layer.norm1, layer.norm2, layer.block, layer.eps, **kw,
                                   residual_scale=scale)


def plain(layer, x, spec):
    """The layer in float64 torch operations; parameters as leaves."""
    src, tgt, prm, H = spec
    leaf = {}

    def p(name, v):
        leaf[name] = None if v is None else v.double().detach().requires_grad_()
        return leaf[name]

    x = p("x", x)
    B, n, E = x.shape
    d = E // H
    a, b, j1, j2 = layer.attention, layer.block, layer.join1, layer.join2
    w = {k: p(k, getattr(a, k)) for k in ("wq", "wk", "wv", "wo", "bq", "bk", "bv", "bo")}

    def norm(v, g):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + layer.eps) * g

    def join(join, i, branch, residual):
        post, gate = p(f"post{i}", join.post), p(f"gate{i}", join.gate)
        z = branch if post is None else norm(branch, post)
        z = z if gate is None else z * (gate if gate.dim() == 1 else gate[:, None])
        return join.residual_scale * residual + z

    n1 = norm(x, p("norm1", layer.norm1))
    q, k, v = (n1 @ w["w" + c].t() + w["b" + c] for c in "qkv")
    s, t = (torch.from_numpy(i).to(x.device) for i in (src, tgt))
    score = (q[:, t].view(B, -1, H, d) * k[:, s].view(B, -1, H, d)).sum(-1) / math.sqrt(d)
    e = torch.exp(score - score.amax())
    z = torch.zeros(B, n, H, dtype=e.dtype, device=e.device).index_add(1, t, e)
    wt = e / z[:, t]
    mix = torch.zeros(B, n, H, d, dtype=e.dtype, device=e.device).index_add(1, t, wt[..., None] * v[:, s].view(B, -1, H, d))
    s1 = join(j1, 1, mix.reshape(B, n, E) @ w["wo"].t() + w["bo"], x)
    n2 = norm(s1, p("norm2", layer.norm2))
    g = n2 @ p("wg", b.wg).t() + p("bg", b.bg)
    u = n2 @ p("wu", b.wu).t() + p("bu", b.bu)
    y = join(j2, 2, (g * torch.sigmoid(g) * u) @ p("wd", b.wd).t() + p("bd", b.bd), s1)
    return y, leaf


def close(name, got, exp, bar):
    rms = float(exp.pow(2).mean().sqrt())
    off = float((got.double() - exp).abs().max())
    assert off <= bar * rms, f"{name}: {off:.3g} > {bar} x {rms:.3g}"


SHAPES = [(64, 256, 2, 32, 4, 88, "f32"), (300, 3000, 2, 128, 8, 344, "bf16")]


@pytest.mark.parametrize("post,gates,scale", [(True, 1, 1.0), (False, 2, 1.25), (True, 0, 0.8), (True, 2, 1.0)])
@pytest.mark.parametrize("n,nnz,B,E,H,F,dt", SHAPES)
def test_layer_and_gradients(n, nnz, B, E, H, F, dt, post, gates, scale):
    base, x, dy, spec = make(n, nnz, B, E, H, F, dt)
    layer = joined(base, 5, post, gates, scale)
    y = layer(x)
    grads = layer.backward(x, dy)
    pmha.pmha_device_status()
    want, leaf = plain(layer, x, spec)
    want.backward(dy.double())
    # the bars of the layer without joins, whose chain two norms make longer by half
    close("y", y, want.detach(), 1.5 * BARS[dt][0])
    for name, v in leaf.items():
        if name == "bk" or v is None:
            assert v is not None or "d" + name not in grads
            continue  # bk: zero in exact arithmetic
        got = grads["dx" if name == "x" else "d" + name]
        assert got.shape == v.shape
        close(name, got, v.grad, 1.5 * BARS[dt][1] * (5 if v.dim() == 1 or name.startswith("gate") else 1))


@pytest.mark.parametrize("kind", ["plain", "joined"])
@pytest.mark.parametrize("n,nnz,B,E,H,F,dt", SHAPES)
def test_step_from_checkpoints(n, nnz, B, E, H, F, dt, kind):
    """The kept training step: the forward pass is the layer's, the gradients are those of the layer at the kept values."""
    layer, x, dy, spec = make(n, nnz, B, E, H, F, dt)
    if kind == "joined":
        layer = joined(layer, 5, True, 2, 0.9)
    y, kept = layer.forward_checkpointed(x)
    exact = layer(x)
    rms = float(exact.double().pow(2).mean().sqrt())
    # the plain layer's join rounds its sum and norm in another order
    assert float((y.double() - exact.double()).abs().max()) <= BARS[dt][0] * rms
    assert (kept.block is None) == (kind == "plain")
    assert kept.nbytes == (2 + (kind != "plain")) * B * n * (E + 2 * (E // 32))
    grads = layer.backward_checkpointed(kept, dy)
    full = layer.backward(x, dy)
    pmha.pmha_device_status()
    assert grads.keys() == full.keys()
    # a code is off by half a scale, 2^-8 of a group's largest value and some 2^-7 of the values' own size: gradients, which
    # are smooth functions of them over few layers, by a few times that in the 2-norm
    for k, v in full.items():
        if v is None or k == "dbk":
            assert grads[k] is not None or v is None
            continue
        off = float((grads[k].double() - v.double()).norm() / v.double().norm())
        assert off < 0.1, f"{k}: {off:.3g}"
    norm = layer.clip_grads(grads, 1.0)
    assert math.isfinite(float(norm))


def test_checkpointed_step_with_mask_captured():
    layer, x, dy, _ = make(200, 1500, 2, 128, 8, 256, "bf16", seed=3)
    layer = joined(layer, 7, True, 2)
    mask = torch.zeros(2, 200, dtype=torch.bool, device=DEV)
    mask[1, 100:] = True

    def step():
        y, kept = layer.forward_checkpointed(x, key_padding_mask=mask)
        return y, layer.backward_checkpointed(kept, dy)

    y, grads = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(grads[k], g2[k]) for k in grads if grads[k] is not None)


@pytest.mark.parametrize("join", [False, True])
def test_served_in_8_and_4_bits(join):
    layer, x, _, _ = make(100, 800, 2, 128, 8, 256, "bf16", seed=5)
    if join:
        layer = joined(layer, 9, True, 1)
    y = layer(x).double()
    s = layer._attend(x, None)[2].double()
    # two operands with 2^-4 at most of error each in both products in 8 bits; in 4 bits values are off by up to 1/6 of a
    # block's largest, 0.1 to 0.15 of the norm a quantized operand, five operands
    for block, bar in ((pmha.FfnQuantizedParams.from_params(layer.block), 0.25),
                       (pmha.FfnMxParams.from_params(layer.block), 0.5)):
        got = layer.serve(x, block).double()
        assert float((got - y).norm() / (y - s).norm()) < bar
    with pytest.raises(TypeError, match="FfnMxParams"):
        layer.serve(x, layer.block)


def test_refusals():
    layer, x, dy, _ = make(64, 256, 1, 32, 4, 40, "f32")
    args = (layer.graph, layer.attention, layer.norm1, layer.norm2, layer.block)
    with pytest.raises(ValueError, match="post1"):
        pmha.PackedEncoderLayer(*args, post1=layer.norm1[:8])
    with pytest.raises(ValueError, match="gate"):
        pmha.PackedEncoderLayer(*args, gate2=torch.ones(3, 8, device=DEV))
    with pytest.raises(pmha.PmhaError, match="divisor"):
        pmha.PackedEncoderLayer(*args, gate1=torch.ones(3, 32, device=DEV))(x)

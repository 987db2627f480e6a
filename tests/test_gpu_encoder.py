"""The encoder layer: norm, packed attention, residual and norm, gated block, its
gradients and their clipping, as one run."""
import math

import numpy as np
import pytest
import torch

import graph_sparse_head_gb300 as pmha
import oracle
import synth
from tests import _encoder_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(n, nnz, B, E, H, F, dt, seed=0):
    rng = np.random.default_rng(seed)
    src, tgt = synth.uniform_graph(rng, n, n, nnz)
    prm = synth.make_params(rng, E, dt)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    graph = pmha.pmha_build_csr(torch.from_numpy(src).to(DEV), torch.from_numpy(tgt).to(DEV), n, n)

    def t(*shape, s=1.0, off=0.0):
        return torch.from_numpy(off + s * rng.standard_normal(shape)).to(dtype).to(DEV)

    block = pmha.FfnParams(t(F, E, s=E ** -0.5), t(F, E, s=E ** -0.5), t(E, F, s=F ** -0.5), t(F, s=0.1), t(F, s=0.1),
                           t(E, s=0.1))
    layer = pmha.PackedEncoderLayer(graph, pmha.Params.from_arrays(prm, H, dtype, DEV), t(E, s=0.1, off=1.0),
                                    t(E, s=0.1, off=1.0), block)
    return layer, t(B, n, E), t(B, n, E), (src, tgt, prm, H)


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
    a, b = layer.attention, layer.block
    w = {k: p(k, getattr(a, k)) for k in ("wq", "wk", "wv", "wo", "bq", "bk", "bv", "bo")}
    norm = lambda v, g: v / torch.sqrt((v * v).mean(-1, keepdim=True) + layer.eps) * g  # noqa: E731
    n1 = norm(x, p("norm1", layer.norm1))
    q, k, v = (n1 @ w["w" + c].t() + w["b" + c] for c in "qkv")
    s, t = (torch.from_numpy(i).to(x.device) for i in (src, tgt))
    score = (q[:, t].view(B, -1, H, d) * k[:, s].view(B, -1, H, d)).sum(-1) / math.sqrt(d)
    e = torch.exp(score - score.amax())
    z = torch.zeros(B, n, H, dtype=e.dtype, device=e.device).index_add(1, t, e)
    wt = e / z[:, t]
    mix = torch.zeros(B, n, H, d, dtype=e.dtype, device=e.device).index_add(1, t, wt[..., None] * v[:, s].view(B, -1, H, d))
    att = mix.reshape(B, n, E) @ w["wo"].t() + w["bo"]
    s1 = x + att
    n2 = norm(s1, p("norm2", layer.norm2))
    g = n2 @ p("wg", b.wg).t() + p("bg", b.bg)
    u = n2 @ p("wu", b.wu).t() + p("bu", b.bu)
    y = s1 + (g * torch.sigmoid(g) * u) @ p("wd", b.wd).t() + p("bd", b.bd)
    return y, leaf


# relative to the largest magnitude class of each tensor: the layer's own bars (2e-2 of the RMS in
# bfloat16, 1e-5 in float32), over the chain's five stages forward and twice as many backward
BARS = {"f32": (5e-5, 1e-4), "bf16": (1e-1, 2e-1)}


@pytest.mark.parametrize("n,nnz,B,E,H,F,dt", [(64, 256, 2, 32, 4, 88, "f32"), (300, 3000, 2, 128, 8, 344, "bf16"),
                                              (130, 900, 1, 256, 8, 512, "bf16")])
def test_layer_and_gradients(n, nnz, B, E, H, F, dt):
    layer, x, dy, spec = make(n, nnz, B, E, H, F, dt)
    y = layer(x)
    grads = layer.backward(x, dy)
    pmha.pmha_device_status()
    want, leaf = plain(layer, x, spec)
    want.backward(dy.double())

    def close(name, got, exp, bar):
        rms = float(exp.pow(2).mean().sqrt())
        off = float((got.double() - exp).abs().max())
        assert off <= bar * rms, f"{name}: {off:.3g} > {bar} x {rms:.3g}"

    close("y", y, want.detach(), BARS[dt][0])
    for name, v in leaf.items():
        if name == "bk":
            continue  # zero in exact arithmetic
        got = grads["dx" if name == "x" else "d" + name]
        close(name, got, v.grad, BARS[dt][1] * (5 if v.dim() == 1 else 1))
    # the clip over what a training step holds: float32 and layer-type gradients together
    before = {k: v.clone() for k, v in grads.items()}
    total = math.sqrt(sum(float((v.double() ** 2).sum()) for k, v in before.items() if k != "dx"))
    norm = layer.clip_grads(grads, 0.5 * total)
    assert abs(float(norm) - total) <= 2.0 ** -18 * total
    assert torch.equal(grads["dx"], before["dx"])
    for k, v in grads.items():
        if k != "dx":
            e = before[k].double() * 0.5 * total / (total + 1e-6)
            assert bool(((v.double() - e).abs() <= (2.0 ** -17 + ref.half_ulp(v.dtype)) * e.abs()).all()), k


def test_layer_with_padding_mask_and_graph_capture():
    layer, x, dy, _ = make(200, 1500, 2, 128, 8, 256, "bf16", seed=3)
    mask = torch.zeros(2, 200, dtype=torch.bool, device=DEV)
    mask[1, 100:] = True
    y = layer(x, key_padding_mask=mask)
    grads = layer.backward(x, dy, key_padding_mask=mask)
    assert not torch.equal(y, layer(x))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = layer(x, key_padding_mask=mask)
        g2 = layer.backward(x, dy, key_padding_mask=mask)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(grads[k], g2[k]) for k in grads if grads[k] is not None)


def test_served_block_in_8_bits():
    """norm -> 8-bit tokens -> quantized block: near the bf16 block by what 8 bits leave."""
    layer, x, _, _ = make(100, 800, 2, 128, 8, 256, "bf16", seed=5)
    q = pmha.FfnQuantizedParams.from_params(layer.block)
    x8, scale, s = pmha.pmha_rms_norm_quantized(x, layer.norm2, layer.eps, residual=x)
    y8 = pmha.pmha_ffn_forward_quantized(q, x8, scale, residual=s)
    n2, s2 = pmha.pmha_rms_norm(x, layer.norm2, layer.eps, residual=x)
    y = pmha.pmha_ffn_forward(layer.block, n2, residual=s2)
    assert torch.equal(s, s2)
    f, f8 = (y.double() - s.double()), (y8.double() - s.double())
    # two operands with 2^-4 at most of error each in both products: far below 1/4 of the norm
    assert float((f - f8).norm() / f.norm()) < 0.25


def test_refusals():
    layer, x, dy, _ = make(64, 256, 1, 32, 4, 40, "f32")
    with pytest.raises(ValueError):
        layer(x.bfloat16())
    with pytest.raises(ValueError):
        pmha.PackedEncoderLayer(layer.graph, layer.attention, layer.norm1[:8], layer.norm2, layer.block)

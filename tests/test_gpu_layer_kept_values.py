"""The checkpointed step's gradients are those of the layer at the kept values, and a served layer's outputs those of the
public calls that it consists of."""
import math

import pytest
import torch

import graph_sparse_head_gb300 as pmha
from tests.test_gpu_encoder import BARS, make
from tests.test_gpu_encoder_joins import close, joined

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def value(k):
    """What a Checkpoint stands for, float64."""
    width = k.shape[-1]
    return k.codes.double() * k.scale.double().repeat_interleave(32, -1)[..., :width]


def at(value, v):
    """v's gradients, at another value."""
    return v + (value - v).detach()


def step_at(layer, kept, spec, mask=None):
    """y of the layer in float64 where its input and its blocks' outputs have the kept values, and the leaves."""
    src, tgt, _, H = spec
    leaf = {}

    def p(name, v):
        leaf[name] = None if v is None else v.double().detach().requires_grad_()
        return leaf[name]

    x = p("x", value(kept.x))
    B, n, E = x.shape
    d = E // H
    a, b = layer.attention, layer.block
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
    if mask is not None:
        e = e * (~mask[:, s])[..., None]
    z = torch.zeros(B, n, H, dtype=e.dtype, device=e.device).index_add(1, t, e)
    z = torch.where(z == 0, 1.0, z)  # no live source: a mix of zeros
    mix = torch.zeros(B, n, H, d, dtype=e.dtype, device=e.device).index_add(
        1, t, (e / z[:, t])[..., None] * v[:, s].view(B, -1, H, d))
    s1 = join(layer.join1, 1, at(value(kept.attention), mix.reshape(B, n, E) @ w["wo"].t() + w["bo"]), x)
    n2 = norm(s1, p("norm2", layer.norm2))
    g = n2 @ p("wg", b.wg).t() + p("bg", b.bg)
    u = n2 @ p("wu", b.wu).t() + p("bu", b.bu)
    f = (g * torch.sigmoid(g) * u) @ p("wd", b.wd).t() + p("bd", b.bd)
    return join(layer.join2, 2, f if kept.block is None else at(value(kept.block), f), s1), leaf


FORMS = {"plain": None, "scale": (False, 0, 1.25), "post": (True, 0, 0.8), "gate": (False, 1, 1.0),
         "all": (True, 2, 0.9)}


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("n,nnz,B,E,H,F,dt", [(64, 256, 2, 32, 4, 88, "f32"), (300, 3000, 2, 128, 8, 344, "bf16")])
def test_gradients_at_the_kept_values(n, nnz, B, E, H, F, dt, form, masked):
    layer, x, dy, spec = make(n, nnz, B, E, H, F, dt)
    if FORMS[form]:
        layer = joined(layer, 5, *FORMS[form])
    mask = None
    if masked:
        mask = torch.zeros(B, n, dtype=torch.bool, device=DEV)
        mask[1, n // 2:] = True
    _, kept = layer.forward_checkpointed(x, key_padding_mask=mask)
    grads = layer.backward_checkpointed(kept, dy)
    pmha.pmha_device_status()
    y, leaf = step_at(layer, kept, spec, mask)
    y.backward(dy.double())
    assert grads.keys() == {"dx" if k == "x" else "d" + k for k, v in leaf.items() if v is not None}
    for name, v in leaf.items():
        if name == "bk" or v is None:
            continue  # bk: zero in exact arithmetic
        got = grads["dx" if name == "x" else "d" + name]
        assert got.shape == v.shape
        # as for the layer's own gradients
        close(name, got, v.grad, 1.5 * BARS[dt][1] * (5 if v.dim() == 1 or name.startswith("gate") else 1))
        # a dozen tensors between x and a gradient are rounded, each value by 2^-8 (float32: 2^-24, and sums of some hundred
        # terms) of itself at most: in norm that much of the whole, were all as large as they can be and of one sign
        off = float((got.double() - v.grad).norm() / v.grad.norm())
        assert off <= (12 * 2.0 ** -8 if dt == "bf16" else 12 * 2.0 ** -17), f"{name}: {off:.3g}"


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("bits", [8, 4])
def test_served_layers_are_their_calls(form, bits):
    layer, x, _, _ = make(100, 800, 2, 128, 8, 256, "bf16", seed=5)
    if FORMS[form]:
        layer = joined(layer, 9, *FORMS[form])
    j1, j2 = layer.join1, layer.join2
    n1, _ = pmha.pmha_rms_norm(x, layer.norm1, layer.eps)
    a, _ = pmha.pmha_forward(layer.graph, layer.attention, n1, n1, n1)
    if form == "plain":
        n2, s = pmha.pmha_rms_norm(a, layer.norm2, layer.eps, residual=x)
    else:
        s, n2 = pmha.pmha_join(j1, a, x)
    residual = s if form == "plain" else None
    if bits == 4:
        block = pmha.FfnMxParams.from_params(layer.block)
        f = pmha.pmha_ffn_forward_mx(block, pmha.pmha_mx_quantize(n2), residual=residual)
    else:
        block = pmha.FfnQuantizedParams.from_params(layer.block)
        q, scale, _ = pmha.pmha_rms_norm_quantized(s, layer.norm2, layer.eps)
        f = pmha.pmha_ffn_forward_quantized(block, q, scale, residual=residual)
    want = f if form == "plain" else pmha.pmha_join(j2, f, s)[0]
    assert torch.equal(layer.serve(x, block), want)

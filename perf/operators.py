"""The encoder operators around the packed attention, as cases to be timed and compared.

A layer built on the packed attention adds the attention's output to its input and
normalises the sum (root mean square), runs a gated feed-forward block on it, and, when it
trains, takes the gradients of all of these and clips them by their global norm. `run`
computes one of these operators, in elementary torch operations where `own` is false, by the
library's calls where it is true. Sizes are those of the workloads in `synth/`: 2 x 64 nodes
of width 32 (float32), 32 x 2,000 and 16 x 20,000 nodes of width 128, 64 samples of 500
pathways and 20,000 genes of width 256, 8 x 1,024 nodes of width 512.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -64  # the smallest scale of an 8-bit row
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the tiny float32 graph's tokens, with the residual's addition: a launch or two
        {"name": "norm tiny f32", "op": "norm", "rows": 128, "width": 32, "dtype": "f32", "residual": True},
        # the 20,000-node graph: every token of 16 samples, attention output + residual stream
        {"name": "norm 20k nodes", "op": "norm", "rows": 320000, "width": 128, "dtype": "bf16", "residual": True},
        # the gene-regulatory graph served with 8-bit activations: the block's input in e4m3 with a scale a token
        {"name": "norm 8 bits genes", "op": "norm_quantized", "rows": 64000, "width": 128, "dtype": "bf16",
         "residual": True},
        # training on the pathway map's genes, the widest token stream: the norm's gradients and the residual's
        {"name": "norm backward map", "op": "norm_backward", "rows": 1280000, "width": 256, "dtype": "bf16",
         "residual": True},
        # one new token through a width-256 block: bound by latency and the weights' read
        {"name": "ffn one token", "op": "ffn", "rows": 1, "width": 256, "hidden": 1024, "dtype": "bf16",
         "act": "silu", "bias": False, "residual": True},
        # float32 layer on the pathway rows of a few samples, hidden width 8/3 of the layer's, not a multiple of 8
        {"name": "ffn f32 odd", "op": "ffn", "rows": 4001, "width": 64, "hidden": 171, "dtype": "f32",
         "act": "silu", "bias": True, "residual": True},
        # the 20,000-node graph's forward pass
        {"name": "ffn 20k nodes", "op": "ffn", "rows": 320000, "width": 128, "hidden": 512, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": True},
        # the complete graph's width-512 layer served from e4m3 tokens and gate / up weights
        {"name": "ffn 8 bits complete", "op": "ffn_quantized", "rows": 8192, "width": 512, "hidden": 2048,
         "dtype": "bf16", "act": "gelu", "bias": False, "residual": True},
        # training on the pathway tokens of the map
        {"name": "ffn backward pathways", "op": "ffn_backward", "rows": 32000, "width": 256, "hidden": 1024,
         "dtype": "bf16", "act": "gelu", "bias": True},
        # training on the 20,000-node graph
        {"name": "ffn backward 20k", "op": "ffn_backward", "rows": 320000, "width": 128, "hidden": 512,
         "dtype": "bf16", "act": "silu", "bias": True},
        # one width-128 layer's gradients: 4 projections and biases in float32, the block's in bfloat16
        {"name": "clip one layer", "op": "clip", "layers": 1, "width": 128, "hidden": 512, "max_norm": 1.0},
        # a stack of width-512 layers
        {"name": "clip stack", "op": "clip", "layers": 24, "width": 512, "hidden": 2048, "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_quantized", "norm_backward", "ffn", "ffn", "ffn_quantized",
                     "ffn_backward", "ffn_backward", "clip"])
    if op == "clip":
        width, hidden = _log(rng, 16, 512), _log(rng, 16, 2048)
        layers = _log(rng, 1, max(2, int(8e7 / (4 * width * width + 3 * width * hidden))))
        return {"op": op, "layers": min(layers, 60), "width": width, "hidden": hidden,
                "max_norm": rng.choice([1.0, 0.1, 1e9])}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # three draws of four are the multiples of 8 that models use, the others any width
    step = rng.choice([8, 8, 64, 1])
    if op.startswith("norm"):
        width = max(1, _log(rng, 24, 2048) // step * step or step)
        rows = _log(rng, 1, min(1280000, 1.6e8 / width))
        return {"op": op, "rows": rows, "width": width, "dtype": dtype, "residual": rng.random() < 0.7}
    if op == "ffn_quantized":
        dtype, step = "bf16", rng.choice([16, 64])
    width = max(step, _log(rng, 16, 1024) // step * step)
    hidden = max(step, min(4096, int(width * rng.uniform(1.0, 4.5))) // step * step)
    most = 2.0e9 if dtype == "f32" else 1.0e10
    rows = _log(rng, 1, max(2, min(320000, most / (width * hidden))))
    case = {"op": op, "rows": rows, "width": width, "hidden": hidden, "dtype": dtype,
            "act": rng.choice(["silu", "gelu"]), "bias": rng.random() < 0.5}
    if op != "ffn_backward":
        case["residual"] = rng.random() < 0.7
    return case


# ---------------------------------------------------------------- inputs

def _quantize_rows(w):
    """Weights in e4m3 with a scale a row: laid out once when a model is loaded."""
    w = w.float()
    scale = (w.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (w / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _layer_sizes(width, hidden):
    """(float32 gradients, layer-type gradients) of one layer, as numbers of values."""
    return [width * width] * 4 + [width] * 4 + [width] * 2, [hidden * width] * 3 + [hidden] * 2 + [width]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype or DTYPES[case["dtype"]])

    s = {"op": case["op"], "case": case}
    if case["op"] == "clip":
        s["max_norm"] = case["max_norm"]
        for key, dtype, sizes in zip(("g32", "g16"), (torch.float32, torch.bfloat16),
                                     _layer_sizes(case["width"], case["hidden"])):
            sizes = sizes * case["layers"]
            places, at = [], 0
            for n in sizes:  # each tensor on a 16-byte boundary of one buffer, as an optimiser lays them out
                places.append((at, n))
                at += (n + 7) // 8 * 8
            flat = normal(at, scale=0.02, dtype=dtype)
            s[key + "_flat"], s[key] = flat, [flat[a:a + n] for a, n in places]
            out = torch.zeros_like(flat)
            s[key + "_out_flat"], s[key + "_out"] = out, [out[a:a + n] for a, n in places]
        return s
    M, E = case["rows"], case["width"]
    if case["op"].startswith("norm"):
        s["x"] = normal(M, E)
        s["residual"] = normal(M, E, scale=2.0) if case["residual"] and case["op"] != "norm_backward" else None
        s["weight"] = (1.0 + normal(E, scale=0.1, dtype=torch.float32)).to(DTYPES[case["dtype"]])
        if case["op"] == "norm_backward":
            s["dout"] = normal(M, E)
            s["dsum"] = normal(M, E) if case["residual"] else None  # the residual stream's own gradient
        return s
    F = case["hidden"]
    s["act"] = case["act"]
    s["x"] = normal(M, E)
    s["wg"], s["wu"] = normal(F, E, scale=E ** -0.5), normal(F, E, scale=E ** -0.5)
    s["wd"] = normal(E, F, scale=F ** -0.5)
    for n, k in (("bg", F), ("bu", F), ("bd", E)):
        s[n] = normal(k, scale=0.1) if case["bias"] else None
    if case["op"] == "ffn_backward":
        s["dout"] = normal(M, E)
    else:
        s["residual"] = normal(M, E) if case["residual"] else None
    if case["op"] == "ffn_quantized":
        s["x8"], s["x_scale"] = _quantize_rows(s.pop("x"))
        s["wg8"], s["wg_scale"] = _quantize_rows(s.pop("wg"))
        s["wu8"], s["wu_scale"] = _quantize_rows(s.pop("wu"))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return _PLAIN[s["op"]](s)


def _run_own(s):
    import graph_sparse_head_gb300 as pmha
    op = s["op"]
    if op == "norm":
        return pmha.pmha_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
    if op == "norm_quantized":
        return pmha.pmha_rms_norm_quantized(s["x"], s["weight"], EPS, residual=s["residual"])
    if op == "norm_backward":
        return pmha.pmha_rms_norm_backward(s["x"], s["weight"], EPS, s["dout"], dsum=s["dsum"])
    if op == "ffn":
        params = pmha.FfnParams(s["wg"], s["wu"], s["wd"], s["bg"], s["bu"], s["bd"], act=s["act"])
        return pmha.pmha_ffn_forward(params, s["x"], residual=s["residual"])
    if op == "ffn_quantized":
        params = pmha.FfnQuantizedParams(s["wg8"], s["wg_scale"], s["wu8"], s["wu_scale"], s["wd"], s["bg"], s["bu"],
                                         s["bd"], act=s["act"])
        return pmha.pmha_ffn_forward_quantized(params, s["x8"], s["x_scale"], residual=s["residual"])
    if op == "ffn_backward":
        params = pmha.FfnParams(s["wg"], s["wu"], s["wd"], s["bg"], s["bu"], s["bd"], act=s["act"])
        return pmha.pmha_ffn_backward(params, s["x"], s["dout"])
    norm = pmha.pmha_clip_grad_norm(s["g32"] + s["g16"], s["max_norm"], out=s["g32_out"] + s["g16_out"])
    return norm, s["g32_out_flat"], s["g16_out_flat"]


def _sum(s):
    """The residual's addition, rounded to the type in which the sum is kept: the norm is of the kept sum."""
    x, residual = s["x"], s["residual"]
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def _plain_norm(s):
    h = _sum(s)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    return y.to(h.dtype), None if s["residual"] is None else h


def _plain_norm_quantized(s):
    # in 64 bits: a value next to a border of the 8-bit grid falls on either side by the last bit of 32
    h = _sum(s)
    f = h.double()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    scale = (y.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN).float()
    q = _to_e4m3(y / scale.double()[:, None])
    return q, scale, None if s["residual"] is None else h


def _to_e4m3(v):
    """e4m3 nearest to 64-bit values, ties to even: 4 significant bits, steps of 2^-9 below 2^-6, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)


def _plain_norm_backward(s):
    x, w, dy = s["x"].float(), s["weight"].float(), s["dout"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * r
    dx = r * (dy * w - xhat * (dy * w * xhat).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0, dtype=torch.float64).float()}


def _linear(x, w, b):
    y = x @ w.float().t()
    return y if b is None else y + b.float()


def _act(name, g):
    """(act(g), its derivative)"""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    p = 0.5 * (1.0 + torch.erf(g * (0.5 ** 0.5)))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _block(s, x, wg, wu):
    h = _act(s["act"], _linear(x, wg, s["bg"]))[0] * _linear(x, wu, s["bu"])
    y = _linear(h, s["wd"], s["bd"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["wd"].dtype)


def _plain_ffn(s):
    return _block(s, s["x"].float(), s["wg"], s["wu"])


def _plain_ffn_quantized(s):
    return _block(s, s["x8"].float() * s["x_scale"][:, None], s["wg8"].float() * s["wg_scale"][:, None],
                  s["wu8"].float() * s["wu_scale"][:, None])


def _plain_ffn_backward(s):
    x, dy = s["x"].float(), s["dout"].float()
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    u = _linear(x, wu, s["bu"])
    a, da = _act(s["act"], _linear(x, wg, s["bg"]))
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    t = s["x"].dtype
    out = {"dx": (dg @ wg + du @ wu).to(t), "dwg": (dg.t() @ x).to(t), "dwu": (du.t() @ x).to(t),
           "dwd": (dy.t() @ (a * u)).to(t)}
    for n, d in (("bg", dg), ("bu", du), ("bd", dy)):
        out["d" + n] = None if s[n] is None else d.sum(0, dtype=torch.float64).to(t)
    return out


def _plain_clip(s):
    total = torch.stack([(g.double() * g.double()).sum() for g in s["g32"] + s["g16"]]).sum()
    norm = torch.sqrt(total)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
    for g, o in zip(s["g32"] + s["g16"], s["g32_out"] + s["g16_out"]):
        o.copy_(g.float() * coef)
    return norm.float(), s["g32_out_flat"], s["g16_out_flat"]


_PLAIN = {"norm": _plain_norm, "norm_quantized": _plain_norm_quantized, "norm_backward": _plain_norm_backward,
          "ffn": _plain_ffn, "ffn_quantized": _plain_ffn_quantized, "ffn_backward": _plain_ffn_backward,
          "clip": _plain_clip}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "clip":
        a, b = (sum(v) * case["layers"] for v in _layer_sizes(case["width"], case["hidden"]))
        return {"bytes": 2 * (4 * a + 2 * b), "flops": 3 * (a + b)}
    M, E, es = case["rows"], case["width"], 4 if case["dtype"] == "f32" else 2
    res = 1 if case.get("residual") else 0
    if case["op"] == "norm":
        return {"bytes": M * E * es * (2 + 2 * res) + E * es, "flops": M * E * (4 + res)}
    if case["op"] == "norm_quantized":
        return {"bytes": M * E * (es * (1 + 2 * res) + 1) + 4 * M + E * es, "flops": M * E * (6 + res)}
    if case["op"] == "norm_backward":
        return {"bytes": M * E * es * (3 + res) + E * (es + 4), "flops": M * E * (9 + res)}
    F, b = case["hidden"], 1 if case["bias"] else 0
    if case["op"] == "ffn_backward":
        return {"bytes": es * (3 * M * E + 6 * E * F + 2 * b * (2 * F + E)), "flops": 16 * M * E * F + 20 * M * F}
    ws, xs = (1, 1) if case["op"] == "ffn_quantized" else (es, es)
    scales = 4 * (M + 2 * F) if case["op"] == "ffn_quantized" else 0
    return {"bytes": M * E * (xs + es * (1 + res)) + 2 * E * F * ws + E * F * es + scales + b * es * (2 * F + E),
            "flops": 6 * M * E * F + 6 * M * F}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op == "clip":
        total = sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["g32"] + s["g16"])
        norm = math.sqrt(total)
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        outs = []
        for key in ("g32", "g16"):
            o = torch.zeros_like(s[key + "_flat"], dtype=torch.float64)
            base = s[key + "_flat"].data_ptr()
            for g in s[key]:
                at = (g.data_ptr() - base) // g.element_size()
                o[at:at + g.numel()] = g.double() * coef
            outs.append(o)
        return torch.tensor(norm, dtype=torch.float64), outs[0], outs[1]
    if op == "norm_backward":
        x, w, dy = d["x"], d["weight"], d["dout"]
        E = case["width"]
        ms = x.square().sum(-1) / E + EPS
        a = dy * w
        dx = a / ms.sqrt()[:, None] - x * ((a * x).sum(-1) / (E * ms * ms.sqrt()))[:, None]
        if d["dsum"] is not None:
            dx += d["dsum"]
        del a
        return {"dx": dx, "dweight": (dy * (x / ms.sqrt()[:, None])).sum(0)}
    if op.startswith("norm"):
        kept = d["x"] if d["residual"] is None else (d["x"] + d["residual"]).float().to(s["x"].dtype).double()
        y = kept / (kept.square().sum(-1, keepdim=True) / case["width"] + EPS).sqrt() * d["weight"]
        kept_out = None if d["residual"] is None else kept
        if op == "norm":
            return y, kept_out
        scale = torch.maximum(y.abs().max(-1).values / E4M3_MAX, torch.tensor(SCALE_MIN, device=y.device)).float()
        v = y / scale.double()[:, None]
        # the 8-bit grid by its exponent: v = m 2^e with m in [1/2, 1), 4 significant bits, not below 2^-9
        e = torch.frexp(v).exponent.clamp_min(-5)
        q = torch.ldexp(torch.round(torch.ldexp(v, 4 - e)), e - 4).clamp(-E4M3_MAX, E4M3_MAX)
        return q, scale.double(), kept_out
    if op == "ffn_quantized":
        x, wg, wu = (d[n + "8"] * d[n + "_scale"][:, None] for n in ("x", "wg", "wu"))
    else:
        x, wg, wu = d["x"], d["wg"], d["wu"]
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    bg, bu, bd = (zero if d[n] is None else d[n] for n in ("bg", "bu", "bd"))
    g, u = torch.einsum("me,fe->mf", x, wg) + bg, torch.einsum("me,fe->mf", x, wu) + bu
    if case["act"] == "silu":
        p = torch.sigmoid(g)
        slope = p + g * p * torch.sigmoid(-g)
    else:
        p = torch.special.ndtr(g)
        slope = p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if op != "ffn_backward":
        y = torch.einsum("mf,ef->me", g * p * u, d["wd"]) + bd
        return y if d["residual"] is None else y + d["residual"]
    dy = d["dout"]
    dh = torch.einsum("me,ef->mf", dy, d["wd"])
    dg, du = dh * u * slope, dh * (g * p)
    out = {"dx": torch.einsum("mf,fe->me", dg, wg) + torch.einsum("mf,fe->me", du, wu),
           "dwg": torch.einsum("mf,me->fe", dg, x), "dwu": torch.einsum("mf,me->fe", du, x),
           "dwd": torch.einsum("me,mf->ef", dy, g * p * u)}
    for n, v in (("bg", dg), ("bu", du), ("bd", dy)):
        out["d" + n] = None if s[n] is None else v.sum(0)
    return out

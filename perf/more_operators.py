"""Operators of the encoder layer's residual stream and of serving it from 4 bits, as cases to be timed and compared.

A stack of encoder layers joins each block's output with the residual stream: the output is
normalised (after the block), multiplied by a gate (a learned one for each channel, or one
for each sample from its condition), added to the residual stream times a scale, and the sum
is normalised again (before the next block). Training keeps the blocks' outputs from the
forward to the backward pass, in 8 bits. Serving takes products of tokens and weights in
microscaled 4-bit floating point. `run` computes one of these operators, in elementary torch
operations where `own` is false, by the library's calls where it is true. Sizes are those of
the workloads in `synth/`: 2 x 64 nodes of width 32 (float32), 32 x 2,000 and 16 x 20,000
nodes of width 128, 64 samples of 500 pathways and 20,000 genes of width 256, 8 x 1,024 nodes
of width 512; one product is larger.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 32              # values of a row that share a scale, in 8 and in 4 bits
LEAST = 2.0 ** -100     # the smallest scale of an 8-bit group
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the tiny float32 graph's tokens: a launch, norms on both sides, a learned gate
        {"name": "join tiny f32", "op": "join", "rows": 128, "width": 32, "dtype": "f32", "post": True, "gates": 1,
         "scale": 1.0},
        # every token of 16 samples of the 20,000-node graph
        {"name": "join 20k nodes", "op": "join", "rows": 320000, "width": 128, "dtype": "bf16", "post": True, "gates": 1,
         "scale": 1.0},
        # the gene-regulatory graph's training step, gates from each sample's condition
        {"name": "join backward genes", "op": "join_backward", "rows": 64000, "width": 128, "dtype": "bf16", "post": True,
         "gates": 32, "scale": 1.0, "dsum": True},
        # the pathway map's genes, the widest token stream; a deep stack scales its residual
        {"name": "join backward map", "op": "join_backward", "rows": 1280000, "width": 256, "dtype": "bf16", "post": True,
         "gates": 1, "scale": 1.5, "dsum": True},
        # an odd width, float32: the last group of a row is a short one
        {"name": "checkpoint f32 odd", "op": "checkpoint", "rows": 4001, "width": 171, "dtype": "f32"},
        # what a layer on the 20,000-node graph keeps of one block
        {"name": "checkpoint 20k nodes", "op": "checkpoint", "rows": 320000, "width": 128, "dtype": "bf16"},
        # one join of a training step, forward and backward through the kept 8 bits: pathway tokens, no norm after the block
        {"name": "step 8 bits pathways", "op": "join_step", "rows": 32000, "width": 256, "dtype": "bf16", "post": False,
         "gates": 64, "scale": 1.0},
        # the same for the 20,000-node graph, norms on both sides
        {"name": "step 8 bits 20k", "op": "join_step", "rows": 320000, "width": 128, "dtype": "bf16", "post": True,
         "gates": 1, "scale": 1.0},
        # one token through a width-512 layer's projection: latency
        {"name": "linear one token", "op": "mx4_linear", "rows": 1, "width": 512, "outputs": 2048, "bias": False,
         "residual": False},
        # a product large enough to be bound by the tensor cores
        {"name": "linear large", "op": "mx4_linear", "rows": 8192, "width": 4096, "outputs": 4096, "bias": True,
         "residual": True},
        # one token through the width-256 block
        {"name": "ffn 4 bits one token", "op": "ffn_mx4", "rows": 1, "width": 256, "hidden": 1024, "act": "silu",
         "bias": False, "residual": True},
        # the complete graph's width-512 layer
        {"name": "ffn 4 bits complete", "op": "ffn_mx4", "rows": 8192, "width": 512, "hidden": 2048, "act": "gelu",
         "bias": True, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join", "join", "join_backward", "join_backward", "checkpoint", "join_step", "mx4_linear",
                     "mx4_linear", "ffn_mx4", "ffn_mx4"])
    step = rng.choice([8, 8, 64, 1])  # three draws of four are the multiples of 8 that models use
    if op == "checkpoint" or op.startswith("join"):
        width = max(16, _log(rng, 16, 2048) // step * step)
        rows = _log(rng, 1, min(1280000, (1.6e8 if op != "join_step" else 4e7) / width))
        case = {"op": op, "rows": rows, "width": width, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"])}
        if op != "checkpoint":
            gates = rng.choice([0, 1, 1, 2])
            if gates == 2:  # a gate a sample
                gates = max(1, min(rows, _log(rng, 2, 64)))
                case["rows"] = rows // gates * gates
            case |= {"post": rng.random() < 0.7, "gates": gates, "scale": rng.choice([1.0, 1.0, 1.5, 0.8])}
        if op == "join_backward":
            case["dsum"] = rng.random() < 0.8
        return case
    width = max(16, _log(rng, 24, 4096 if op == "mx4_linear" else 1024) // step * step)
    if op == "mx4_linear":
        outputs = max(16, _log(rng, 24, 4096) // step * step)
        return {"op": op, "rows": _log(rng, 1, max(2, min(320000, 3e10 / (width * outputs), 3e8 / outputs))), "width": width,
                "outputs": outputs, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    hidden = max(16, min(4096, int(width * rng.uniform(1.0, 4.5))) // step * step)
    return {"op": op, "rows": _log(rng, 1, max(2, min(320000, 1e10 / (width * hidden)))), "width": width,
            "hidden": hidden, "act": rng.choice(["silu", "gelu"]), "bias": rng.random() < 0.5,
            "residual": rng.random() < 0.7}


# ---------------------------------------------------------------- microscaled 4 bits

def _up(n, m):
    return (n + m - 1) // m * m


def _power(e):
    """2^e of whole numbers -1022 .. 1023 in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx4(x):
    """(codes, exponents) of a matrix in blocks of 32 along its rows: the least power of two 2^e, e >= -127, with
    max|block| <= 6 2^e, and the e2m1 value nearest to x 2^-e (ties to the even code). In 64 bits: exact."""
    rows, width = x.shape
    b = torch.zeros(rows, _up(width, GROUP), dtype=torch.float64, device=x.device)
    b[:, :width] = x
    b = b.view(rows, -1, GROUP)
    m, e = torch.frexp(b.abs().amax(-1))          # amax = m 2^e, m in [1/2, 1)
    e = torch.where(m > 0.75, e - 2, e - 3)       # 6 2^(e - 3) = 0.75 2^e
    e = torch.where(m == 0, -127, e).clamp_min(-127)
    v = b * _power(-e)[..., None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    up = torch.bucketize(v.abs(), mid)            # how many borders lie below: a tie stays at the lower code
    tie = (v.abs()[..., None] == mid[1::2]).any(-1)  # and goes up where the lower code is odd
    code = up + tie + 8 * (b < 0)
    return code.view(rows, -1).to(torch.uint8), e


def _pack(x):
    """A matrix as the library lays it out in 4 bits: two codes a byte, the lower column in the low half, rows of a
    multiple of 16 bytes; scale bytes e + 127 in tiles of 128 rows by 4 blocks (512 bytes), row r of a tile at
    16 (r % 32) + 4 (r / 32)."""
    code, e = _mx4(x)
    rows, blocks = e.shape
    packed = code[:, 0::2] | code[:, 1::2] << 4
    s = torch.zeros(_up(rows, 128), _up(blocks, 4), dtype=torch.uint8, device=x.device)
    s[:rows, :blocks] = (e + 127).to(torch.uint8)
    s = s.view(-1, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(s.shape[0] // 128, -1, 512)
    return packed, s


def _unpack(packed, s, width):
    """The values that such a matrix stands for."""
    rows = packed.shape[0]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    v = torch.stack((grid[(packed & 15).long()], grid[(packed >> 4).long()]), -1).view(rows, -1, GROUP)
    e = s.view(s.shape[0], s.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(s.shape[0] * 128, -1)
    e = e[:rows, :v.shape[1]].int() - 127
    return (v * _power(e).float()[..., None]).view(rows, -1)[:, :width]


def _through_mx4(x):
    """x rounded to the 4-bit blocks, as float32 values."""
    code, e = _mx4(x)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
    v = grid[code.long()].view(x.shape[0], -1, GROUP) * _power(e).float()[..., None]
    return v.view(x.shape[0], -1)[:, :x.shape[1]]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype or DTYPES[case.get("dtype", "bf16")])

    op, M, E = case["op"], case["rows"], case["width"]
    s = {"op": op, "case": case}
    if op == "checkpoint":
        s["x"] = normal(M, E)
        return s
    if op.startswith("join"):
        s["branch"], s["residual"] = normal(M, E, scale=0.5), normal(M, E, scale=2.0)
        f32 = torch.float32
        s["pre"] = (1.0 + normal(E, scale=0.1, dtype=f32)).to(s["branch"].dtype)
        s["post"] = (1.0 + normal(E, scale=0.1, dtype=f32)).to(s["branch"].dtype) if case["post"] else None
        s["gate"] = normal(case["gates"], E, scale=0.7) if case["gates"] else None
        if op != "join":
            s["dout"] = normal(M, E)
            s["dsum"] = normal(M, E) if case.get("dsum", True) else None
        if op == "join_backward":  # the forward pass left its sum
            s["sum"] = _plain_join(s)[0]
            del s["residual"]
        return s
    # tokens with a few strong channels, as norms leave them
    s["x"] = (normal(M, E, dtype=torch.float32) * torch.exp(normal(E, scale=0.7, dtype=torch.float32))).bfloat16()
    if op == "mx4_linear":
        N = case["outputs"]
        s["w"] = _pack(normal(N, E, scale=E ** -0.5))
        s["bias"] = normal(N, scale=0.1) if case["bias"] else None
        s["residual"] = normal(M, N) if case["residual"] else None
        return s
    F = case["hidden"]
    s["wg"], s["wu"] = _pack(normal(F, E, scale=E ** -0.5)), _pack(normal(F, E, scale=E ** -0.5))
    s["wd"] = _pack(normal(E, F, scale=F ** -0.5))
    for n, k in (("bg", F), ("bu", F), ("bd", E)):
        s[n] = normal(k, scale=0.1) if case["bias"] else None
    s["residual"] = normal(M, E) if case["residual"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return _PLAIN[s["op"]](s)


def _run_own(s):
    import graph_sparse_head_gb300 as pmha
    op, case = s["op"], s["case"]
    if op == "checkpoint":
        return pmha.pmha_checkpoint_restore(pmha.pmha_checkpoint(s["x"]))
    if op.startswith("join"):
        p = pmha.JoinParams(pre=s["pre"], post=s["post"], gate=s["gate"], residual_scale=case["scale"], eps=EPS)
        if op == "join":
            return pmha.pmha_join(p, s["branch"], s["residual"])
        if op == "join_backward":
            return pmha.pmha_join_backward(p, s["branch"], s["sum"], s["dout"], s["dsum"])
        h, n, kept, _ = pmha.pmha_join_checkpointed(p, s["branch"], s["residual"], keep_residual=False)
        return {"sum": h, "out": n, **pmha.pmha_join_backward(p, kept, h, s["dout"], s["dsum"])}
    x = pmha.pmha_mx_quantize(s["x"])
    E = case["width"]
    if op == "mx4_linear":
        w = pmha.MxTensor(*s["w"], (case["outputs"], E))
        return pmha.pmha_mx_linear(x, w, bias=s["bias"], residual=s["residual"])
    F = case["hidden"]
    wg, wu, wd = (pmha.MxTensor(*s[n], shape) for n, shape in (("wg", (F, E)), ("wu", (F, E)), ("wd", (E, F))))
    params = pmha.FfnMxParams(wg, wu, wd, s["bg"], s["bu"], s["bd"], act=case["act"])
    return pmha.pmha_ffn_forward_mx(params, x, residual=s["residual"])


def _gates(s):
    """The gate of every row, or 1."""
    if s["gate"] is None:
        return 1.0
    g = s["gate"].float()
    return g.repeat_interleave(s["case"]["rows"] // g.shape[0], 0) if g.shape[0] > 1 else g


def _root(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_join(s):
    z = s["branch"].float()
    if s["post"] is not None:
        z = z * _root(z) * s["post"].float()
    h = (s["case"]["scale"] * s["residual"].float() + _gates(s) * z).to(s["branch"].dtype)  # kept, and normalised as kept
    f = h.float()
    return h, (f * _root(f) * s["pre"].float()).to(h.dtype)


def _through_norm(x, a):
    """The gradient of x for a = the gradient of x / sqrt(mean(x^2) + eps)."""
    r = _root(x)
    return r * (a - x * (r * r * (a * x).mean(-1, keepdim=True)))


def _backward(s, b, h):
    t = s["branch"].dtype
    f, dy = h.float(), s["dout"].float()
    d = _through_norm(f, dy * s["pre"].float())
    if s["dsum"] is not None:
        d = d + s["dsum"].float()
    out = {"dresidual": (s["case"]["scale"] * d).to(t),
           "dpre": (dy * (f * _root(f))).sum(0, dtype=torch.float64).float()}
    z, dz = b, _gates(s) * d
    out["dpost"] = None
    if s["post"] is not None:
        bhat = b * _root(b)
        out["dpost"] = (dz * bhat).sum(0, dtype=torch.float64).float()
        z = bhat * s["post"].float()
        dz = _through_norm(b, dz * s["post"].float())
    out["dbranch"] = dz.to(t)
    out["dgate"] = None
    if s["gate"] is not None:
        G, E = s["gate"].shape
        out["dgate"] = (d * z).view(G, -1, E).sum(1, dtype=torch.float64).float()
    return {n: out[n] for n in ("dbranch", "dresidual", "dpre", "dpost", "dgate")}


def _plain_backward(s):
    return _backward(s, s["branch"].float(), s["sum"])


def _through_8_bits(x):
    """x rounded to codes of -127 .. 127 times a bfloat16 scale a group of 32, in 64 bits: a value next to a border falls
    on either side by the last bit of 32."""
    rows, width = x.shape
    b = torch.zeros(rows, _up(width, GROUP), dtype=torch.float64, device=x.device)
    b[:, :width] = x
    b = b.view(rows, -1, GROUP)
    most = b.abs().amax(-1) / 127.0
    m, e = torch.frexp(most)
    scale = (torch.ceil(m * 256.0) * _power(e - 8)).clamp_min(LEAST)  # max|group| / 127 rounded up to 8 bits
    return (torch.round(b / scale[..., None]) * scale[..., None]).view(rows, -1)[:, :width]


def _plain_checkpoint(s):
    return _through_8_bits(s["x"]).to(s["x"].dtype)


def _plain_step(s):
    h, n = _plain_join(s)
    return {"sum": h, "out": n, **_backward(s, _through_8_bits(s["branch"]).float(), h)}


def _product(x, w, bias):
    y = x @ w.t()
    return y if bias is None else y + bias.float()


def _plain_linear(s):
    y = _product(_through_mx4(s["x"]), _unpack(*s["w"], s["case"]["width"]), s["bias"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.bfloat16()


def _act(name, g):
    return g / (1.0 + torch.exp(-g)) if name == "silu" else g * 0.5 * (1.0 + torch.erf(g * (0.5 ** 0.5)))


def _plain_ffn(s):
    E, F = s["case"]["width"], s["case"]["hidden"]
    x = _through_mx4(s["x"])
    h = _act(s["case"]["act"], _product(x, _unpack(*s["wg"], E), s["bg"])) * _product(x, _unpack(*s["wu"], E), s["bu"])
    y = _product(_through_mx4(h), _unpack(*s["wd"], F), s["bd"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.bfloat16()


_PLAIN = {"join": _plain_join, "join_backward": _plain_backward, "join_step": _plain_step, "checkpoint": _plain_checkpoint,
          "mx4_linear": _plain_linear, "ffn_mx4": _plain_ffn}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    M, E, es = case["rows"], case["width"], 4 if case.get("dtype") == "f32" else 2
    op = case["op"]
    if op == "checkpoint":  # there and back: the tensor read, the restored one written
        return {"bytes": 2 * M * E * es, "flops": 3 * M * E}
    if op.startswith("join"):
        weights = E * es * (1 + case["post"] + case["gates"])
        sums = 4 * E * (1 + case["post"] + case["gates"])
        if op == "join":
            return {"bytes": 4 * M * E * es + weights, "flops": 12 * M * E}
        if op == "join_backward":
            needs_branch = 1 if case["post"] or case["gates"] else 0
            return {"bytes": (4 + needs_branch + case["dsum"]) * M * E * es + weights + sums, "flops": 24 * M * E}
        return {"bytes": 8 * M * E * es + weights + sums, "flops": 40 * M * E}
    b, r = 1 if case["bias"] else 0, 1 if case["residual"] else 0
    if op == "mx4_linear":
        N = case["outputs"]
        return {"bytes": 2 * M * E + 17 * N * E // 32 + 2 * M * N * (1 + r) + 2 * b * N, "flops": 2 * M * N * E}
    F = case["hidden"]
    return {"bytes": 2 * M * E * (2 + r) + 17 * 3 * F * E // 32 + 2 * b * (2 * F + E), "flops": 6 * M * E * F + 6 * M * F}


# ---------------------------------------------------------------- the definition, in 64 bits

def _powers(device):
    return torch.tensor([2.0 ** e for e in range(-127, 129)], dtype=torch.float64, device=device)


def _grid4(x):
    """x on its blocks' e2m1 grid: the scale is the first power of two whose sixfold reaches the largest value."""
    pad = -x.shape[1] % GROUP
    b = torch.nn.functional.pad(x.double(), (0, pad)).unflatten(1, (-1, GROUP))
    powers = _powers(x.device)
    scale = powers[torch.searchsorted(6.0 * powers, b.abs().amax(-1, keepdim=True))]
    v = b / scale
    step = torch.where(v.abs() < 2.0, 0.5, torch.where(v.abs() < 4.0, 1.0, 2.0))  # 2 significant bits, steps of 1/2 below 1
    return (torch.round(v / step) * step * scale).flatten(1)[:, :x.shape[1]]


def _grid8(x):
    pad = -x.shape[1] % GROUP
    b = torch.nn.functional.pad(x.double(), (0, pad)).unflatten(1, (-1, GROUP))
    least = b.abs().amax(-1, keepdim=True) / 127.0
    powers = _powers(x.device)
    ulp = powers[torch.searchsorted(powers, least.clamp_min(LEAST), right=True) - 1] / 128.0  # of 8 significant bits
    scale = (torch.ceil(least / ulp) * ulp).clamp_min(LEAST)
    return (torch.round(b / scale) * scale).flatten(1)[:, :x.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return _grid8(s["x"])
    if op.startswith("join"):
        t = s["branch"].dtype
        d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
        E = case["width"]
        gate = None if d["gate"] is None else d["gate"].unsqueeze(1)  # (G, 1, E) beside (G, rows, E)

        def gated(v):
            return v if gate is None else (v.view(gate.shape[0], -1, E) * gate).view(v.shape)

        out = []
        if op != "join_backward":
            z = d["branch"]
            if d["post"] is not None:
                z = z / (z.square().sum(-1, keepdim=True) / E + EPS).sqrt() * d["post"]
            kept = torch.add(gated(z), d["residual"], alpha=case["scale"]).to(t).double()
            out = [kept, kept / (kept.square().sum(-1, keepdim=True) / E + EPS).sqrt() * d["pre"]]
            if op == "join":
                return tuple(out)
            branch = _grid8(s["branch"])
        else:
            kept, branch = d["sum"], d["branch"]
        ms = (kept.square().sum(-1, keepdim=True) / E + EPS).sqrt()
        a = d["dout"] * d["pre"]
        D = a / ms - kept * ((a * kept).sum(-1, keepdim=True) / (E * ms ** 3))
        if d["dsum"] is not None:
            D += d["dsum"]
        grads = {"dresidual": case["scale"] * D, "dpre": torch.einsum("me,me->e", d["dout"], kept / ms), "dpost": None,
                 "dgate": None}
        if d["post"] is None:
            unit, dz = branch, gated(D)
        else:
            mb = (branch.square().sum(-1, keepdim=True) / E + EPS).sqrt()
            unit = branch / mb
            grads["dpost"] = torch.einsum("me,me->e", gated(D), unit)
            a = gated(D) * d["post"]
            dz = (a - unit * ((a * unit).sum(-1, keepdim=True) / E)) / mb
            unit = unit * d["post"]
        grads["dbranch"] = dz
        if gate is not None:
            grads["dgate"] = torch.einsum("gre,gre->ge", D.view(gate.shape[0], -1, E), unit.view(gate.shape[0], -1, E))
        grads = {n: grads[n] for n in ("dbranch", "dresidual", "dpre", "dpost", "dgate")}
        return grads if op == "join_backward" else {"sum": out[0], "out": out[1], **grads}
    zero = torch.zeros((), dtype=torch.float64, device=s["x"].device)
    x = _grid4(s["x"])

    def value(name, width):
        return _unpack(*s[name], width).double()

    def term(name):
        return zero if s[name] is None else s[name].double()

    if op == "mx4_linear":
        return torch.einsum("me,ne->mn", x, value("w", case["width"])) + term("bias") + term("residual")
    E, F = case["width"], case["hidden"]
    g = torch.einsum("me,fe->mf", x, value("wg", E)) + term("bg")
    u = torch.einsum("me,fe->mf", x, value("wu", E)) + term("bu")
    h = g * (torch.sigmoid(g) if case["act"] == "silu" else torch.special.ndtr(g)) * u
    return torch.einsum("mf,ef->me", _grid4(h), value("wd", F)) + term("bd") + term("residual")

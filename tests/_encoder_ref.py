"""Plain 64-bit forms of the encoder operators, with first-order error bounds.

Bounds count roundings: a rounding to type t is off by at most
finfo(t).eps / 2 of the value. Products on the tensor cores accumulate in
float32; their adders may cut instead of round, so that a sum of K products is
held to K * 2^-22 of the sum of magnitudes (twice the two bits that alignment
and cutting can cost), one on the CUDA cores to K * 2^-24."""
import math

import torch

EPS = 1e-6


def half_ulp(dtype):
    return torch.finfo(dtype).eps / 2


def norm(x, w, eps=EPS):
    """(y, 1/rms) of rows in float64."""
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r * (1.0 if w is None else w.double()), r


def stat_tol(width):
    """Relative error of the float32 root: a lane's chain of at most width / 32 + 32 squares, its
    shuffles, the division, the root (2 ulp) and the two products."""
    return (width / 32 + 48) * 2.0 ** -24


def norm_backward(x, w, dy, ds, eps=EPS):
    """dx, dw and the magnitudes that their rounding errors are relative to."""
    width = x.shape[-1]
    _, r = norm(x, None, eps)
    x, dy = x.double(), dy.double()
    a = dy * (1.0 if w is None else w.double())
    k = (a * x).sum(-1, keepdim=True) * r * r / width
    dx = r * (a - x * k)
    k_mag = (a * x).abs().sum(-1, keepdim=True) * r * r / width
    mag = r * (a.abs() + x.abs() * k_mag)
    if ds is not None:
        dx, mag = dx + ds.double(), mag + ds.double().abs()
    flat = (dy * x * r).reshape(-1, width)
    return dx, mag, flat.sum(0), flat.abs().sum(0)


def e4m3_round(v):
    """Nearest E4M3 value, ties to even, of float64 values."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def quantized(y):
    scale = (y.abs().amax(-1) / 448.0).clamp_min(2.0 ** -64).float()
    return e4m3_round(y / scale.double()[..., None]), scale


def act(name, g):
    """act(g), its slope, a bound of the slope's own derivative."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    p = torch.special.ndtr(g)
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


class Block:
    """A gated block's tensors (any type) and its formulas in float64."""

    def __init__(self, wg, wu, wd, bg, bu, bd, name):
        self.w = [t.double() for t in (wg, wu, wd)]
        self.b = [None if t is None else t.double() for t in (bg, bu, bd)]
        self.name, self.dtype = name, wd.dtype
        self.bf16 = wd.dtype == torch.bfloat16
        self.acc = 2.0 ** -22 if self.bf16 else 2.0 ** -24
        self.store = half_ulp(torch.bfloat16) if self.bf16 else half_ulp(torch.float32)
        # the activation's own arithmetic: 2^-20 covers the approximate exponential and division
        self.act_tol = 2.0 ** -19 if self.bf16 else 2.0 ** -21

    def hidden(self, x):
        (wg, wu, _), (bg, bu, _) = self.w, self.b
        z = torch.zeros((), dtype=torch.float64, device=x.device)
        g = x @ wg.t() + (z if bg is None else bg)
        u = x @ wu.t() + (z if bu is None else bu)
        k = (x.shape[-1] + 4) * self.acc
        dg = k * (x.abs() @ wg.abs().t() + (z if bg is None else bg.abs()))
        du = k * (x.abs() @ wu.abs().t() + (z if bu is None else bu.abs()))
        return g, u, dg, du

    def forward(self, x, residual):
        """y and a bound of each value's error."""
        x = x.double()
        g, u, eg, eu = self.hidden(x)
        a, slope = act(self.name, g)
        h = a * u
        eh = (slope.abs() + 0.5 * eg) * eg * u.abs() + a.abs() * eu + self.act_tol * (a.abs() + 2.0 ** -20) * u.abs()
        eh = eh + self.store * h.abs()
        wd, bd = self.w[2], self.b[2]
        y = h @ wd.t()
        mag = h.abs() @ wd.abs().t()
        if bd is not None:
            y, mag = y + bd, mag + bd.abs()
        if residual is not None:
            y, mag = y + residual.double(), mag + residual.double().abs()
        err = eh @ wd.abs().t() + (h.shape[-1] + 4) * self.acc * mag + half_ulp(self.dtype) * y.abs()
        return y, 1.01 * err + 1e-30

    def backward(self, x, dy):
        """{name: (gradient, bound)}"""
        x, dy = x.double(), dy.double()
        wg, wu, wd = self.w
        rows = x.shape[0]
        g, u, eg, eu = self.hidden(x)
        a, slope = act(self.name, g)
        ea = (slope.abs() + 0.5 * eg) * eg + self.act_tol * (a.abs() + 2.0 ** -20)
        es = eg + self.act_tol * (1.0 + slope.abs())  # |second derivative| < 1 for both
        dh = dy @ wd
        edh = (x.shape[-1] + 4) * self.acc * (dy.abs() @ wd.abs())
        h, du, dg = a * u, dh * a, dh * u * slope
        eh = ea * u.abs() + a.abs() * eu + self.store * h.abs()
        edu = edh * a.abs() + dh.abs() * ea + self.store * du.abs()
        edg = edh * (u * slope).abs() + dh.abs() * (eu * slope.abs() + u.abs() * es) + self.store * dg.abs()
        t = half_ulp(self.dtype)
        F = h.shape[-1]

        def product(p, ep, q, k):
            return p @ q, ep @ q.abs() + (k + 4) * self.acc * (p.abs() @ q.abs())

        out = {}
        d1, e1 = product(dg, edg, wg, 2 * F)
        d2, e2 = product(du, edu, wu, 2 * F)
        out["dx"] = (d1 + d2, e1 + e2)
        out["dwg"] = product(dg.t(), edg.t(), x, rows)
        out["dwu"] = product(du.t(), edu.t(), x, rows)
        v, e = product(h.t(), eh.t(), dy, rows)
        out["dwd"] = (v.t(), e.t())
        for n, d, ed in (("dbg", dg, edg), ("dbu", du, edu), ("dbd", dy, torch.zeros_like(dy))):
            out[n] = (d.sum(0), ed.sum(0) + (rows + 4) * 2.0 ** -24 * d.abs().sum(0))
        return {n: (v, 1.01 * (e + t * v.abs()) + 1e-30) for n, (v, e) in out.items()}


def assert_within(name, got, ref, bound):
    """Every value within its bound; the message tells the worst."""
    assert got.shape == ref.shape, f"{name}: shape {tuple(got.shape)}, want {tuple(ref.shape)}"
    over = (got.double() - ref).abs() / bound
    worst = float(over.nan_to_num(nan=math.inf).max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound at {int(over.nan_to_num(nan=math.inf).argmax())}"

"""Plain 64-bit forms of the join with the residual stream and of tensors kept in
8 bits, with error bounds that count float32 roundings (2^-24 each) relative to
the magnitudes they are made on, and the last one to the type."""
import torch

from tests._encoder_ref import half_ulp


def tol(width):
    """A statistic's float32 chain (a thread's part of the row, its team's sums), the root and a few products."""
    return (width / 32 + 64) * 2.0 ** -24


def kept(x):
    """(codes as float64, scales) of a tensor kept in 8 bits."""
    rows, width = x.reshape(-1, x.shape[-1]).shape
    b = torch.zeros(rows, (width + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    b[:, :width] = x.reshape(rows, width)
    b = b.view(rows, -1, 32)
    m, e = torch.frexp(b.abs().amax(-1) / 127.0)
    scale = (torch.ceil(m * 256) * 2.0 ** -8 * ((e.long() + 1023) << 52).view(torch.float64)).clamp_min(2.0 ** -100)
    codes = torch.round(b / scale[..., None]).view(rows, -1)[:, :width]
    return codes.reshape(x.shape), scale.reshape(*x.shape[:-1], -1)


def restored(x):
    """What a kept tensor stands for, in float64."""
    codes, scale = kept(x)
    return codes * scale.repeat_interleave(32, -1)[..., :x.shape[-1]]


def gates_of(gate, rows):
    """Gate rows of all rows, in float64."""
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    g = gate.double().reshape(-1, gate.shape[-1])
    return g.repeat_interleave(rows // g.shape[0], 0)


def root(x, eps):
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def join_sum(branch, residual, post, gate, alpha, eps):
    """sum before its rounding and the bound of its error with it; float64 rows."""
    width = residual.shape[-1]
    z = torch.zeros_like(residual) if branch is None else branch
    t = 0.0
    if post is not None:
        z = z * root(z, eps) * post.double()
        t = tol(width)
    z = z * gates_of(gate, residual.shape[0]).to(z.device)
    s = alpha * residual + z
    # alpha itself is rounded to float32
    return s, (t + 2.0 ** -22) * z.abs() + 2.0 ** -23 * (alpha * residual).abs()


def backward(branch, s, dout, dsum, post, gate, pre, alpha, eps):
    """{name: (gradient, bound)} of float64 rows; `final` roundings to the type are added by the caller's dtype."""
    like = dsum if dout is None else dout
    rows, width = like.shape
    t = tol(width)
    D = torch.zeros_like(like) if dsum is None else dsum.clone()
    mag = D.abs()
    out = {}
    if dout is not None:
        r = root(s, eps)
        u, a = s * r, dout * pre.double()
        k = (a * u).mean(-1, keepdim=True)
        k_mag = (a * u).abs().mean(-1, keepdim=True)
        D = D + r * (a - u * k)
        mag = mag + r * (a.abs() + u.abs() * k_mag)
        q = (dout * u).abs().sum(0)
        out["dpre"] = ((dout * u).sum(0), 2 * t * q + 160 * 2.0 ** -24 * q)
    eD = 2 * t * mag
    out["dresidual"] = (alpha * D, abs(alpha) * (eD + 2.0 ** -23 * D.abs()))
    w = gates_of(gate, rows).to(D.device).expand_as(D).clone()
    if branch is not None or post is None:
        u = branch
        if post is not None:
            rb = root(branch, eps)
            u = branch * rb
        if u is not None:
            term, mterm = D * u, mag * u.abs()
            if post is not None:
                m = (w * mterm).abs().sum(0)
                out["dpost"] = ((w * term).sum(0), (4 * t + 160 * 2.0 ** -24) * m)
            if gate is not None:
                p = 1.0 if post is None else post.double()
                G = gate.reshape(-1, width).shape[0]
                sums = (term * p).view(G, -1, width).sum(1)
                m = (mterm * p).abs().view(G, -1, width).sum(1)
                out["dgate"] = (sums.view(gate.shape), ((4 * t + 160 * 2.0 ** -24) * m).view(gate.shape))
        if post is None:
            out["dbranch"] = (D * w, (w * (eD + 2.0 ** -22 * D.abs())).abs())
        else:
            a, amag = D * w * post.double(), (mag * w * post.double()).abs()
            k = (a * u).mean(-1, keepdim=True)
            k_mag = (amag * u.abs()).mean(-1, keepdim=True)
            out["dbranch"] = (rb * (a - u * k), 4 * t * rb * (amag + u.abs() * k_mag))
    return out


def with_rounding(v, bound, dtype):
    return v, 1.01 * (bound + half_ulp(dtype) * v.abs()) + 1e-37

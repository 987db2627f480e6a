"""Plain 64-bit forms of microscaled 4-bit floating point."""
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def blocks_of(x):
    """(rows, blocks, 32) in float64, zeros past the width."""
    rows, width = x.shape
    b = torch.zeros(rows, (width + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    b[:, :width] = x
    return b.view(rows, -1, 32)


def quantize(x):
    """(codes (rows, blocks, 32), exponents (rows, blocks)) of a finite matrix."""
    b = blocks_of(x)
    top = b.abs().amax(-1)
    e = torch.full(top.shape, -127, dtype=torch.long, device=x.device)
    for k in range(-127, 127):  # the least power whose sixfold reaches the largest value
        e = torch.where(top > 6.0 * 2.0 ** k, k + 1, e)
    v = (b / power(e)[..., None]).abs()
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    d = (v[..., None] - grid).abs()
    near = d.amin(-1, keepdim=True)
    hit = d == near
    # of two codes as near, the even one
    score = torch.where(hit, torch.arange(8, device=x.device) % 2, 9)
    code = score.argmin(-1)
    return code + 8 * torch.signbit(b), e  # a zero keeps its sign


def values(x):
    """What the quantized matrix stands for, float64."""
    code, e = quantize(x)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=x.device)
    return (grid[code] * power(e)[..., None]).flatten(1)[:, :x.shape[1]]


def packed(x):
    """(codes, scale) as the library lays them out."""
    code, e = quantize(x)
    c = code.flatten(1).to(torch.uint8)
    rows, blocks = e.shape
    s = torch.zeros((rows + 127) // 128 * 128, (blocks + 3) // 4 * 4, dtype=torch.uint8, device=x.device)
    s[:rows, :blocks] = (e + 127).to(torch.uint8)
    out = torch.zeros(s.shape[0] // 128, s.shape[1] // 4, 512, dtype=torch.uint8, device=x.device)
    for r in range(128):
        for k in range(4):
            out[:, :, 16 * (r % 32) + 4 * (r // 32) + k] = s[r::128, k::4]
    return c[:, 0::2] | c[:, 1::2] << 4, out

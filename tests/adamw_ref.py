"""The AdamW step in 64 bits (torch float64, CPU), from its definition."""
import torch

F64 = torch.float64
U = 2.0 ** -24  # fp32 unit roundoff


def hash32(x):
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ (x >> shift)) * factor) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(seed, t, tensor, index):
    """32 random bits of the elements `index` (int64 tensor) of one tensor."""
    key = hash32(hash32(t & 0xFFFFFFFF) ^ seed)
    key = hash32((key + tensor) & 0xFFFFFFFF)
    return hash32((hash32((key + (index >> 32)) & 0xFFFFFFFF) + (index & 0xFFFFFFFF)) & 0xFFFFFFFF)


def e4m3_grid():
    low = [k * 2.0 ** -9 for k in range(8)]
    return torch.tensor(low + [(8 + k) * 2.0 ** (e - 3) for e in range(-6, 9) for k in range(8)][:119], dtype=F64)


def two_to(e):
    return torch.pow(torch.tensor(2.0, dtype=F64), e.to(F64))  # (exact on the CPU)


def held(x, bits16, least):
    """What 8-bit moments hold of x (64 bits, one tensor): values, and how far
    each element was from turning to the other of its two codes (in units of
    their distance)."""
    n = x.numel()
    b = torch.zeros((n + 31) // 32 * 32, dtype=F64)
    b[:n] = x
    b = b.view(-1, 32)
    r = torch.zeros(b.numel(), dtype=F64)
    r[:n] = bits16.to(F64) / 65536
    top = b.abs().amax(1)
    f, k = torch.frexp(top)
    e = torch.where(top > 0, (k - 9 + (f > 0.875).to(k.dtype)).clamp_min(-127), -127)
    a = b.abs() / two_to(e).unsqueeze(1)
    grid = e4m3_grid()
    at = torch.searchsorted(grid, a.contiguous(), right=True) - 1
    low, high = grid[at], grid[(at + 1).clamp_max(grid.numel() - 1)]
    gap = torch.where(high > low, high - low, 1.0)
    over = (a - low) / gap + r.view(-1, 32) - 1
    q = torch.where(over >= 0, high, low)
    if least:
        q = torch.where((a > 0) & (q == 0), grid[1], q)
    v = torch.copysign(q, b) * two_to(e).unsqueeze(1)
    return v.view(-1)[:n], over.abs().view(-1)[:n]


def step(w, m, v, g, t, lr, betas, eps, wd, c=1.0):
    """(w, m, v) after step t (1-based) of one tensor; c: the clipping factor."""
    b1, b2 = betas
    g = g.to(F64) * c
    m = m.to(F64) * b1 + g * (1 - b1)
    v = v.to(F64) * b2 + (g * g) * (1 - b2)
    w = w.to(F64)
    w = w * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    return w, m, v

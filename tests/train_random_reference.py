"""8-bit codes rounded at random, operation by operation as the library's step
rounds them (float32 and 32-bit integers; beside train_reference.py)."""
import torch

from tests import train_reference as R

M32 = 0xFFFFFFFF


def mixed(x, salt):
    """32 bits (in int64) that look random, of two times 32 others."""
    x = (x * 0x6A09E667 + salt) & M32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & M32
    x = x ^ (x >> 16)
    return (x * 0x3C6EF373) & M32


def bits(x):
    return x.contiguous().view(torch.int32).to(torch.int64) & M32


def floats(b):
    b = torch.where(b >= 1 << 31, b - (1 << 32), b)
    return b.to(torch.int32).view(torch.float32)


def chances(v, steps):
    """The chances of roots and of m (32 bits each) for rows of 256 second
    moments, in the step after `steps`."""
    salt = mixed(torch.tensor(steps & M32), mixed(torch.tensor(steps >> 32), 1))
    h = mixed(bits(v), (salt + torch.arange(256) * 0x9E3779B9) & M32)
    return h, (h * 0x9E3779B9) & M32


def random_code(x, chance):
    """The upper 20 bits of the chance are added to the way between two codes."""
    b = (bits(x * 2.0 ** -120) + (chance >> 12)) & 0xFFF00000
    return torch.clamp(floats(b) * 2.0 ** 120, -448, 448)


def neighbours(y):
    """The codes at or below and above y >= 0."""
    lo = bits(y * 2.0 ** -120) & 0xFFF00000
    return floats(lo) * 2.0 ** 120, floats(lo + 0x100000) * 2.0 ** 120


def random_root(y, chance):
    lo, hi = neighbours(y)
    d = lambda t: t.double()  # noqa: E731
    way, gap = (d(y) ** 2 - d(lo) ** 2).float(), (d(hi) ** 2 - d(lo) ** 2).float()
    u = (chance >> 9).float() * 2.0 ** -23
    return torch.clamp(torch.where(way > u * gap, hi, lo), max=448)


def encode(m, v, steps):
    """((codes, scale) of m, (codes, scale) of the root of v) for finite float32
    rows of 256, in the step after `steps` ones."""
    (h, hm), root = chances(v, steps), v.sqrt()
    out = []
    for x, code in ((m, lambda y: random_code(y, hm)), (root, lambda y: random_root(y, h))):
        scale = x.abs().amax(1).clamp(min=2.0 ** -100) * torch.tensor(1 / 448, dtype=torch.float32)
        inv = torch.ones_like(scale) / scale
        out.append((code(x * inv[:, None]), scale))
    (m, ms), (r, rs) = out
    r = torch.where((root > 0) & (r == 0), 2.0 ** -9, r.double()).float()
    return (m.to(torch.float8_e4m3fn), ms), (r.to(torch.float8_e4m3fn), rs)


def step(g, state, steps, b1, b2):
    """New (m codes, m scale, root codes, root scale) and the float32 m and v
    before their rounding."""
    m, ms, r, rs = state
    r = R.decode(r, rs)
    m, v, _ = R.adamw_moments(g, R.decode(m, ms), r * r, b1, b2)
    (mc, ms), (rc, rs) = encode(m, v, steps)
    return (mc, ms, rc, rs), m, v

"""Plain float64 forms of the serving operators, on the CPU, and the error
bounds their tests allow.  Nothing of the library is used here.

Bounds.  U32 = 2^-23 bounds one float32 step of a sum on the tensor cores
(which may truncate) or the FMA units; a sum of R terms is within
R * U32 * sum|terms| of its exact value.  HALF[dtype] is the half-ulp of the
final rounding, relative to the value."""
import math

import torch

U32 = 2.0 ** -23
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def rotate(x, table, positions, interleaved):
    """x (n, heads, D) float64 rotated; also sum of the magnitudes of the two products."""
    R = table.shape[1]
    y, mag = x.clone(), x.abs()
    for t, p in enumerate(positions):
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c, s = table[p, i], table[p, R // 2 + i]
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
            mag[t, :, a] = (x[t, :, a] * c).abs() + (x[t, :, b] * s).abs()
            mag[t, :, b] = (x[t, :, b] * c).abs() + (x[t, :, a] * s).abs()
    return y, mag


def gather(cache, table_row, first, last):
    """(kv_heads, last - first, D): the tokens of one sequence."""
    P = cache.shape[2]
    return torch.stack([cache[int(table_row[j // P]), :, j % P] for j in range(first, last)], 1)


def attend(q, kc, vc, table, lens, window, scale, p_err):
    """out, lse and the bound on |out error| before the final rounding; kc and
    vc in float64 (scales applied).  p_err: relative error of the
    probabilities' own format."""
    B, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        first = max(0, n - window) if window else 0
        k, v = gather(kc, table[b], first, n), gather(vc, table[b], first, n)
        for h in range(Hq):
            s = (k[h // G] * q[b, h]).sum(1) * scale
            ds = D * U32 * ((k[h // G] * q[b, h]).abs().sum(1) * abs(scale)).max()
            # a score in base 2 is rounded once more, as is exp's argument
            ds = ds + 4 * U32 * s.abs().max()
            m = s.max()
            p = (s - m).exp()
            out[b, h] = (p[:, None] * v[h // G]).sum(0) / p.sum()
            lse[b, h] = m + p.sum().log()
            spread = (p[:, None] * v[h // G].abs()).sum(0) / p.sum()
            bound[b, h] = (2 * ds + p_err + 4 * (n - first + 64) * U32) * spread
    return out, lse, bound


def unpack_w4(words, scales):
    """(E, C, R) float64 weights of packed codes and group scales."""
    w = words.long() & 0xffffffff
    code = torch.stack([(w >> (4 * (j // 2) + 16 * (j % 2))) & 15 for j in range(8)], -1)
    code = code.flatten(-2).double() - 8
    g = code.shape[-1] // scales.shape[-1]
    return code * scales.double().repeat_interleave(g, -1)


def experts(x, idx, tw, w13, w2):
    """y and the bound on its error before the final rounding; w13 (E, 2I, H)
    and w2 (E, H, I) in float64, invalid ids contribute nothing."""
    n, H = x.shape
    I = w2.shape[2]
    E = w13.shape[0]
    y = torch.zeros(n, H, dtype=torch.float64)
    bound = torch.zeros_like(y)
    for t in range(n):
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            if not 0 <= e < E:
                continue
            a = w13[e] @ x[t]
            ea = H * U32 * (w13[e].abs() @ x[t].abs())
            g, u, eg, eu = a[:I], a[I:], ea[:I], ea[I:]
            silu = g / (1 + (-g).exp())
            h = silu * u
            # |SiLU'| <= 1.1; h in two bf16 parts, exp and a division in float32
            eh = 1.1 * eg * u.abs() + silu.abs() * eu + eg * eu + (2.0 ** -16 + 2.0 ** -20) * h.abs()
            w = float(tw[t, k])
            y[t] += w * (w2[e] @ h)
            bound[t] += abs(w) * (w2[e].abs() @ eh + (I + 8) * U32 * (w2[e].abs() @ h.abs()))
    return y, bound

"""Plain float64 forms of the training operators, and how far a float32
evaluation may be from them.

u = 2^-24 is half a step of float32.  A sum of k float32 terms added in any
fixed order with chains of at most L additions is within L u sum|terms|."""
import torch

U32 = 2.0 ** -24
SLACK = 1 + 1e-3  # products of two of the small terms below


def half_step(t, dtype):
    """What one rounding to dtype may move a value of magnitude |t| by."""
    return (torch.finfo(dtype).eps / 2) * t.abs() + torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def row_chain(H):
    """Longest chain of additions of a row's sum: 32 values of a thread (rows
    longer than its CTA's registers: one value in 1024), five steps inside
    warps, twice."""
    return max(32, H // 1024 + 8) + 12


def norm(s, weight, bias, eps, rms):
    """(y, bound, mean, its bound, r, its relative bound) of rows s, all float64."""
    H = s.shape[1]
    L = row_chain(H)
    mean = torch.zeros_like(s[:, :1]) if rms else s.mean(1, keepdim=True)
    d = s - mean
    var = d.square().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    # the mean: its last rounding, and the sum of the deviations from the first one, which is
    # itself off by at most (L + 2) u mean|s|, an amount that the second pass sees and takes out
    e_mean = torch.zeros_like(mean)
    if not rms:
        first = (L + 2) * U32 * s.abs().mean(1, keepdim=True)
        e_mean = 2 * U32 * (mean.abs() + first) + (L + 3) * U32 * (d.abs().mean(1, keepdim=True) + first)
    sigma = (var + eps).sqrt()
    e_d = e_mean + U32 * d.abs()  # of a deviation
    # the squares: twice each deviation's error, their own roundings and sum; the correction off^2
    e_var = 2 * (d.abs() * e_d).mean(1, keepdim=True) + e_d.square().mean(1, keepdim=True) + (L + 4) * U32 * var
    if not rms:
        e_var = e_var + 2 * first.square() * (1 + L * U32) * U32 + 2 * U32 * var + 2 * first * e_mean
    e_r = 0.5 * e_var / sigma.square() + 4 * U32
    xh = d * r
    e_xh = xh.abs() * (2 * U32 + e_r) + e_d * r
    y = xh * weight + (0 if bias is None else bias)
    e_y = weight.abs() * e_xh + 2 * U32 * ((xh * weight).abs() + y.abs())
    return y, e_y * SLACK, mean[:, 0], e_mean[:, 0] * SLACK, r[:, 0], (e_r * SLACK)[:, 0]


def norm_backward(dy, s, mean, r, weight, ds, rms, rows_chain):
    """((dx, bound), (dweight, bound), (dbias, bound)), all float64, for given
    statistics; rows_chain: longest chain of the sums over rows."""
    H = s.shape[1]
    L = row_chain(H)
    xh = (s - mean[:, None]) * r[:, None]
    t = dy * weight
    mean_of = lambda v: v.sum(1, keepdim=True) / H  # noqa: E731
    c2 = mean_of(t * xh)
    c1 = torch.zeros_like(c2) if rms else mean_of(t)
    v = t - c1 - xh * c2
    e_xh = 2 * U32 * xh.abs()
    e_c1 = 0 if rms else (L + 4) * U32 * mean_of(t.abs())
    e_c2 = (L + 7) * U32 * mean_of((t * xh).abs())
    e_v = U32 * t.abs() + e_c1 + xh.abs() * e_c2 + c2.abs() * e_xh + 3 * U32 * (t.abs() + c1.abs() + (xh * c2).abs())
    dx = r[:, None] * v
    e_dx = r[:, None] * e_v + 2 * U32 * dx.abs()
    if ds is not None:
        dx = dx + ds
        e_dx = e_dx + U32 * dx.abs()
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw = (rows_chain + 4) * U32 * (dy * xh).abs().sum(0)
    e_db = rows_chain * U32 * dy.abs().sum(0)
    return (dx, e_dx * SLACK), (dw, e_dw * SLACK), (db, e_db * SLACK)


# ------------------------------------------------------------------- AdamW
BLOCK = 256


def blocks(x, fill=0.0):
    """A tensor's values in rows of 256, the last one filled up."""
    x = x.reshape(-1)
    pad = -x.numel() % BLOCK
    return torch.cat([x, x.new_full((pad,), fill)]).view(-1, BLOCK)


def decode(codes, scale):
    return codes.float() * scale[:, None]


def encode(x, positive):
    """Codes and scales of float32 rows of 256, operation by operation as the
    interface states it."""
    size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    scale = size.amax(1).clamp(min=2.0 ** -100) * torch.tensor(1 / 448, dtype=torch.float32)
    inv = torch.ones_like(scale) / scale
    code = x * inv[:, None]
    if positive:
        code = torch.where(x > 0, code.clamp(min=2.0 ** -9), code)
    code = torch.where(torch.isfinite(x), code.clamp(-448, 448), torch.full_like(x, float("nan")))
    return code.to(torch.float8_e4m3fn), scale


def adamw_moments(g, m, v, b1, b2):
    """m, v and sqrt(v) in float32: the gradient's terms rounded, the rest fused
    (a product of two float32 values is exact in float64)."""
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    fma = lambda a, b, c: (a.double() * b.double() + c.double()).float()  # noqa: E731
    m = fma(m, f(b1), g * f(1 - b1))
    v = fma(v, f(b2), (g * f(1 - b2)) * g)
    return m, v, v.sqrt()


def adamw_param(p, m, v, lr, wd, b1, b2, eps, t):
    """The step in float64 from the float32 moments, and its bound: four
    roundings of the decayed parameter, eight of the step."""
    p, m, v = p.double(), m.double(), v.double()
    step = lr / (1 - b1 ** t) * m / (v.sqrt() / (1 - b2 ** t) ** 0.5 + eps)
    want = p * (1 - lr * wd) - step
    return want, (4 * U32 * p.abs() + 8 * U32 * step.abs() + U32 * want.abs()) * SLACK + 1e-44

"""The training operators around the MoE layer's backward pass, as they are measured: the layer norm
before the layer and its gradients, the global norm of the gradients, and the AdamW step over all of a
model's tensors.

`run` computes each operator in plain torch operations (float32, rounded once at the end) while `own`
is false, and through the library's public calls while it is true.
"""
import math

import torch

own = False

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16}
E4M3_MAX = 448.0
BLOCK = 256  # values of a tensor that share a scale where states are held in 8 bits
BETA1, BETA2, EPS, LR = 0.9, 0.95, 1e-8, 3e-4


# ------------------------------------------------------------------ cases
def _norm(n, H, dtype, weight, rms, bias, residual):
    return dict(op="norm", n=n, H=H, dtype=dtype, weight=weight, rms=rms, bias=bias,
                residual=residual)


def _norm_backward(n, H, dtype, weight, rms, bias, residual):
    return dict(_norm(n, H, dtype, weight, rms, bias, residual), op="norm_backward")


def _adamw(layers, H, I, E, dtype, master, grad, state, clip):
    """The tensors of `layers` MoE layers: norm weight, router, and the experts' w13 and w2."""
    return dict(op="adamw", layers=layers, H=H, I=I, E=E, dtype=dtype, master=master, grad=grad,
                state=state, clip=clip)


def _grad_norm(layers, H, I, E, grad):
    return dict(op="grad_norm", layers=layers, H=H, I=I, E=E, grad=grad)


def listed():
    return [
        # serving: one new token, before the router of an OLMoE-shaped layer; latency counts
        dict(_norm(1, 2048, "bf16", "bf16", True, False, True), name="norm_one_token"),
        # training: a micro-batch of the OLMoE-shaped layer, the residual added on the way
        dict(_norm(4096, 2048, "bf16", "f32", False, True, True), name="norm_batch"),
        # float32 rows of odd length and number
        dict(_norm(1777, 1031, "f32", "f32", False, True, False), name="norm_odd_f32"),
        # the gradients of the micro-batch, the residual stream's gradient added on the way
        dict(_norm_backward(4096, 2048, "bf16", "f32", False, True, True), name="norm_backward_batch"),
        # the DeepSeek-V3-sized layer's rows
        dict(_norm_backward(8192, 7168, "bf16", "bf16", True, False, True), name="norm_backward_wide"),
        # few float32 rows of odd length
        dict(_norm_backward(301, 1031, "f32", "f32", False, True, False), name="norm_backward_odd_f32"),
        # a small model: sixteen layers of small tensors, all in float32
        dict(_adamw(16, 128, 64, 8, "f32", False, "f32", "f32", False), name="adamw_small_f32"),
        # the OLMoE-shaped layer: bf16 weights with float32 master copies, clipped float32 gradients
        dict(_adamw(1, 2048, 1024, 64, "bf16", True, "f32", "f32", True), name="adamw_layer_f32"),
        # odd sizes, 8-bit states, bf16 throughout
        dict(_adamw(5, 515, 129, 7, "bf16", False, "bf16", "e4m3", False), name="adamw_odd_e4m3"),
        # the OLMoE-shaped layer with 8-bit states
        dict(_adamw(1, 2048, 1024, 64, "bf16", True, "f32", "e4m3", True), name="adamw_layer_e4m3"),
        # the gradients of the small model
        dict(_grad_norm(16, 128, 64, 8, "f32"), name="grad_norm_small"),
        # the gradients of the OLMoE-shaped layer
        dict(_grad_norm(1, 2048, 1024, 64, "f32"), name="grad_norm_layer"),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    while True:
        op = rng.choice(["norm", "norm_backward", "adamw", "grad_norm"])
        if op in ("norm", "norm_backward"):
            dtype = rng.choice(["bf16", "bf16", "f32"])
            H = _log(rng, 8, 16384)
            if rng.random() < 0.6:  # hidden sizes are mostly round
                H = max(8, H // 64 * 64) if H >= 64 else max(8, H // 8 * 8)
            rms = rng.random() < 0.5
            c = dict(_norm(_log(rng, 1, 16384), H, dtype, rng.choice(["f32", dtype]), rms,
                           not rms and rng.random() < 0.8, rng.random() < 0.5), op=op)
        else:
            H, I, E = _log(rng, 16, 2048), _log(rng, 8, 1024), _log(rng, 1, 64)
            if rng.random() < 0.5:
                H, I = max(16, H // 16 * 16), max(8, I // 8 * 8)
            layers, grad = rng.randint(1, 15), rng.choice(["f32", "f32", "bf16"])
            if op == "adamw":
                dtype = rng.choice(["f32", "bf16", "bf16"])
                c = _adamw(layers, H, I, E, dtype, dtype == "bf16" and rng.random() < 0.6, grad,
                           rng.choice(["f32", "e4m3"]), rng.random() < 0.5)
            else:
                c = _grad_norm(layers, H, I, E, grad)
        if work(c)["bytes"] <= most[op]:
            return c


def _sizes(c):
    H, I, E = c["H"], c["I"], c["E"]
    return [H, H * E, E * H * 2 * I, E * I * H] * c["layers"]


def _bytes(kind):
    return {"f32": 4, "bf16": 2}[kind]


def work(c):
    if c["op"] in ("norm", "norm_backward"):
        n, H, e = c["n"], c["H"], _bytes(c["dtype"])
        vectors = H * _bytes(c["weight"]) * (1 + c["bias"])
        if c["op"] == "norm":  # x, residual; s, y; the statistics
            return {"bytes": n * H * e * (2 + 2 * c["residual"]) + vectors + 8 * n,
                    "flops": 8.0 * n * H}
        return {"bytes": n * H * e * (3 + c["residual"]) + H * _bytes(c["weight"]) + 8 * n
                + 4 * H * (1 + c["bias"]), "flops": 14.0 * n * H}
    values = sum(_sizes(c))
    if c["op"] == "grad_norm":
        return {"bytes": values * _bytes(c["grad"]), "flops": 2.0 * values}
    param = 8 + _bytes(c["dtype"]) if c["master"] else 2 * _bytes(c["dtype"])
    states = 16.0 if c["state"] == "f32" else 4.0 + 16.0 / BLOCK
    return {"bytes": values * (param + _bytes(c["grad"]) + states), "flops": 15.0 * values}


# ---------------------------------------------------------------- inputs
def _randn(g, shape, std=1.0, dtype=F32):
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _quantised(x):
    """e4m3 codes (blocks, 256) and scales (blocks,) of non-negative or signed values."""
    scale = x.abs().amax(1) * (1.0 / E4M3_MAX)
    code = (x * torch.where(scale > 0, 1.0 / scale, 0.0)[:, None]).clamp_(-E4M3_MAX, E4M3_MAX)
    return code.to(E4M3), scale


def _blocks(c):
    """Where each tensor lies in one buffer of whole blocks: its first block, and how many there are."""
    first, total = [], 0
    for n in _sizes(c):
        first.append(total)
        total += -(-n // BLOCK)
    return first, total


def _views(c, flat):
    """The case's tensors, each the start of its blocks in the buffer."""
    first, _ = _blocks(c)
    line = flat.view(-1)
    return [line[b * BLOCK:b * BLOCK + n] for b, n in zip(first, _sizes(c))]


def _filled(c, total, dtype, make):
    """A buffer of blocks; what lies behind the end of a tensor is zero."""
    flat = torch.zeros((total, BLOCK), device="cuda", dtype=dtype)
    made = make((total, BLOCK)).to(dtype)
    for to, value in zip(_views(c, flat), _views(c, made)):
        to.copy_(value)
    return flat


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s = {"case": c}
    if c["op"] in ("norm", "norm_backward"):
        return _prepare_norm(c, s, g)
    _, total = _blocks(c)
    # gradients of very unequal size from tensor part to tensor part; an expert that no token chose has none
    size = torch.empty((total, 1), device="cuda").uniform_(-5.0, -2.0, generator=g)
    size = torch.where(torch.rand((total, 1), device="cuda", generator=g) < 0.03, 0.0, 10.0 ** size)
    s["grad"] = _filled(c, total, TYPES[c["grad"]], lambda sh: _randn(g, sh) * size)
    if c["op"] == "grad_norm":
        s["max_norm"] = 1.0
        s["norm"], s["factor"] = (torch.empty(1, device="cuda") for _ in range(2))
        if own:
            import top_routing_dispatch_gb300 as M
            s["norm_of"] = M.GradNorm(_views(c, s["grad"]))
        return s
    kept = size * (torch.rand((total, 1), device="cuda", generator=g) < 0.97)  # some have never had any
    s["param"] = _filled(c, total, TYPES[c["dtype"]], lambda sh: _randn(g, sh, 0.02))
    s["master"] = None
    if c["master"]:
        s["master"] = _filled(c, total, F32, lambda sh: s["param"].float() * (1.0 + _randn(g, sh, 2.0 ** -11)))
    m = _filled(c, total, F32, lambda sh: _randn(g, sh) * kept * 0.3)
    r = _filled(c, total, F32, lambda sh: (1.0 + _randn(g, sh, 0.2)).abs_() * kept)
    s["steps"] = 700  # taken before this one
    s["m_scale"] = s["v_scale"] = None
    if c["state"] == "f32":
        s["m"], s["v"] = m, r.square_()
    else:
        (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _quantised(m), _quantised(r)
    decay = [0.0, 0.1, 0.1, 0.1] * c["layers"]  # norm weights do not decay
    s["decay"] = torch.repeat_interleave(
        torch.tensor(decay, device="cuda"),
        torch.tensor([-(-n // BLOCK) for n in _sizes(c)], device="cuda"))[:, None]
    s["grad_scale"] = torch.empty(1, device="cuda").uniform_(0.2, 1.0, generator=g) if c["clip"] else None
    if own:
        import top_routing_dispatch_gb300 as M
        s["optimizer"] = M.AdamW(
            _views(c, s["param"]), _views(c, s["grad"]), lr=LR, betas=(BETA1, BETA2), eps=EPS,
            weight_decay=decay, state=F32 if c["state"] == "f32" else E4M3,
            masters=_views(c, s["master"]) if c["master"] else None)
        s["optimizer"].load_state_dict({"steps": s["steps"], "m": s["m"], "v": s["v"],
                                        "m_scale": s["m_scale"], "v_scale": s["v_scale"]})
        for name in ("m", "v", "m_scale", "v_scale"):
            s[name] = getattr(s["optimizer"], name)  # the optimizer holds the states
    return s


def _prepare_norm(c, s, g):
    n, H, T, W = c["n"], c["H"], TYPES[c["dtype"]], TYPES[c["weight"]]
    # rows of unequal size around a mean of their own, as a residual stream has them
    rows = torch.empty((n, 1), device="cuda").uniform_(0.5, 3.0, generator=g)
    s["x"] = (_randn(g, (n, H)) * rows + _randn(g, (n, 1), 0.5)).to(T)
    s["weight"] = (1.0 + _randn(g, (H,), 0.2)).to(W)
    s["bias"] = _randn(g, (H,), 0.1).to(W) if c["bias"] else None
    s["eps"] = 1e-6 if c["rms"] else 1e-5
    s["stats"] = torch.empty((2, n), device="cuda")
    if c["op"] == "norm":
        s["residual"] = _randn(g, (n, H), 1.0, T) if c["residual"] else None
        s["y"], s["s"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    else:
        x = s["x"].double()
        mean = torch.zeros((n, 1), device="cuda", dtype=torch.float64) if c["rms"] else x.mean(1, keepdim=True)
        s["stats"][0], s["stats"][1] = mean[:, 0], torch.rsqrt((x - mean).square().mean(1) + s["eps"])
        s["dy"] = _randn(g, (n, H), 1.0, T)
        s["ds"] = _randn(g, (n, H), 1.0, T) if c["residual"] else None
        s["dx"] = torch.empty_like(s["x"])
        s["dweight"] = torch.empty(H, device="cuda")
        s["dbias"] = torch.empty(H, device="cuda") if c["bias"] else None
    if own:
        import top_routing_dispatch_gb300 as M
        s["norm"] = M.LayerNorm(s["weight"], s["bias"], eps=s["eps"], rms=c["rms"], dtype=T)
    return s


# ------------------------------------------------------------ the passes
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "adamw": _plain_adamw,
                "grad_norm": _plain_grad_norm}[op](s)
    if op == "norm":
        s["norm"](s["x"], s["residual"], y=s["y"], s=s["s"] if s["residual"] is not None else None,
                  stats=s["stats"])
        return _norm_outputs(s)
    if op == "norm_backward":
        s["norm"].backward(s["dy"], s["x"], s["stats"], ds=s["ds"], dx=s["dx"],
                           dweight=s["dweight"], dbias=s["dbias"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "adamw":
        s["optimizer"].step(grad_scale=s["grad_scale"])
        return _adamw_outputs(s)
    s["norm_of"](s["max_norm"], norm=s["norm"], factor=s["factor"])
    return {"norm": s["norm"], "factor": s["factor"]}


def _norm_outputs(s):
    return {"y": s["y"], "s": s["s"] if s["residual"] is not None else None,
            "mean": None if s["case"]["rms"] else s["stats"][0], "rstd": s["stats"][1]}


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale")}


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    if s["residual"] is not None:
        s["s"] = (x + s["residual"].float()).to(s["x"].dtype)
        x = s["s"].float()
    mean = torch.zeros((), device="cuda") if c["rms"] else x.sum(1, keepdim=True) / c["H"]
    x = x - mean
    r = torch.rsqrt((x * x).sum(1, keepdim=True) / c["H"] + s["eps"])
    y = x * r * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["y"] = y.to(s["x"].dtype)
    s["stats"] = torch.stack([mean.expand(c["n"], 1)[:, 0], r[:, 0]])
    return _norm_outputs(s)


def _plain_norm_backward(s):
    c, dy = s["case"], s["dy"].float()
    mean, r = s["stats"][0][:, None], s["stats"][1][:, None]
    xh = (s["x"].float() - mean) * r
    t = dy * s["weight"].float()
    dx = t - xh * ((t * xh).sum(1, keepdim=True) / c["H"])
    if not c["rms"]:
        dx = dx - t.sum(1, keepdim=True) / c["H"]
    dx = dx * r
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xh).sum(0),
            "dbias": dy.sum(0) if c["bias"] else None}


def _stored(x, positive):
    """Values as 8-bit codes with a scale per block: rounded to nearest; a positive value whose
    nearest code is zero keeps the smallest one where `positive` says so."""
    scale = x.abs().amax(1).clamp_(min=2.0 ** -100) * (1.0 / E4M3_MAX)
    code = x * torch.reciprocal(scale)[:, None]
    if positive:
        code = torch.where(x > 0, code.clamp(min=2.0 ** -9), code)
    return code.clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def _plain_adamw(s):
    c = s["case"]
    s["steps"] += 1
    t = s["steps"]
    g = s["grad"].float()
    if s["grad_scale"] is not None:
        g = g * s["grad_scale"]
    m, v = s["m"].float(), s["v"].float()
    if c["state"] == "e4m3":
        m = m * s["m_scale"][:, None]
        v = v * s["v_scale"][:, None]  # the root of the second moment is held
        v = v * v
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    root = torch.sqrt(v)
    p = (s["param"] if s["master"] is None else s["master"]).float()
    step = m / (root * (1.0 / math.sqrt(1.0 - BETA2 ** t)) + EPS)
    p = p * (1.0 - LR * s["decay"]) - step * (LR / (1.0 - BETA1 ** t))
    if s["master"] is not None:
        s["master"].copy_(p)
    s["param"].copy_(p)
    if c["state"] == "f32":
        s["m"], s["v"] = m, v
    else:
        (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _stored(m, False), _stored(root, True)
    return _adamw_outputs(s)


def _plain_grad_norm(s):
    norm = s["grad"].float().square().sum(dtype=torch.float64).sqrt().float().view(1)
    return {"norm": norm, "factor": (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)}


# ------------------------------------------------------- the definition
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "adamw": _exact_adamw,
                "grad_norm": _exact_grad_norm}[case["op"]](s)


def _exact_norm(s):
    c, x = s["case"], s["x"].double()
    total = None
    if s["residual"] is not None:
        total = x + s["residual"].double()
        x = total.to(s["x"].dtype).double()  # the rows that are normalised are the stored ones
    mean = x.mean(1) if not c["rms"] else torch.zeros_like(x[:, 0])
    rstd = (torch.var(x, 1, correction=0) if not c["rms"] else x.pow(2).mean(1)).add(s["eps"]).pow(-0.5)
    y = torch.addcmul(torch.zeros_like(x), (x - mean[:, None]) * rstd[:, None], s["weight"].double())
    if s["bias"] is not None:
        y += s["bias"].double()
    return {"y": y, "s": total, "mean": None if c["rms"] else mean, "rstd": rstd}


def _exact_norm_backward(s):
    c = s["case"]
    # the projection form: dx = r P t, P taking out the row's constant and its own direction
    z = (s["x"].double() - s["stats"][0].double()[:, None]) * s["stats"][1].double()[:, None]
    dy = s["dy"].double()
    t = dy * s["weight"].double()
    along = torch.einsum("nh,nh->n", t, z) / c["H"]
    dx = t - along[:, None] * z
    if not c["rms"]:
        dx -= t.mean(1, keepdim=True)
    dx *= s["stats"][1].double()[:, None]
    if s["ds"] is not None:
        dx += s["ds"].double()
    return {"dx": dx, "dweight": torch.einsum("nh,nh->h", dy, z),
            "dbias": torch.einsum("nh->h", dy) if c["bias"] else None}


def _exact_adamw(s):
    c, t = s["case"], s["steps"] + 1
    out = dict.fromkeys(("param", "master", "m", "v", "m_scale", "v_scale"))
    p0 = s["param"] if s["master"] is None else s["master"]
    out["param"] = torch.empty(p0.shape, device="cuda", dtype=torch.float64)
    held = {k: torch.empty_like(out["param"]) for k in ("m", "v")}
    step = 1 << 18  # blocks at a time
    for a in range(0, p0.shape[0], step):
        at = slice(a, a + step)
        g = s["grad"][at].double() * (1.0 if s["grad_scale"] is None else s["grad_scale"].double())
        m, v = s["m"][at].double(), s["v"][at].double()
        if c["state"] == "e4m3":
            m, v = m * s["m_scale"][at].double()[:, None], (v * s["v_scale"][at].double()[:, None]) ** 2
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g ** 2 - v)
        up = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        out["param"][at] = p0[at].double() - LR * (up + s["decay"][at].double() * p0[at].double())
        held["m"][at], held["v"][at] = m, v
    if s["master"] is not None:
        out["master"] = out["param"]
    if c["state"] == "f32":
        out.update(held)
    else:  # the codes' values before their rounding
        held["v"].sqrt_()
        for k in held:
            scale = held[k].abs().amax(1).clamp(min=2.0 ** -100) / E4M3_MAX
            out[k], out[k + "_scale"] = held[k] / scale[:, None], scale
    return out


def _exact_grad_norm(s):
    norm = torch.linalg.vector_norm(s["grad"].double().view(-1)).view(1)
    return {"norm": norm, "factor": (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)}

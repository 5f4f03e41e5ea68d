"""The serving operators around the MoE layer, as they are measured: appending to a paged key-value
cache, attention of one new token per sequence over that cache, and the routed experts on 4-bit
weights for few tokens.

`run` computes each operator in plain torch operations (float32, rounded once at the end) while
`own` is false, and through the library's public calls while it is true.
"""
import math

import torch

own = False

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
CACHE = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _append(tokens, seqs, heads, dim, page, cache, rope, interleaved, context):
    return dict(op="append", tokens=tokens, seqs=seqs, q_heads=heads[0], kv_heads=heads[1],
                head_dim=dim, page=page, cache=cache, rope=rope, interleaved=interleaved,
                context=context)


def _attend(seqs, idle, shortest, longest, heads, dim, page, cache, window=0):
    return dict(op="attend", seqs=seqs, idle=idle, shortest=shortest, longest=longest,
                q_heads=heads[0], kv_heads=heads[1], head_dim=dim, page=page, cache=cache,
                window=window)


def _experts(tokens, H, I, E, K, group):
    return dict(op="experts", tokens=tokens, H=H, I=I, E=E, K=K, group=group)


def listed():
    return [
        # one user, one token: the step's latency
        dict(_append(1, 1, (16, 16), 128, 16, "bf16", 128, False, 1000), name="append_one_token"),
        # a decode batch of odd size over an 8-bit cache, partly rotated heads, interleaved pairs
        dict(_append(61, 61, (32, 8), 128, 64, "e4m3", 64, True, 900), name="append_batch_e4m3"),
        # a prefill chunk: a few prompts of unequal lengths written at once (H = 2048 heads)
        dict(_append(8191, 5, (16, 16), 128, 64, "bf16", 128, False, 700), name="append_prefill"),
        # one short conversation
        dict(_attend(1, 0, 137, 137, (16, 16), 128, 16, "bf16"), name="attend_one_short"),
        # a serving batch of very unequal conversations with two idle rows, a head for each query head
        dict(_attend(64, 2, 17, 8191, (16, 16), 128, 64, "bf16"), name="attend_batch_ragged"),
        # one long document, eight query heads on each cached head
        dict(_attend(1, 0, 131071, 131071, (32, 4), 128, 128, "bf16"), name="attend_one_long"),
        # a large batch on shared heads over an 8-bit cache
        dict(_attend(128, 0, 500, 12001, (64, 8), 128, 32, "e4m3"), name="attend_batch_e4m3"),
        # the float32 layer type, small heads, sliding window
        dict(_attend(12, 1, 30, 5000, (12, 4), 64, 16, "f32", 2000), name="attend_window_f32"),
        # one token through the OLMoE-shaped layer
        dict(_experts(1, 2048, 1024, 64, 8, 128), name="experts_one_token"),
        # a decode batch through the OLMoE-shaped layer: every expert hit, about 15 rows each
        dict(_experts(120, 2048, 1024, 64, 8, 64), name="experts_batch"),
        # few tokens through the DeepSeek-V3-sized layer
        dict(_experts(3, 7168, 2048, 256, 8, 128), name="experts_wide_few"),
        # a decode batch through the DeepSeek-V3-sized layer
        dict(_experts(61, 7168, 2048, 256, 8, 32), name="experts_wide_batch"),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; no dimension of 3072."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if v != 3072:
            return min(max(v, lo), hi)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    while True:
        op = rng.choice(["append", "attend", "experts"])
        if op == "experts":
            E = _log(rng, 4, 256)
            H, I = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 16)
            c = _experts(_log(rng, 1, 128), H, I, E, rng.randint(1, min(8, E)),
                         rng.choice([32, 64, 128]))
            if 3072 in (H, I, 2 * I):
                continue
        else:
            dim = rng.choice([64, 128, 128, 256])
            kv = rng.choice([1, 2, 3, 4, 8, 16])
            heads = (kv * rng.choice([1, 2, 3, 4, 7, 8, 12, 16]), kv)
            cache = rng.choice(["bf16", "bf16", "e4m3", "f32"])
            page = rng.choice([16, 32, 48, 64, 128])
            if heads[0] > 128 or (heads[0] + 2 * kv) * dim == 3072 or heads[0] * dim == 3072:
                continue
            if op == "append":
                seqs = _log(rng, 1, 200)
                tokens = seqs if rng.random() < 0.5 else _log(rng, seqs, 8191)
                rope = rng.choice([0, dim // 2, dim, dim])
                c = _append(tokens, seqs, heads, dim, page, cache, rope, rng.random() < 0.5,
                            _log(rng, 1, 2000))
            else:
                longest = _log(rng, 1, 131071)
                seqs = _log(rng, 1, 200)
                window = 0 if rng.random() < 0.7 else _log(rng, 1, longest)
                c = _attend(seqs, rng.randint(0, seqs // 8), _log(rng, 1, longest), longest, heads,
                            dim, page, cache, window)
                # the plain form lays the cache out for the longest sequence of the batch
                if seqs * longest * kv * dim > 2_000_000_000:
                    continue
        if work(c)["bytes"] <= most[op]:
            return c


def _lengths(c):
    """The lengths of an attention case: spread over the logarithm of its range; idle rows have none."""
    live = c["seqs"] - c["idle"]
    a, b = math.log(c["shortest"]), math.log(c["longest"])
    got = [int(round(math.exp(a + (b - a) * i / max(1, live - 1)))) for i in range(live)]
    got[-1] = c["longest"]
    return got + [0] * c["idle"]


def _shares(c):
    """New tokens of each sequence of an append case, unequal, in a fixed order."""
    n, s = c["tokens"], c["seqs"]
    if n == s:
        return [1] * s
    w = [1.0 + (i * 7 % 5) for i in range(s)]
    cum, tot, acc = [0], sum(w), 0.0
    for x in w:
        acc += x
        cum.append(int(round(n * acc / tot)))
    return [b - a for a, b in zip(cum, cum[1:])]


def work(c):
    if c["op"] == "experts":
        n, H, I, E, K, g = (c[k] for k in ("tokens", "H", "I", "E", "K", "group"))
        hit = E * (1.0 - (1.0 - K / E) ** n)  # distinct experts of n tokens with K of E each
        return {"bytes": hit * 3 * H * I * (0.5 + 2.0 / g) + 4 * n * H + 8 * n * K,
                "flops": 6.0 * n * K * H * I}
    Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    elem = {"f32": 4, "bf16": 2, "e4m3": 1}[c["cache"]]
    act = 4 if c["cache"] == "f32" else 2
    if c["op"] == "append":
        n = c["tokens"]
        return {"bytes": n * ((2 * Hq + 2 * Hkv) * D * act + 2 * Hkv * D * elem + 4 * c["rope"] + 8),
                "flops": 3.0 * n * (Hq + Hkv) * c["rope"]}
    seen = sum(min(l, c["window"]) if c["window"] else l for l in _lengths(c))
    return {"bytes": seen * (2 * Hkv * D * elem + 4.0 / c["page"]) + 2 * c["seqs"] * Hq * D * act,
            "flops": 4.0 * seen * Hq * D}


# ---------------------------------------------------------------- inputs
def _randn(g, shape, std=1.0, dtype=F32):
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _rope_table(rows, dim):
    """(rows, dim) float32: the cosines, then the sines, of each position's dim/2 angles."""
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pages(c, lens, g):
    """A page table whose pages lie anywhere in the pool; entries past a sequence's end are -1."""
    P, B = c["page"], c["seqs"]
    need = [-(-l // P) for l in lens]
    cols, pool = max(1, max(need)), sum(need) + 3
    ids = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    col = torch.arange(cols, device="cuda")
    n = torch.tensor(need, device="cuda")
    first = n.cumsum(0) - n
    table = torch.where(col < n[:, None], ids[(first[:, None] + col).clamp(max=pool - 1)], -1)
    return table.to(torch.int32).contiguous(), pool


def _cache(c, pool, g):
    shape = (pool, c["kv_heads"], c["page"], c["head_dim"])
    dt = CACHE[c["cache"]]
    if dt != E4M3:
        return _randn(g, shape, 1.0, dt), _randn(g, shape, 1.0, dt), None, None
    ks, vs = (torch.empty(c["kv_heads"], device="cuda").uniform_(0.008, 0.012, generator=g)
              for _ in range(2))
    make = lambda s: (_randn(g, shape) / s[:, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)  # noqa: E731
    return make(ks), make(vs), ks, vs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    s = {"case": c}
    if c["op"] == "experts":
        n, H, I, E, K, gr = (c[k] for k in ("tokens", "H", "I", "E", "K", "group"))
        s["x"] = _randn(g, (n, H), 1.0, BF16)
        p = torch.softmax(_randn(g, (n, E)), 1)
        w, idx = p.topk(K, dim=1)
        s["topk_w"], s["topk_idx"] = w.contiguous(), idx.to(torch.int32).contiguous()
        for name, rows, red in (("w13", 2 * I, H), ("w2", H, I)):
            s[name + "_q"] = torch.randint(-2 ** 31, 2 ** 31, (E, rows, red // 8), device="cuda",
                                           generator=g, dtype=torch.int32)
            mid = 1.0 / (4.6 * math.sqrt(red))  # codes spread evenly over -8..7 have a deviation of 4.6
            s[name + "_s"] = torch.empty((E, rows, red // gr), device="cuda").uniform_(
                0.5 * mid, 1.5 * mid, generator=g).to(BF16)
        s["y"] = torch.empty((n, H), device="cuda", dtype=BF16)
        if own:
            import top_routing_dispatch_gb300 as M
            s["experts"] = M.W4Experts(s["w13_q"], s["w13_s"], s["w2_q"], s["w2_s"], K=K,
                                       max_tokens=n)
        return s
    B, Hq, Hkv, D = c["seqs"], c["q_heads"], c["kv_heads"], c["head_dim"]
    act = F32 if c["cache"] == "f32" else BF16
    extra = {}
    if c["op"] == "append":
        new = torch.tensor(_shares(c))
        had = [(c["context"] * (3 + 5 * i % 7)) // 9 for i in range(B)]
        lens = [h + int(k) for h, k in zip(had, new)]
        s["seq_ids"] = torch.repeat_interleave(torch.arange(B), new).to("cuda", torch.int32)
        s["positions"] = torch.cat([torch.arange(h, l) for h, l in zip(had, lens)]).to("cuda", torch.int32)
        # the projections' one output buffer: a row holds q, k and v of a token
        qkv = _randn(g, (c["tokens"], (Hq + 2 * Hkv) * D), 1.0, act)
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split(
            [Hq * D, Hkv * D, Hkv * D], 1))
        s["q_out"] = torch.empty((c["tokens"], Hq, D), device="cuda", dtype=act)
        if c["rope"]:
            s["rope"] = _rope_table(max(lens) + 1, c["rope"])
            extra = dict(rope=s["rope"], rope_interleaved=c["interleaved"])
    else:
        at = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
        some = _lengths(c)
        lens = [some[i] for i in at]
        s["seq_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["q"] = _randn(g, (B, Hq, D), 2.0, act)
        s["out"] = torch.empty((B, Hq, D), device="cuda", dtype=act)
    s["page_table"], pool = _pages(c, lens, g)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(c, pool, g)
    if own:
        import top_routing_dispatch_gb300 as M
        s["cache"] = M.PagedKVCache(s["k_cache"], s["v_cache"], s["page_table"], q_heads=Hq,
                                    k_scale=s["k_scale"], v_scale=s["v_scale"], **extra)
    return s


# ------------------------------------------------------------ the passes
def run(s):
    c = s["case"]
    if own:
        if c["op"] == "append":
            q = s["cache"].append(s["q"], s["k"], s["v"], s["seq_ids"], s["positions"],
                                  q_out=s["q_out"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if c["op"] == "attend":
            return s["cache"].attend(s["q"], s["seq_lens"], out=s["out"], window=c["window"])
        return s["experts"](s["x"], s["topk_idx"], s["topk_w"], y=s["y"])
    return {"append": _plain_append, "attend": _plain_attend, "experts": _plain_experts}[c["op"]](s)


def _rotate(x, rope, positions, interleaved):
    """x (n, heads, D) in float32 with its first rope.shape[1] dimensions rotated by position."""
    half = rope.shape[1] // 2
    row = rope[positions.long()][:, None, :]
    cos, sin = row[..., :half], row[..., half:]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _plain_append(s):
    c, P = s["case"], s["case"]["page"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["rope"]:
        q = _rotate(q, s["rope"], s["positions"], c["interleaved"])
        k = _rotate(k, s["rope"], s["positions"], c["interleaved"])
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    pos = s["positions"].long()
    page, slot = s["page_table"][s["seq_ids"].long(), pos // P].long(), pos % P
    for name, x in (("k_cache", k), ("v_cache", v)):
        cache, x = s[name], x.to(s[name].dtype)
        if cache.dtype == E4M3:  # the bits move; torch need not know the type
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[page, :, slot] = x
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D = c["seqs"], c["q_heads"], c["kv_heads"], c["head_dim"]
    table = s["page_table"].clamp(min=0).long()

    def rows(cache, scale):  # (B, Hkv, longest, D) float32
        t = cache.view(torch.uint8)[table].view(E4M3) if cache.dtype == E4M3 else cache[table]
        t = t.float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
        return t if scale is None else t.mul_(scale[:, None, None])

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, rows(s["k_cache"], s["k_scale"]).transpose(2, 3)) / math.sqrt(D)
    j, n = torch.arange(x.shape[-1], device="cuda"), s["seq_lens"].long()[:, None]
    seen = j < n
    if c["window"]:
        seen &= j >= n - c["window"]
    x = x.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(n[:, :, None, None] > 0, top, 0.0)).exp_()
    o = torch.matmul(p, rows(s["v_cache"], s["v_scale"]))
    o = torch.where(n[:, :, None, None] > 0, o / p.sum(-1, keepdim=True), 0.0)
    return o.reshape(B, Hq, D).to(s["q"].dtype)


_SHIFT = (0, 16, 4, 20, 8, 24, 12, 28)  # where the eight codes of a word lie


def _dequantised(words, scales):
    """(..., rows, reduction) float32 of packed codes (..., rows, reduction / 8) and group scales."""
    sh = torch.tensor(_SHIFT, device="cuda", dtype=torch.int32)
    q = (words[..., None] >> sh).bitwise_and_(15).sub_(8).float()
    q = q.view(*scales.shape, -1).mul_(scales.float()[..., None])
    return q.flatten(-2).view(*words.shape[:-1], -1)


def _plain_experts(s):
    c, x, idx = s["case"], s["x"].float(), s["topk_idx"].long()
    n, I, E, K = c["tokens"], c["I"], c["E"], c["K"]
    few = n * K <= E  # the chosen experts' weights, else every expert's on every token
    pick = (lambda t: t[idx.reshape(-1)]) if few else (lambda t: t)
    rows = x.repeat_interleave(K, 0)[:, None] if few else x[None].expand(E, -1, -1)
    g, u = torch.matmul(rows, _dequantised(pick(s["w13_q"]), pick(s["w13_s"])).transpose(1, 2)).split(I, 2)
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.matmul(h, _dequantised(pick(s["w2_q"]), pick(s["w2_s"])).transpose(1, 2))
    if few:
        y = (y.view(n, K, -1) * s["topk_w"][..., None]).sum(1)
    else:
        w = torch.zeros((n, E), device="cuda").scatter_add_(1, idx, s["topk_w"])
        y = (y * w.t()[..., None]).sum(0)
    return y.to(BF16)


# ------------------------------------------------------- the definition
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _exact_append, "attend": _exact_attend, "experts": _exact_experts}[case["op"]](s)


def _exact_append(s):
    c, P, R = s["case"], s["case"]["page"], s["case"]["rope"]
    pos = s["positions"].long()
    out = []
    for x in (s["q"], s["k"]):
        x = x.double().clone()
        if R:
            i = torch.arange(R // 2, device="cuda")
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
            # as a product with a unit complex number, at the table's own values
            t = s["rope"].double()[pos]
            z = torch.complex(x[..., a], x[..., b]) * torch.complex(t[:, :R // 2], t[:, R // 2:])[:, None]
            x[..., a], x[..., b] = z.real, z.imag
        out.append(x)
    v = s["v"].double()
    k = out[1]
    if s["k_scale"] is not None:
        k = (k / s["k_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    page = s["page_table"].long()[s["seq_ids"].long(), pos // P]
    caches = []
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        flat = cache.double().transpose(1, 2).reshape(-1, c["kv_heads"], c["head_dim"])
        flat[page * P + pos % P] = x
        caches.append(flat.view(-1, P, c["kv_heads"], c["head_dim"]).transpose(1, 2).contiguous())
    return {"q": out[0], "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attend(s):
    c = s["case"]
    G, P, D = c["q_heads"] // c["kv_heads"], c["page"], c["head_dim"]
    out = torch.zeros((c["seqs"], c["q_heads"], D), device="cuda", dtype=torch.float64)
    for b, n in enumerate(s["seq_lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        ids = s["page_table"][b, :-(-n // P)].long()

        def rows(cache, scale):
            t = cache.view(torch.uint8)[ids].view(E4M3) if cache.dtype == E4M3 else cache[ids]
            t = t.transpose(1, 2).reshape(-1, c["kv_heads"], D)[first:n].double()
            return t if scale is None else t * scale.double()[:, None]

        k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
        for h in range(c["kv_heads"]):
            x = s["q"][b, h * G:(h + 1) * G].double() @ k[:, h].t() * D ** -0.5
            out[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v[:, h]
    return out


def _exact_experts(s):
    c, gr = s["case"], s["case"]["group"]
    x, w, idx = s["x"].double(), s["topk_w"].double(), s["topk_idx"].long()
    y = torch.zeros_like(x)

    def weight(name, e):
        words = s[name + "_q"][e].long() & 0xffffffff
        code = torch.stack([words >> sh & 15 for sh in _SHIFT], -1).flatten(1)
        return (code - 8).double() * s[name + "_s"][e].double().repeat_interleave(gr, 1)

    for e in sorted(set(idx.flatten().tolist())):
        t, k = (idx == e).nonzero(as_tuple=True)
        g, u = (x[t] @ weight("w13", e).t()).chunk(2, 1)
        y.index_add_(0, t, (g * torch.sigmoid(g) * u) @ weight("w2", e).t() * w[t, k][:, None])
    return y

"""The serving operators on the GPU against their plain float64 forms: paged
cache append, paged attention, experts on 4-bit weights."""
import math

import pytest
import torch

from tests import decode_reference as R

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
CACHES = {"f32": (F32, F32), "bf16": (BF16, BF16), "e4m3": (BF16, E4M3)}


def M():
    import top_routing_dispatch_gb300 as m
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def f64(t):
    return t.detach().float().cpu().double()


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def scaled(cache, scale):
    x = f64(cache)
    return x if scale is None else x * scale.cpu().double()[None, :, None, None]


def make_cache(kind, pages, Hkv, P, D, seed, gap=0):
    """k and v caches (with `gap` unused heads' worth of values between pages)."""
    dt = CACHES[kind][1]
    g = gen(seed)

    def one():
        x = torch.randn((pages, Hkv + gap, P, D), generator=g)
        return (x / 0.01).clamp(-448, 448).to(dt).cuda() if dt == E4M3 else x.to(dt).cuda()
    sc = [None, None]
    if dt == E4M3:
        sc = [(0.008 + 0.004 * torch.rand(Hkv, generator=g)).cuda() for _ in range(2)]
    return one()[:, :Hkv], one()[:, :Hkv], sc[0], sc[1]


def make_table(lens, P, extra_pages, seed, cols=None):
    need = [-(-n // P) for n in lens]
    cols = max(1, max(need)) if cols is None else cols
    ids = torch.randperm(sum(need) + extra_pages, generator=gen(seed))
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = ids[at:at + k].int()
        at += k
    return table.cuda(), sum(need) + extra_pages


# ---------------------------------------------------------------- append
APPEND = [
    # kind, Hq, Hkv, D, P, rope, interleaved, (tokens per sequence)
    ("bf16", 16, 16, 128, 16, 128, False, (1,)),
    ("bf16", 8, 2, 64, 16, 32, True, (1, 1, 1, 1, 1)),
    ("bf16", 5, 1, 256, 48, 256, False, (33, 1, 0, 17)),
    ("bf16", 3, 3, 128, 32, 64, False, (70, 3)),
    ("e4m3", 8, 4, 128, 32, 64, True, (2, 31, 1)),
    ("e4m3", 4, 4, 64, 16, 64, False, (9, 9)),
    ("e4m3", 2, 1, 256, 64, 0, False, (130,)),
    ("f32", 6, 2, 64, 16, 64, False, (5, 1, 40)),
    ("f32", 2, 2, 256, 16, 16, True, (18,)),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("fused", [True, False])
def test_append(case, fused):
    kind, Hq, Hkv, D, P, rd, inter, shares = case
    m = M()
    act, store = CACHES[kind]
    had = [(7 * i + 5) % 29 for i in range(len(shares))]
    lens = [h + n for h, n in zip(had, shares)]
    table, pages = make_table(lens, P, 2, 3)
    kc, vc, ks, vs = make_cache(kind, pages, Hkv, P, D, 4, gap=1)
    rope = m.rope_table(max(lens) + 1, rd) if rd else None
    cache = m.PagedKVCache(kc, vc, table, Hq, k_scale=ks, v_scale=vs, rope=rope,
                           rope_interleaved=inter)
    n = sum(shares)
    g = gen(5)
    if fused:  # views of one row per token, with a tail that belongs to neither
        qkv = torch.randn((n, (Hq + 2 * Hkv) * D + 16), generator=g).to(act).cuda()
        q, k, v = (qkv[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in (
            (0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    else:
        q, k, v = (torch.randn((n, h, D), generator=g).to(act).cuda() for h in (Hq, Hkv, Hkv))
    seq = torch.cat([torch.full((c,), i) for i, c in enumerate(shares)]).int().cuda()
    pos = torch.cat([torch.arange(h, e) for h, e in zip(had, lens)]).int().cuda()
    k0, v0 = kc.clone(), vc.clone()
    got_q = cache.append(q, k, v, seq, pos)
    cache.check()
    p = pos.tolist()
    want = {}
    for name, x in (("q", q), ("k", k)):
        want[name] = R.rotate(f64(x), rope.cpu().double(), p, inter) if rd else (f64(x), f64(x).abs())
    want["v"] = (f64(v), f64(v).abs())

    def close(got, name, dt, scale=None):
        y, mag = want[name]
        if scale is not None:
            y, mag = y / scale[:, None], mag / scale[:, None]
        step = 3 * 2.0 ** -24 * mag  # two products and their sum, a division
        if dt == E4M3:
            y = y.clamp(-448, 448)
            tol = step + torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10).double())
        else:
            tol = step + R.HALF[dt] * (y.abs() + step)
        assert ((f64(got) - y).abs() <= tol * (1 + 1e-6) + 1e-37).all(), name
    close(got_q, "q", act)
    at = [(int(table[s, t // P]), t % P) for s, t in zip(seq.tolist(), p)]
    close(torch.stack([kc[a, :, b] for a, b in at]), "k", store, None if ks is None else ks.cpu().double())
    close(torch.stack([vc[a, :, b] for a, b in at]), "v", store, None if vs is None else vs.cpu().double())
    # every other slot, and what lies between the pages, is as it was
    for new, old in ((kc, k0), (vc, v0)):
        new = new.clone()
        for a, b in at:
            bits(new)[a, :, b] = bits(old)[a, :, b]
        assert torch.equal(bits(new), bits(old))


def test_append_in_place_and_without_queries():
    m = M()
    table, pages = make_table([40], 16, 0, 1)
    rope = m.rope_table(64, 128)
    g = gen(2)
    q, k, v = (torch.randn((11, h, 128), generator=g).bfloat16().cuda() for h in (4, 2, 2))
    seq, pos = torch.zeros(11).int().cuda(), torch.arange(20, 31).int().cuda()
    outs = []
    for mode in ("new", "in place", "none"):
        kc, vc = (torch.zeros((pages, 2, 16, 128), dtype=BF16, device="cuda") for _ in range(2))
        c = m.PagedKVCache(kc, vc, table, 4, rope=rope)
        qq = None if mode == "none" else q.clone()
        r = c.append(qq, k, v, seq, pos, q_out=qq if mode == "in place" else None)
        c.check()
        outs.append((r, kc, vc))
    assert outs[2][0] is None
    assert torch.equal(outs[0][0], outs[1][0])
    for o in outs[1:]:
        assert torch.equal(outs[0][1], o[1]) and torch.equal(outs[0][2], o[2])


def test_append_special_values_e4m3():
    """Overflow saturates, infinities too, NaN stays NaN, zeros keep their sign."""
    m = M()
    table, pages = make_table([1], 16, 0, 1)
    kc, vc = (torch.zeros((pages, 1, 16, 64), device="cuda").to(E4M3) for _ in range(2))
    one = torch.ones(1, device="cuda")
    c = m.PagedKVCache(kc, vc, table, 1, k_scale=one, v_scale=2 * one)
    x = torch.zeros(1, 1, 64)
    x[0, 0, :8] = torch.tensor([500.0, -1e30, math.inf, -math.inf, math.nan, -0.0, 2.0 ** -9, 2.0 ** -10])
    x = x.bfloat16().cuda()
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(None, x, x, z, z)
    page = int(table[0, 0])
    got = kc[page, 0, 0].float().tolist()
    assert got[:4] == [448.0, -448.0, 448.0, -448.0] and math.isnan(got[4])
    assert got[5] == 0 and math.copysign(1, got[5]) == -1 and got[6] == 2.0 ** -9 and got[7] == 0
    assert vc[page, 0, 0].float().tolist()[0] == 256.0  # 250 to the nearest


def test_append_skips_padding_and_flags_bad_places():
    m = M()
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((3, 2, 16, 64), dtype=BF16, device="cuda") for _ in range(2))
    rope = m.rope_table(30, 64)
    c = m.PagedKVCache(kc, vc, table, 2, rope=rope)
    n = 7
    q, k, v = (torch.ones((n, 2, 64), dtype=BF16, device="cuda") for _ in range(3))
    # padding | fine | sequence 2 | negative position | past the table | past the rope | bad page
    seq = torch.tensor([-1, 0, 2, 0, 0, 0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 5, 0, -1, 32, 31, 17], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    c.append(q[:2], k[:2], v[:2], seq[:2], pos[:2], q_out=out[:2])
    c.check()
    for t in range(2, n):
        c.append(q[t:t + 1], k[t:t + 1], v[t:t + 1], seq[t:t + 1], pos[t:t + 1],
                 q_out=out[t:t + 1])
        with pytest.raises(m.MoEError) as e:
            c.check()
        assert e.value.status == 8
        c.status.zero_()
    keep = torch.ones(n, dtype=torch.bool)
    keep[1] = False
    assert (out[keep.cuda()] == 7).all() and not (out[1] == 7).any()
    assert int((vc != 0).sum()) == 2 * 64 and (vc[0, :, 5] == 1).all()


# ------------------------------------------------------------- attention
ATTEND = [
    # kind, Hq, Hkv, D, P, window, lens
    ("bf16", 16, 16, 128, 16, 0, (137,)),
    ("bf16", 1, 1, 64, 16, 0, (1,)),
    ("bf16", 2, 2, 128, 16, 0, (1, 2, 15, 16, 17, 63, 64, 65, 0, 128, 129)),
    ("bf16", 14, 2, 64, 48, 0, (300, 47, 48, 49)),
    ("bf16", 12, 1, 128, 32, 0, (1000, 0, 5)),
    ("bf16", 16, 1, 256, 16, 0, (700, 33)),
    ("bf16", 40, 2, 64, 64, 0, (77, 1500)),
    ("bf16", 4, 2, 256, 16, 0, (500,)),
    ("bf16", 4, 4, 128, 16, 100, (1, 99, 100, 101, 117, 1000)),
    ("bf16", 8, 1, 128, 128, 1, (640, 3)),
    ("bf16", 8, 1, 128, 64, 0, (9000,)),
    ("e4m3", 16, 2, 128, 32, 0, (513, 1, 31)),
    ("e4m3", 3, 3, 64, 16, 0, (200, 0, 77)),
    ("e4m3", 12, 1, 64, 16, 33, (200, 20)),
    ("e4m3", 6, 2, 256, 16, 0, (129, 600)),
    ("e4m3", 16, 1, 256, 32, 0, (90,)),
    ("f32", 6, 2, 64, 16, 0, (1, 300, 0, 33)),
    ("f32", 8, 1, 128, 16, 50, (400, 20)),
    ("f32", 20, 2, 64, 32, 0, (65, 700)),
    ("f32", 2, 2, 256, 48, 0, (100, 1111)),
]
P_ERR = {"bf16": 2.0 ** -16, "e4m3": 2.0 ** -11, "f32": 2.0 ** -22}


def attend_case(case, seed=0, q_std=2.0, poison=False):
    kind, Hq, Hkv, D, P, window, lens = case
    act = CACHES[kind][0]
    table, pages = make_table(lens, P, 2, 11 + seed)
    kc, vc, ks, vs = make_cache(kind, pages, Hkv, P, D, 12 + seed, gap=1)
    if poison:  # everything outside the visible tokens: NaN and infinities
        seen = torch.zeros((pages, P), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(max(0, n - window) if window else 0, n):
                seen[int(table[b, j // P]), j % P] = True
        at = ~seen.cuda()
        for c, bad in ((kc, math.nan), (vc, math.nan if kind == "e4m3" else math.inf)):
            x = c.float()
            x.permute(0, 2, 1, 3)[at] = bad
            c.copy_(x.to(c.dtype))
    q = (q_std * torch.randn((len(lens), Hq, D), generator=gen(13 + seed))).to(act).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = M().PagedKVCache(kc, vc, table, Hq, k_scale=ks, v_scale=vs)
    return cache, q, n, window, kind


def check_attend(cache, q, n, window, kind, out, lse, scale=None):
    scale = 1 / math.sqrt(cache.head_dim) if scale is None else scale
    want, wl, bound = R.attend(f64(q), scaled(cache.k_cache, cache.k_scale),
                               scaled(cache.v_cache, cache.v_scale), cache.page_table.cpu(),
                               n.cpu(), window, scale, P_ERR[kind])
    tol = bound + R.HALF[cache.dtype] * (want.abs() + bound) * (1 + 1e-6)
    err = (f64(out) - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    empty = n.cpu() == 0
    assert (f64(out)[empty] == 0).all()
    if lse is not None:
        got = lse.cpu().double()
        assert (got[empty] == -math.inf).all()
        live = ~empty
        if live.any():
            # the bound on scores, and float32's own rounding of the result
            assert ((got - wl)[live].abs() <= 1e-3).all()


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c[:6])) + "-n%d" % len(c[6]))
def test_attend(case):
    cache, q, n, window, kind = attend_case(case)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = cache.attend(q, n, lse=lse, window=window)
    cache.check()
    check_attend(cache, q, n, window, kind, out, lse)
    # again on the same workspace, without lse: bitwise the same
    assert torch.equal(out, cache.attend(q, n, window=window))
    assert int(cache.ws[:4 * q.shape[0] * cache.kv_heads].sum()) == 0


@pytest.mark.parametrize("case", [ATTEND[i] for i in (2, 3, 8, 12, 13, 16, 17)],
                         ids=lambda c: "-".join(map(str, c[:6])))
def test_attend_never_sees_masked_values(case):
    clean = attend_case(case)
    dirty = attend_case(case, poison=True)
    a = clean[0].attend(clean[1], clean[2], window=clean[3])
    b = dirty[0].attend(dirty[1], dirty[2], window=dirty[3])
    assert torch.isfinite(b.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attend_strided_queries_scale_and_stream(kind):
    case = (kind, 8, 4, 128, 16, 0, (90, 300, 7))
    cache, q, n, window, _ = attend_case(case)
    wide = torch.zeros((3, 12, 128), dtype=q.dtype, device="cuda")
    wide[:, 2:10] = q
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = cache.attend(wide[:, 2:10], n, scale=0.05, stream=s)
    s.synchronize()
    check_attend(cache, q, n, window, kind, out, None, scale=0.05)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attend_extreme_scores(kind):
    """Scores that rise far along the sequence, and infinite or NaN ones."""
    case = (kind, 2, 1, 64, 16, 0, (400,))
    cache, q, n, window, _ = attend_case(case, q_std=1.0)
    T = cache.page_table[0].tolist()
    for j in range(0, 400, 37):  # ever larger keys along the query
        cache.k_cache[T[j // 16], 0, j % 16] = (q[0, 0].float() * (0.2 * j / 37)).to(cache.dtype)
    out = cache.attend(q, n)
    check_attend(cache, q, n, window, kind, out, None)
    keep = cache.k_cache.clone()
    for bad in (math.inf, -math.inf, math.nan):
        cache.k_cache.copy_(keep)
        cache.k_cache[T[3], 0, 5, 7] = bad
        got = cache.attend(q, n).float().cpu()
        s = q[0, :, 7].float().cpu() * bad
        for h in range(2):
            if math.isnan(float(s[h])) or float(s[h]) > 0:  # as softmax gives
                assert torch.isnan(got[0, h]).all()
            else:  # exp(-inf): the token drops out
                assert torch.isfinite(got[0, h]).all()


def test_attend_flags_bad_lengths_and_pages():
    m = M()
    cache, q, n, _, _ = attend_case(("bf16", 2, 2, 64, 16, 0, (40, 20, 33)))
    good = cache.attend(q, n).clone()
    for change in ("long", "negative", "page"):
        lens, keep = n.clone(), cache.page_table.clone()
        if change == "long":
            lens[1] = cache.page_table.shape[1] * 16 + 1
        elif change == "negative":
            lens[1] = -1
        else:
            cache.page_table[1, 1] = 10 ** 6
        out = cache.attend(q, lens)
        with pytest.raises(m.MoEError) as e:
            cache.check()
        assert e.value.status == 8
        cache.status.zero_()
        cache.page_table.copy_(keep)
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    assert torch.equal(cache.attend(q, n), good)
    cache.check()


def test_attend_in_a_cache_past_32_bit_offsets():
    """Pages whose first element lies beyond 2^31 (and 2^32 bytes)."""
    m = M()
    Hkv, P, D, pages = 8, 128, 128, 17000
    assert pages * Hkv * P * D > 2 ** 31
    kc, vc = (torch.zeros((pages, Hkv, P, D), dtype=BF16, device="cuda") for _ in range(2))
    ids = [pages - 1, 16500, 3]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    small = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    big = m.PagedKVCache(kc, vc, table, Hkv)
    ref = m.PagedKVCache(*(torch.zeros((3, Hkv, P, D), dtype=BF16, device="cuda") for _ in range(2)),
                         small, Hkv)
    k, v = (torch.randn((300, Hkv, D), generator=gen(i)).bfloat16().cuda() for i in (1, 2))
    seq, pos = torch.zeros(300).int().cuda(), torch.arange(300).int().cuda()
    q, n = k[:1].contiguous(), torch.tensor([300], dtype=torch.int32, device="cuda")
    outs = []
    for c in (big, ref):
        c.append(None, k, v, seq, pos)
        outs.append(c.attend(q, n))
        c.check()
    assert torch.equal(*outs)
    for i, p in enumerate(ids):
        assert torch.equal(kc[p], ref.k_cache[i]) and torch.equal(vc[p], ref.v_cache[i])


# --------------------------------------------------------------- experts
EXPERTS = [
    # n, H, I, E, K, group
    (1, 256, 128, 8, 2, 128),
    (1, 128, 128, 1, 1, 32),
    (3, 384, 256, 7, 3, 64),
    (9, 256, 384, 5, 2, 32),
    (40, 256, 128, 4, 4, 128),   # 40 rows per expert: two entries, two column groups
    (17, 640, 128, 16, 5, 64),
    (33, 128, 256, 3, 1, 32),
    (64, 256, 128, 2, 1, 128),
]
# reductions long enough for two warps a unit, few and many pairs, odd records
EXPERTS_LONG = [
    (1, 1024, 1024, 4, 2, 64),
    (1, 1152, 1152, 5, 3, 128),
    (2, 1024, 1152, 6, 4, 32),
    (1, 2048, 128, 40, 8, 32),
    (3, 1280, 1024, 64, 8, 128),
    (70, 1152, 256, 2, 2, 32),
]


def make_w4(E, H, I, group, seed):
    g = gen(seed)
    out = []
    for rows, red in ((2 * I, H), (H, I)):
        out.append(torch.randint(-2 ** 31, 2 ** 31, (E, rows, red // 8), generator=g).int().cuda())
        s = (0.5 + torch.rand((E, rows, red // group), generator=g)) / (4.6 * math.sqrt(red))
        out.append(s.bfloat16().cuda())
    return out


def routing(n, E, K, seed):
    w, idx = torch.softmax(torch.randn((n, E), generator=gen(seed)), 1).topk(K, 1)
    return idx.int().cuda(), w.float().contiguous().cuda()


def check_experts(y, x, idx, tw, w):
    want, bound = R.experts(f64(x), idx.cpu(), tw.cpu().double(), R.unpack_w4(w[0].cpu(), w[1].cpu().float()),
                            R.unpack_w4(w[2].cpu(), w[3].cpu().float()))
    err = (f64(y) - want).abs()
    tol = bound + R.HALF[BF16] * (want.abs() + bound) * (1 + 1e-6)
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    norm = want.norm()
    if norm > 0:  # the final rounding is at most 2^-8 of each value; sums add far less on average
        assert float((f64(y) - want).norm() / norm) <= R.HALF[BF16] + 3e-4


@pytest.mark.parametrize("case", EXPERTS, ids=str)
def test_experts(case):
    n, H, I, E, K, group = case
    w = make_w4(E, H, I, group, 1)
    x = torch.randn((n, H), generator=gen(2)).bfloat16().cuda()
    idx, tw = routing(n, E, K, 3)
    m = M().W4Experts(*w, K=K, max_tokens=n + 5)
    y = m(x, idx, tw)
    m.check()
    check_experts(y, x, idx, tw, w)
    assert torch.equal(y, m(x, idx, tw))
    # a token's result does not depend on the others of the call
    t = n // 2
    assert torch.equal(y[t:t + 1], m(x[t:t + 1], idx[t:t + 1], tw[t:t + 1]))


@pytest.mark.parametrize("case", EXPERTS_LONG, ids=str)
def test_experts_long_reductions(case):
    n, H, I, E, K, group = case
    w = make_w4(E, H, I, group, 1)
    x = torch.randn((n, H), generator=gen(2)).bfloat16().cuda()
    idx, tw = routing(n, E, K, 3)
    m = M().W4Experts(*w, K=K, max_tokens=n)
    y = m(x, idx, tw)
    m.check()
    check_experts(y, x, idx, tw, w)
    assert torch.equal(y, m(x, idx, tw))
    bad = idx.clone()
    bad[0, 0] = -3
    y = m(x, bad, tw)
    assert int(m.status.item()) == 1
    check_experts(y, x, bad, tw, w)


def test_experts_invalid_and_repeated_ids():
    n, H, I, E, K = 6, 256, 128, 5, 3
    m = M()
    w = make_w4(E, H, I, 64, 1)
    x = torch.randn((n, H), generator=gen(2)).bfloat16().cuda()
    idx, tw = routing(n, E, K, 3)
    ex = m.W4Experts(*w, K=K, max_tokens=n)
    ex(x, idx, tw)
    ex.check()
    idx[1, 0], idx[2, 1] = -1, E  # skipped, and flagged
    idx[4] = 2                    # one expert three times
    idx[5] = E + 7                # nothing left: a zero row
    y = ex(x, idx, tw)
    with pytest.raises(m.MoEError) as e:
        ex.check()
    assert e.value.status == 4
    check_experts(y, x, idx, tw, w)
    assert (y[5] == 0).all()


def test_experts_do_not_read_other_tokens_infinities():
    n, H, I, E, K = 5, 256, 128, 4, 2
    w = make_w4(E, H, I, 128, 1)
    x = torch.randn((n, H), generator=gen(2)).bfloat16().cuda()
    idx, tw = routing(n, E, K, 3)
    ex = M().W4Experts(*w, K=K, max_tokens=n)
    y = ex(x, idx, tw).clone()
    x2 = x.clone()
    x2[2, 3], x2[4, 0] = math.inf, math.nan
    y2 = ex(x2, idx, tw)
    keep = torch.tensor([0, 1, 3]).cuda()
    assert torch.equal(y[keep], y2[keep])
    assert torch.isnan(y2[4].float()).all()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_w4(group):
    """The codes are the nearest ones, and W4Experts on them is the layer on
    the quantised weights."""
    m = M()
    E, H, I, K, n = 3, 256, 128, 2, 4
    g = gen(7)
    w13 = (torch.randn((E, H, 2 * I), generator=g) / 16).bfloat16().cuda()
    w2 = (torch.randn((E, I, H), generator=g) / 11).bfloat16().cuda()
    w13[1, :group, 5] = 0  # a group of zeros
    q = m.quantize_weights_w4(w13, w2, group)
    for w, words, s in ((w13, q[0], q[1]), (w2, q[2], q[3])):
        wt = f64(w).transpose(1, 2)
        top = wt.abs().unflatten(2, (-1, group)).amax(-1)
        assert torch.equal(s.cpu(), (top.float() / 7).bfloat16())
        sr = f64(s).repeat_interleave(group, 2)
        code = torch.where(sr > 0, (wt / sr).float().round().double().clamp(-8, 7), 0.0)
        assert torch.equal(R.unpack_w4(words.cpu(), s.cpu().float()), code * sr)
    x = torch.randn((n, H), generator=g).bfloat16().cuda()
    idx, tw = routing(n, E, K, 3)
    check_experts(m.W4Experts(*q, K=K, max_tokens=n)(x, idx, tw), x, idx, tw, q)


def test_zero_tokens_and_sequences():
    m = M()
    w = make_w4(2, 128, 128, 128, 1)
    ex = m.W4Experts(*w, K=1, max_tokens=4)
    z = torch.zeros((0, 128), dtype=BF16, device="cuda")
    assert ex(z, torch.zeros((0, 1), dtype=torch.int32, device="cuda"),
              torch.zeros((0, 1), device="cuda")).shape == (0, 128)
    cache, q, n, _, _ = attend_case(("bf16", 2, 2, 64, 16, 0, (0, 0)))
    assert (cache.attend(q, n) == 0).all()
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    kv = torch.zeros((0, 2, 64), dtype=BF16, device="cuda")
    assert cache.append(kv, kv, kv, e, e).shape == (0, 2, 64)
    cache.check()


def test_calls_can_be_captured_in_a_graph():
    """Every call of a step works under stream capture and replays on new data."""
    m = M()
    cache, q, n, _, kind = attend_case(("bf16", 8, 4, 128, 16, 0, (90, 300, 0)))
    w = make_w4(4, 256, 128, 64, 1)
    ex = m.W4Experts(*w, K=2, max_tokens=3)
    x = torch.randn((3, 256), generator=gen(1)).bfloat16().cuda()
    idx, tw = routing(3, 4, 2, 3)
    out, y = torch.empty_like(q), torch.empty_like(x)
    kv = torch.randn((2, 4, 128), generator=gen(2)).bfloat16().cuda()
    seq, pos = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ((0, 1), (89, 299)))

    def step():
        cache.append(None, kv, kv, seq, pos)
        cache.attend(q, n, out=out)
        ex(x, idx, tw, y=y)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in range(2):
        kv.copy_(torch.randn((2, 4, 128), generator=gen(20 + s)))
        x.copy_(torch.randn((3, 256), generator=gen(30 + s)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_attend(cache, q, n, 0, kind, out, None)
        check_experts(y, x, idx, tw, w)

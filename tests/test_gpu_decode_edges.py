"""Edges of the serving operators on the GPU, against their plain float64
forms: steep softmaxes, shared workspaces, very long sequences and pages,
values near the limits of their types, streams."""
import ctypes
import math
import threading

import pytest
import torch

from tests import decode_reference as R
from tests import test_gpu_decode as T

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


# ----------------------------------------------------- a steep softmax
STEEP = [
    # Hq, Hkv, D, P, lens
    (2, 1, 64, 16, (300, 17)),
    (4, 4, 128, 32, (3000,)),
    (16, 2, 128, 64, (900, 2, 8192)),
    (4, 1, 256, 16, (640,)),
    (12, 1, 128, 16, (333, 64)),
]


@pytest.mark.parametrize("nats", [12, 17, 25, 60])
@pytest.mark.parametrize("case", STEEP, ids=lambda c: "-".join(map(str, c[:4])))
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attend_keeps_the_tail_of_a_steep_softmax(kind, case, nats):
    """The first token of a sequence stands `nats` above the others and its
    value is zero, so that the result is the others' alone.

    Bound: scores as in the reference's (their sums, and the roundings of
    score and exponent), each probability rounded to no more than 2^-16 of
    itself however small it is (float32: 2^-22), sums in float32."""
    Hq, Hkv, D, P, lens = case
    cache, q, n, window, _ = T.attend_case((kind, Hq, Hkv, D, P, 0, lens), q_std=1.0)
    if kind == "e4m3":  # room for the first key below 448
        cache.k_cache.copy_((cache.k_cache.float() / 8).to(E4M3))
        cache.k_scale.mul_(8)
    G = Hq // Hkv
    for b in range(len(lens)):
        page = int(cache.page_table[b, 0])
        for h in range(Hkv):
            sc = 1.0 if cache.k_scale is None else float(cache.k_scale[h])
            u = q[b, h * G].float()
            k = u * (nats * math.sqrt(D) / float(u.square().sum())) / sc
            cache.k_cache[page, h, 0] = k.to(cache.k_cache.dtype)
            cache.v_cache[page, h, 0] = torch.zeros(D, device="cuda").to(cache.v_cache.dtype)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = cache.attend(q, n, lse=lse)
    cache.check()
    p_err = 2.0 ** -22 if kind == "f32" else 2.0 ** -16
    scale = 1 / math.sqrt(D)
    kc, vc = T.scaled(cache.k_cache, cache.k_scale), T.scaled(cache.v_cache, cache.v_scale)
    assert torch.isfinite(kc).all()
    table, qd = cache.page_table.cpu(), T.f64(q)
    want, wl, bound = R.attend(qd, kc, vc, table, n.cpu(), 0, scale, p_err)
    tol = bound + R.HALF[cache.dtype] * (want.abs() + bound) * (1 + 1e-6)
    err = (T.f64(out) - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    # lse moves by no more than the scores, the sum's relative error, and its
    # own rounding (in base 2, then by ln 2)
    for b, ln in enumerate(lens):
        k = R.gather(kc, table[b], 0, ln)
        for h in range(Hq):
            x = k[h // G] * qd[b, h] * scale
            ds = D * R.U32 * float(x.abs().sum(1).max()) + 4 * R.U32 * float(x.sum(1).abs().max())
            t = 2 * ds + 4 * (ln + 64) * R.U32 + 4 * R.U32 * abs(float(wl[b, h]))
            assert abs(float(lse[b, h]) - float(wl[b, h])) <= t


# ------------------------------------------- queries of very unequal values
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(2, 2), (12, 1)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attend_keeps_small_query_values(kind, heads, dim):
    """One value of each query is 2^20 times the others' size, and the cache
    holds zeros there: the scores are the others'.  The bound has nothing for
    the large value's products, which are zero."""
    cache, q, n, window, _ = T.attend_case((kind, *heads, dim, 16, 0, (150, 33)))
    q[..., 5] = 2.0 ** 20
    x = cache.k_cache.float()
    x[..., 5] = 0
    cache.k_cache.copy_(x.to(cache.k_cache.dtype))
    out = cache.attend(q, n)
    cache.check()
    T.check_attend(cache, q, n, window, "bf16", out, None)


@pytest.mark.parametrize("power", [-125, -100, 100, 120])
def test_attend_queries_of_any_size_e4m3(power):
    cache, q, n, window, _ = T.attend_case(("e4m3", 4, 2, 128, 16, 0, (150, 33)), q_std=1.0)
    q = (q.float() * 2.0 ** power).to(BF16)
    scale = 2.0 ** -power / math.sqrt(128) if power > -110 else 2.0 ** 120
    out = cache.attend(q, n, scale=scale)
    cache.check()
    T.check_attend(cache, q, n, window, "bf16", out, None, scale=scale)


# ------------------------------------------------------ shared workspaces
def test_attend_calls_of_any_sizes_share_a_workspace():
    """One workspace, zeroed once, for calls of other batches, head layouts and
    types: each result is that of a workspace of its own, and the counters (the
    first 6 KB) are left zero."""
    cases = [
        ("bf16", 16, 16, 64, 16, 0, tuple(300 + 7 * (i % 40) for i in range(200))),
        ("bf16", 16, 16, 64, 16, 0, (700, 90, 4000)),
        ("f32", 6, 1, 64, 16, 0, (3000, 2000)),
        ("e4m3", 24, 2, 128, 32, 0, (9000, 100, 0, 5)),
        ("bf16", 8, 1, 256, 16, 0, (20000,)),
        ("f32", 20, 2, 64, 32, 100, (65, 700)),
    ]
    made = [T.attend_case(c, seed=i) for i, c in enumerate(cases)]
    want = [cache.attend(q, n, window=w) for cache, q, n, w, _ in made]
    ws = torch.zeros(max(c[0].ws.numel() for c in made), dtype=torch.uint8, device="cuda")
    lib = T.M()._lib.load()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for i in (0, 1, 0, 2, 3, 0, 4, 5, 0, 4, 3, 0):
        cache, q, n, w, _ = made[i]
        out = torch.full_like(want[i], 7.0)
        assert lib.moe_paged_attention(
            ctypes.byref(cache.desc), q.data_ptr(), q.stride(0), n.data_ptr(), w,
            1 / math.sqrt(cache.head_dim), out.data_ptr(), None, ws.data_ptr(), ws.numel(),
            cache.status.data_ptr(), stream) == 0
        cache.check()
        assert torch.equal(out, want[i]), i
    assert int(ws[:6144].sum()) == 0


# --------------------------------------------------- very large pages, lengths
def test_attend_and_append_in_pages_past_32_bit_offsets():
    """A token's place inside its page lies beyond 2^31 bytes (the last tokens of
    a page of 8.4 million, seen through a window)."""
    P, D, w = 2 ** 23 + 16, 64, 30
    n = P - 6
    kc, vc = (torch.zeros((1, 1, P, D), device="cuda") for _ in range(2))
    big = T.M().PagedKVCache(kc, vc, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 2)
    k, v = (torch.randn((w, 1, D), generator=T.gen(i)).cuda() for i in (1, 2))
    seq = torch.zeros(w, dtype=torch.int32, device="cuda")
    big.append(None, k, v, seq, torch.arange(n - w, n, device="cuda").int())
    assert torch.equal(kc[0, :, n - w:n], k.transpose(0, 1))
    assert torch.equal(vc[0, :, n - w:n], v.transpose(0, 1))
    q = torch.randn((1, 2, D), generator=T.gen(3)).cuda()
    out = big.attend(q, torch.tensor([n], dtype=torch.int32, device="cuda"), window=w)
    big.check()
    small = T.M().PagedKVCache(*(torch.zeros((2, 1, 16, D), device="cuda") for _ in range(2)),
                               torch.arange(2, dtype=torch.int32, device="cuda").view(1, 2), 2)
    small.append(None, k, v, seq, torch.arange(w, device="cuda").int())
    T.check_attend(small, q, torch.tensor([w], dtype=torch.int32), 0, "f32", out, None)


def test_attend_lengths_near_the_end_of_32_bits():
    """The longest sequences (a page table may name one page many times), seen
    through a window; longer ones are out of range."""
    m, P, D, w, top = T.M(), 2 ** 24, 64, 100, 2 ** 31 - 1024
    kc, vc = (torch.zeros((1, 1, P, D), dtype=BF16, device="cuda") for _ in range(2))
    last = top % P
    for i, c in enumerate((kc, vc)):
        c[0, 0, last - w:last] = torch.randn((w, D), generator=T.gen(i)).cuda().to(BF16)
    cache = m.PagedKVCache(kc, vc, torch.zeros((2, 128), dtype=torch.int32, device="cuda"), 4)
    q = torch.randn((2, 4, D), generator=T.gen(3)).cuda().to(BF16)
    out = cache.attend(q, torch.tensor([top, 7], dtype=torch.int32, device="cuda"), window=w)
    cache.check()
    small = m.PagedKVCache(
        *(torch.nn.functional.pad(c[0, 0, last - w:last], (0, 0, 0, 12)).reshape(7, 1, 16, D)
          for c in (kc, vc)), torch.arange(7, dtype=torch.int32, device="cuda").view(1, 7), 4)
    T.check_attend(small, q[:1], torch.tensor([w], dtype=torch.int32), 0, "bf16", out[:1], None)
    for length in (top + 1, 2 ** 31 - 1):
        again = cache.attend(q, torch.tensor([length, 7], dtype=torch.int32, device="cuda"), window=w)
        with pytest.raises(m.MoEError) as e:
            cache.check()
        assert e.value.status == 8
        cache.status.zero_()
        assert torch.equal(again[1], out[1])


# ------------------------------------- experts: h at the ends of its range
def one_hot_layer(gates, ups, group, w2_code, w2_scale, n):
    """A layer of one expert (H = I = 128) in which every token's h[i] is
    SiLU(gates[i]) * ups[i], each a bf16 value, for the first i and 0 beyond;
    w2's codes are w2_code (H, I)."""
    H = I = 128
    codes = torch.full((1, 2 * I, H), 8)
    s13 = torch.ones((1, 2 * I, H // group))
    for base, values in ((0, gates), (I, ups)):
        for i, v in enumerate(values):
            codes[0, base + i, 0] = 9 if v >= 0 else 7
            s13[0, base + i, 0] = abs(v)

    def pack(c):
        c = c.unflatten(-1, (-1, 8)).long()
        w = sum(c[..., j] << (4 * (j // 2) + 16 * (j % 2)) for j in range(8))
        return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int().cuda()
    w = [pack(codes), s13.bfloat16().cuda(), pack(w2_code[None]),
         torch.full((1, H, I // group), w2_scale).bfloat16().cuda()]
    assert R.unpack_w4(w[0].cpu(), w[1].cpu().float())[0, :len(gates), 0].tolist() == list(gates)
    x = torch.zeros((n, H), dtype=BF16, device="cuda")
    x[:, 0] = 1
    idx = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    return w, x, idx, torch.ones((n, 1), device="cuda")


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("group", [32, 128])
def test_experts_h_beyond_bf16(n, group):
    """Finite float32 h that rounds to an infinite bf16, of both signs."""
    a = 181 / 128  # its square is 1.99957
    code = torch.full((128, 128), 8)
    code[:, 0], code[::2, 1], code[1::2, 2] = 9, 7, 9
    w, x, idx, tw = one_hot_layer([a * 2.0 ** 63, a * 2.0 ** 60, a * 2.0 ** 63],
                                  [a * 2.0 ** 64, a * 2.0 ** 60, -a * 2.0 ** 64], group, code, 2.0 ** -20, n)
    ex = T.M().W4Experts(*w, K=1, max_tokens=n)
    y = ex(x, idx, tw)
    assert torch.isfinite(y.float()).all()
    T.check_experts(y, x, idx, tw, w)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("group", [32, 128])
def test_experts_infinite_h(n, group):
    """An infinite h among finite ones gives infinities, as the sum does, where
    no code is zero, and NaN where its own code is."""
    code = torch.full((128, 128), 9)
    code[1] = 7
    code[2, 1] = 8
    w, x, idx, tw = one_hot_layer([3.0, 2.0 ** 70], [1.0, 2.0 ** 70], group, code, 0.5, n)
    y = T.M().W4Experts(*w, K=1, max_tokens=n)(x, idx, tw).float()
    assert (y[:, 0] == math.inf).all() and (y[:, 1] == -math.inf).all()
    assert torch.isnan(y[:, 2]).all() and (y[:, 3:] == math.inf).all()
    w, x, idx, tw = one_hot_layer([3.0, 2.0 ** 70], [1.0, 2.0 ** 70], group, code, 0.5, n)
    x[:, 0] = math.nan
    assert torch.isnan(T.M().W4Experts(*w, K=1, max_tokens=n)(x, idx, tw).float()).all()


@pytest.mark.parametrize("n", [1, 40])
def test_experts_strongly_negative_gates(n):
    """SiLU far below zero, raised to ordinary size by a large `up`: exp(-88)
    and exp(-90) are subnormal, within 2^-18 of themselves."""
    gates = [-1.0, -20.0, -60.0, -80.0, -87.0, -88.0, -90.0, 90.0]
    ups = [2.0 ** round(-g * math.log2(math.e) - math.log2(abs(g))) if g < 0 else 1 / 64 for g in gates]
    code = torch.full((128, 128), 8)
    for i in range(len(gates)):
        code[i::16, i] = 9
        code[8 + i::16, i] = 15
    w, x, idx, tw = one_hot_layer(gates, ups, 32, code, 0.5, n)
    y = T.M().W4Experts(*w, K=1, max_tokens=n)(x, idx, tw)
    T.check_experts(y, x, idx, tw, w)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_quantize_keeps_non_finite_weights_visible(bad):
    """A group with an infinite or NaN weight gets a NaN scale and codes 8; the
    other groups are as without it."""
    m, E, H, I, group = T.M(), 2, 256, 128, 64
    w13 = (torch.randn((E, H, 2 * I), generator=T.gen(1)) / 16).bfloat16().cuda()
    w2 = (torch.randn((E, I, H), generator=T.gen(2)) / 11).bfloat16().cuda()
    want = m.quantize_weights_w4(w13, w2, group)
    w13[1, 70, 9], w2[0, 3, 200] = bad, bad
    got = m.quantize_weights_w4(w13, w2, group)
    for (q, s, q0, s0), at in (((*got[:2], *want[:2]), (1, 9, 1)), ((*got[2:], *want[2:]), (0, 200, 0))):
        e, c, g = at
        words = group // 8
        assert torch.isnan(s[at].float())
        assert (q[e, c, g * words:(g + 1) * words] == 0x88888888 - 2 ** 32).all()
        q, s = q.clone(), s.clone()
        s[at] = s0[at]
        q[e, c, g * words:(g + 1) * words] = q0[e, c, g * words:(g + 1) * words]
        assert torch.equal(q, q0) and torch.equal(s, s0)


# ------------------------------------------------------- threads and streams
def test_experts_object_shared_by_threads():
    """Threads with token counts of their own call one object on one stream."""
    H, I, E, K = 256, 128, 8, 2
    ex = T.M().W4Experts(*T.make_w4(E, H, I, 64, 1), K=K, max_tokens=64)
    work = []
    for i, n in enumerate((1, 3, 40, 64)):
        x = torch.randn((n, H), generator=T.gen(i)).bfloat16().cuda()
        idx, tw = T.routing(n, E, K, 10 + i)
        work.append((x, idx, tw, ex(x, idx, tw).clone(), []))
    torch.cuda.synchronize()

    def calls(x, idx, tw, want, got):
        for _ in range(30):
            got.append(ex(x, idx, tw))
    threads = [threading.Thread(target=calls, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    ex.check()
    for *_, want, got in work:
        assert len(got) == 30 and all(torch.equal(want, g) for g in got)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attend_on_two_streams_at_once(kind):
    """Calls of one cache on two streams, with lengths of their own."""
    cache, q, n, _, _ = T.attend_case((kind, 8, 4, 128, 16, 0, (3000, 40, 7000)))
    cases = [(q, n), (q + 1, torch.tensor([500, 0, 6001], dtype=torch.int32, device="cuda"))]
    want = [cache.attend(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(q) for _ in range(25)] for _ in cases]
    for i in range(25):
        for c, s, o in zip(cases, streams, outs):
            cache.attend(*c, out=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
    assert torch.equal(cache.attend(*cases[0]), want[0])
    cache.check()


def test_experts_on_two_streams_at_once():
    H, I, E, K = 1024, 512, 16, 4
    ex = T.M().W4Experts(*T.make_w4(E, H, I, 64, 1), K=K, max_tokens=60)
    cases = []
    for i, n in enumerate((60, 5)):
        x = torch.randn((n, H), generator=T.gen(i)).bfloat16().cuda()
        cases.append((x, *T.routing(n, E, K, 10 + i)))
    want = [ex(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(c[0]) for _ in range(25)] for c in cases]
    for i in range(25):
        for c, s, o in zip(cases, streams, outs):
            ex(*c, y=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
    ex.check()


def test_first_call_on_another_stream_waits_for_the_constructor():
    H, I, E, K, n = 2048, 1024, 64, 8, 2
    w = T.make_w4(E, H, I, 128, 1)
    x = torch.randn((n, H), generator=T.gen(2)).bfloat16().cuda()
    idx, tw = T.routing(n, E, K, 3)
    want = T.M().W4Experts(*w, K=K, max_tokens=n)(x, idx, tw)
    cache, q, lens, _, _ = T.attend_case(("bf16", 16, 16, 128, 16, 0, (5000,)))
    rows = cache.attend(q, lens)
    table = cache.page_table
    for _ in range(3):
        s, y, o = torch.cuda.Stream(), torch.empty_like(x), torch.empty_like(q)
        torch.cuda.synchronize()
        T.M().W4Experts(*w, K=K, max_tokens=n)(x, idx, tw, y=y, stream=s)
        T.M().PagedKVCache(cache.k_cache, cache.v_cache, table, 16).attend(q, lens, out=o, stream=s)
        s.synchronize()
        assert torch.equal(y, want) and torch.equal(o, rows)
        torch.cuda.synchronize()


def test_results_of_a_side_stream_spare_the_current_streams_memory():
    """A result that a call on another stream allocates is not in memory that
    the current stream's work still uses."""
    cache, q, n, _, _ = T.attend_case(("bf16", 8, 4, 128, 16, 0, (90, 300, 7)))
    want = cache.attend(q, n)
    s = torch.cuda.Stream()
    big = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        old = torch.full_like(want, 3.0)
        for _ in range(20):
            big.add_(1)  # holds the current stream up
        kept = old + 1
        del old          # free for the current stream, which has yet to read it
        out = cache.attend(q, n, stream=s)
        torch.cuda.synchronize()
        assert (kept == 4).all() and torch.equal(out, want)
    codes = T.M().quantize_weights_w4(*(torch.randn((2, 128, m), generator=T.gen(1)).bfloat16().cuda()
                                        for m in (256, 128)), group=64)
    ex = T.M().W4Experts(*codes, K=1, max_tokens=4)
    x = torch.randn((4, 128), generator=T.gen(2)).bfloat16().cuda()
    idx, tw = T.routing(4, 2, 1, 3)
    want = ex(x, idx, tw)
    torch.cuda.synchronize()
    got = ex(x, idx, tw, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_objects_made_on_a_side_stream_serve_the_default_one():
    _, q, n, _, _ = made = T.attend_case(("bf16", 8, 4, 128, 16, 0, (90, 3000, 7)))
    w = T.make_w4(4, 256, 128, 64, 1)
    x = torch.randn((3, 256), generator=T.gen(1)).bfloat16().cuda()
    idx, tw = T.routing(3, 4, 2, 3)
    rows, y = made[0].attend(q, n), T.M().W4Experts(*w, K=2, max_tokens=3)(x, idx, tw)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        cache = T.M().PagedKVCache(made[0].k_cache, made[0].v_cache, made[0].page_table, 8)
        ex = T.M().W4Experts(*w, K=2, max_tokens=3)
    for stream in (None, 0, torch.cuda.default_stream()):
        assert torch.equal(cache.attend(q, n, stream=stream), rows)
        assert torch.equal(ex(x, idx, tw, stream=stream), y)
    assert len(cache._pointers) == 2 and len(ex._pointers) == 2
    cache.check()
    ex.check()

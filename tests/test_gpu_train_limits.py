"""The training calls at the ends of their ranges, on the GPU: gradient norms
that float32 squares do not hold, steps counted on other streams, calls that
are refused."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def M():
    import top_routing_dispatch_gb300 as m
    return m


# ----------------------------------------------------------- clipping factor
@pytest.mark.parametrize("bad", [1e25, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
def test_nothing_is_clipped_without_a_limit(state, bad):
    """max_norm infinite: the factor is 1 whatever the norm, but for a NaN; the
    step that takes it changes every other value as if there were no factor."""
    start, g = torch.linspace(-1, 1, 700, device="cuda"), torch.linspace(-2, 3, 700, device="cuda")
    g[300] = bad
    params = [start.clone() for _ in range(2)]
    norm, factor = M().GradNorm([g])()
    if math.isnan(bad):
        assert math.isnan(float(norm)) and math.isnan(float(factor))
        return
    assert [float(norm), float(factor)] == [math.inf, 1.0]
    for p, scale in zip(params, (factor, None)):
        M().AdamW([p], [g], state=state).step(grad_scale=scale)
    keep = (torch.arange(700) != 300).cuda()
    assert torch.isfinite(params[0][keep]).all() and not torch.equal(params[0][keep], start[keep])
    assert torch.equal(params[0][keep], params[1][keep])
    # a limit, however large, clips an infinite norm to nothing
    assert float(M().GradNorm([g])(3e38)[1]) == 0.0


# ------------------------------------------------------- steps of other streams
def test_steps_waits_for_every_stream():
    """The number of steps, and a state to be saved, while steps on another
    stream are still to run."""
    p, g = torch.ones(5000, device="cuda"), torch.ones(5000, device="cuda")
    opt = M().AdamW([p], [g])
    opt.step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms of work before the steps
    for _ in range(3):
        opt.step(stream=side)
    assert opt.steps == 4
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    opt.step(stream=side)
    d = opt.state_dict()
    assert d["steps"] == 5


@pytest.mark.parametrize("kind", [(F32, F32, None, 0), (BF16, F32, True, 0), (BF16, BF16, None, 0), (F32, BF16, None, 1),
                                  (BF16, F32, True, 3)], ids=["f32", "master", "bf16", "bf16-grad-off", "master-off"])
def test_random_codes_are_the_stated_ones(kind):
    """Every code and scale of five steps, from the hash of the step's number."""
    from tests import train_random_reference as Q
    from tests import train_reference as R
    dtype, grad, masters, off = kind
    shapes = [(1,), (255,), (257,), (100, 33), (30011,)]
    gen = torch.Generator()
    gen.manual_seed(3)

    def make(n, dt, std):
        buf = torch.empty(n + off, dtype=dt, device="cuda")
        buf[off:] = (torch.randn(n, generator=gen) * std).to(dt).cuda()
        return buf[off:]
    params = [make(math.prod(s), dtype, 0.02).view(s) for s in shapes]
    grads = [make(math.prod(s), grad, 10.0 ** -i).view(s) for i, s in enumerate(shapes)]
    opt = M().AdamW(params, grads, lr=1e-3, betas=(0.9, 0.99), state=E4M3, masters=masters)
    held = []
    for s in shapes:
        rows = -(-math.prod(s) // 256)
        held.append((torch.zeros(rows, 256), torch.zeros(rows), torch.zeros(rows, 256), torch.zeros(rows)))
    for t in range(5):
        opt.step()
        for i, (g, n) in enumerate(zip(grads, map(math.prod, shapes))):
            held[i] = Q.step(R.blocks(g.cpu().float()), held[i], t, 0.9, 0.99)[0]
            b, e = opt.offsets[i], opt.offsets[i] + len(held[i][1])
            live = torch.arange(256 * (e - b)).view(-1, 256) < n
            for got, want in ((opt.m, held[i][0]), (opt.v, held[i][2])):
                got, want = got[b:e].cpu().float(), want.float()
                assert torch.equal(got[live], want[live]) and not got[~live].any()
            assert torch.equal(opt.m_scale[b:e].cpu(), held[i][1])
            assert torch.equal(opt.v_scale[b:e].cpu(), held[i][3])
        for g in grads:
            g.copy_((torch.randn(g.shape, generator=gen) * 10.0 ** -(t % 3)))


def test_rounding_goes_by_beta2_unless_given():
    """To nearest up to 31/32, at random above; either where asked for."""
    def codes(b2, rounding):
        g = torch.linspace(-1, 1.7, 4000, device="cuda")
        opt = M().AdamW([torch.zeros(4000, device="cuda")], [g], betas=(0.9, b2), state=E4M3, rounding=rounding)
        for _ in range(2):
            opt.step()
        return torch.cat([opt.m.view(torch.uint8), opt.v.view(torch.uint8)])
    for b2, default, other in ((0.5, "nearest", "random"), (31 / 32, "nearest", "random"),
                               (0.969, "random", "nearest"), (0.999, "random", "nearest")):
        assert torch.equal(codes(b2, None), codes(b2, default))
        assert not torch.equal(codes(b2, None), codes(b2, other))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_random_codes_keep_a_bad_gradient_where_it_is(bad):
    def run(value):
        g = torch.linspace(-1, 2, 700, device="cuda")
        g[300] = value
        p = torch.ones(700, device="cuda")
        opt = M().AdamW([p], [g], state=E4M3)
        for _ in range(3):
            opt.step()
        return p, opt
    (p, opt), (q, good) = run(bad), run(0.0)
    keep = (torch.arange(700) != 300).cuda()
    assert torch.equal(p[keep], q[keep]) and torch.isfinite(p[keep]).all()
    for a, b in ((opt.m, good.m), (opt.v, good.v)):
        a, b = a.float().view(-1)[:700], b.float().view(-1)[:700]
        assert torch.isnan(a[300]) and torch.equal(a[keep], b[keep])
    assert torch.equal(opt.m_scale, good.m_scale) and torch.equal(opt.v_scale, good.v_scale)


def test_random_codes_of_a_captured_step_are_the_eager_ones():
    def make():
        g = torch.linspace(-1, 1.7, 40_000, device="cuda")
        return M().AdamW([torch.zeros(40_000, device="cuda")], [g], state=E4M3)
    eager, captured = make(), make()
    captured.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for _ in range(4):
        graph.replay()
    for _ in range(5):
        eager.step()
    assert captured.steps == eager.steps == 5
    assert torch.equal(captured.params[0], eager.params[0])
    for a, b in ((captured.m, eager.m), (captured.v, eager.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------- 8-bit states over many steps
def long_run(b2, quiet, steps, **kw):
    """An optimizer with 8-bit states and one with float32 states on the same
    random gradients of unit size, a quarter of each block `quiet` times that
    after 500 steps."""
    n = 256 * 256
    g, size = torch.empty(n, device="cuda"), torch.ones(256, 256, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    opts = [M().AdamW([torch.zeros(n, device="cuda")], [g], lr=1e-3, betas=(0.9, b2), weight_decay=0.0, state=s, **k)
            for s, k in ((E4M3, kw), (F32, {}))]
    for t in range(steps):
        if t == 500:
            size[:, :64] = quiet
        g.normal_(generator=gen).mul_(size.view(-1))
        if t == steps - 400:
            kept = opts[0].params[0].clone()
        for o in opts:
            o.step()
    small, full = opts
    m = small.m.double() * small.m_scale.double()[:, None]
    v = (small.v.double() * small.v_scale.double()[:, None]).square()
    return m, v, full.m.double(), full.v.double(), (small.params[0] - kept).view(256, 256)


@pytest.mark.parametrize("b2,kw", [(0.999, {}), (0.98, {}), (0.95, dict(rounding="random"))],
                         ids=["0.999", "0.98", "0.95-random"])
def test_moments_in_8_bits_follow_their_recurrences(b2, kw):
    """The sums of v over many values, and each m, against float32 states.

    v: each step's rounding is unbiased, so V8 - V32 is a sum of martingale
    differences times powers of b2.  Before a step v lies on a code; the step
    moves it, against the codes at the new scale, by at most (1 - b2) c v with c
    = 1 + g^2/v + |g_top^2/v_top - 1|, on average about 3.  The variance of a
    rounding is at most the distance to one neighbour times the gap, 0.27 v:
    0.8 (1 - b2) v^2 a step, 0.4 v^2 in all, for which v^2 = V32^2 (1 + cv^2):
    cv^2 = 0.4 / 0.6, cv at most 0.82.  Six deviations of a mean of N values, and
    (1000 steps of 3 u) 2e-4.  The values share each gradient's chance.

    m: a rounding's deviation is at most half a gap, |m| / 16, and those of
    earlier steps count 0.81 each: sqrt(1 / 0.19) / 16 = 0.144 of m's root mean
    square, taken over 16384 values of a spread below 1.5 (six deviations of
    their mean square: 1.5 * 6 / 128 = 7 %)."""
    m, v, m32, v32, _ = long_run(b2, 0.01, 500 + int(14 / (1 - b2)), **kw)
    for part in (slice(0, 64), slice(64, 256)):
        N = v[:, part].numel()
        assert abs(float(v[:, part].sum() / v32[:, part].sum()) - 1) <= 6 * 0.82 / N ** 0.5 + 2e-4
        off = (m - m32)[:, part].square().mean().sqrt() / m32[:, part].square().mean().sqrt()
        assert float(off) <= 0.144 * 1.07


@pytest.mark.parametrize("b2,kw", [(0.999, {}), (0.98, {}), (0.95, dict(rounding="random"))],
                         ids=["0.999", "0.98", "0.95-random"])
def test_no_gradient_no_step_in_8_bits(b2, kw):
    """Values without a gradient, beside others that have one: m goes to zero
    and the parameter stays (a code of the smallest size has a chance of one in
    ten to go at each step)."""
    m, v, m32, v32, moved = long_run(b2, 0.0, 3000, **kw)
    assert not m[:, :64].any() and (v[:, :64] > 0).all()
    assert not moved[:, :64].any() and moved[:, 64:].all()


# --------------------------------------------------- gradient norm's range
def check_grad_norm(grads, slack=0):
    total = math.sqrt(math.fsum(float(t.detach().cpu().double().square().sum()) for t in grads))
    norm, factor = M().GradNorm(grads)(1.0)
    # nine roundings of a square and of its short sum, halved by the root, and the root's own;
    # the result may be subnormal
    tol = (4.5 + 1) * 2.0 ** -24 * total + 2.0 ** -150
    assert abs(float(norm) - total) <= tol, (float(norm), total)
    want = min(1.0, 1 / (total + 1e-6))
    assert abs(float(factor) - want) <= (5.5 + 4) * 2.0 ** -24 * want + 2.0 ** -150


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("size", [4e18, 1.3e19, 1.84e19])
def test_grad_norm_of_large_values(T, off, size):
    """Squares that float32 holds (below 3.4e38, the square of 1.84e19), sums of
    them that it does not: beside each other, one at the end, on all threads."""
    for n, at in ((64, slice(0, 64)), (70_003, slice(5_000, 5_128)), (30_011, slice(30_004, 30_011)),
                  (40_000, slice(0, 40_000))):
        t = torch.full((n + off,), 1e-3, device="cuda")[off:]
        t[at] = size
        check_grad_norm([t.to(T) if not off else torch.cat([t[:1], t]).to(T)[1:]])


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("size", [1e-21, 1e-23, 3e-30, 1.2e-38, 1e-44])
def test_grad_norm_of_small_values(T, off, size):
    """Values whose squares float32 rounds to few bits, or to zero."""
    if T == BF16 and size < 1e-40:
        size = 1e-40  # a subnormal of bfloat16
    for n in (1, 3, 64, 5_003, 100_000):
        t = torch.full((n + off,), size, device="cuda")
        t[off::2] *= -1
        t = t.to(T)[off:]
        check_grad_norm([t, torch.zeros(3000, device="cuda")])
    check_grad_norm([torch.full((3000,), size, device="cuda", dtype=T), torch.full((10,), 1e-19, device="cuda"),
                     torch.full((5000,), 1e-17, device="cuda")])


def test_grad_norm_of_zeros():
    z = torch.zeros(70_001, device="cuda")
    assert [float(t) for t in M().GradNorm([z, -z, z.to(BF16)])(1.0)] == [0.0, 1.0]


# ------------------------------------------------------------ refused calls
def test_a_refused_backward_changes_no_gradient():
    """Every argument of a block's backward is checked before its first kernel."""
    from tests.test_gpu_train_step import make_block
    block, x, r, dout, ds = make_block(40, False, True)
    block.forward(x, r)
    block.backward(dout, ds)
    want = [g.clone() for g in block.grads] + [block.d_in.clone()]
    wide = torch.empty(40, 512, dtype=BF16, device="cuda")
    for kw in (dict(ds=ds.float()), dict(ds=ds[:5]), dict(ds=ds.t().contiguous().t()), dict(ds=ds.cpu()),
               dict(ds=ds[:1].expand(40, 256)),
               dict(dx=ds.float()), dict(dx=ds[:5]), dict(dx=wide[:, ::2]), dict(dx=wide[:, :256]),
               dict(dx=ds.cpu())):
        with pytest.raises(ValueError):
            block.backward(ds if kw.get("ds") is None else r, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, block.grads + [block.d_in]))
    # rows of ds a stride apart are taken
    wide[:, :256] = ds
    assert torch.equal(block.backward(dout, wide[:, :256]), block.backward(dout, ds))


# ------------------------------------------------------------- scratch memory
def norm_inputs(n, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x, dy = (torch.randn(n, H, device="cuda", generator=g).to(BF16) for _ in range(2))
    layer, stats = M().LayerNorm(torch.ones(H, device="cuda"), torch.zeros(H, device="cuda"), dtype=BF16), None
    stats = torch.empty((2, n), device="cuda")
    layer(x, stats=stats)
    return layer, dy, x, stats


def test_scratch_of_long_rows_is_not_kept():
    from top_routing_dispatch_gb300 import train
    layer, dy, x, stats = norm_inputs(320, 65536, 1)
    want = layer.backward(dy, x, stats)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for _ in range(3):
            got = layer.backward(dy, x, stats, stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(t.numel() <= 32 << 20 for t in train._scratch.values())


def test_calls_on_the_threads_own_streams():
    """Backward calls and gradient norms of two threads, each on its thread's
    default stream (handle 2)."""
    import threading
    work = []
    for seed, (n, H) in enumerate(((600, 2048), (500, 1024))):
        args = norm_inputs(n, H, seed)
        norm = M().GradNorm([args[1], args[2]])
        work.append((args, norm, [*args[0].backward(*args[1:]), *norm(1.0)], []))
    torch.cuda.synchronize()

    def calls(args, norm, want, got):
        layer, *rest = args
        for _ in range(25):
            got.append([*layer.backward(*rest, stream=2), *norm(1.0, stream=2)])
        torch.cuda.ExternalStream(2).synchronize()
    threads = [threading.Thread(target=calls, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for *_, want, got in work:
        assert len(got) == 25 and all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_a_block_refuses_results_in_its_inputs():
    """out in the memory of what the backward reads again, or of an input."""
    from tests.test_gpu_train_step import make_block
    block, x, r, dout, ds = make_block(40, False, True)
    line = torch.empty(60, 256, dtype=BF16, device="cuda")
    for kw in (dict(x=x, out=x), dict(x=x, residual=r, out=x), dict(x=x, residual=r, out=r),
               dict(x=x, residual=r, out=block.s), dict(x=x, out=block.h_in), dict(x=line[:40], out=line[20:]),
               dict(x=line[20:], residual=r, out=line[:40])):
        with pytest.raises(ValueError, match="memory"):
            block.forward(**kw)
    out, s = block.forward(line[:20].repeat(2, 1), r, out=line[20:])
    assert out.data_ptr() == line[20:].data_ptr()
    block.forward(x, r)
    for kw in (dict(dx=block.d_in), dict(dx=block.s)):
        with pytest.raises(ValueError, match="memory"):
            block.backward(dout, ds, **kw)


# -------------------------------------------------------------- rows at the range's end
@pytest.mark.parametrize("H", [64, 257, 2048, 20000, 70001])
@pytest.mark.parametrize("T", [F32, BF16])
def test_rows_beyond_float32(T, H):
    """Squares beyond float32: y is the bias.  A sum of the row itself beyond it:
    NaN, in that row only; without a mean there is no such sum."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(20, H, device="cuda", generator=g).to(T)
    b = torch.randn(H, device="cuda", generator=g)
    w = torch.ones(H, device="cuda")
    for rms in (False, True):
        layer = M().LayerNorm(w, b, rms=rms, dtype=T)
        want = layer(x)
        wild = x.clone()
        wild[3] = 3e38  # their sum is infinite
        wild[7] = torch.where(torch.arange(H, device="cuda") % 2 == 0, 1e25, -1e25).to(T)
        got = layer(wild)
        keep = torch.ones(20, dtype=torch.bool, device="cuda")
        keep[3] = keep[7] = False
        assert torch.equal(got[keep], want[keep])
        assert torch.equal(got[7], b.to(T))
        assert torch.equal(got[3], b.to(T)) if rms else torch.isnan(got[3].float()).all()


def test_a_resumed_optimizer_rounds_as_the_first_one():
    """beta2 0.999, 8 bits: states and their number of steps are all that the
    random rounding depends on."""
    def make():
        return M().AdamW([torch.linspace(-1, 1, 5000, device="cuda")], [torch.linspace(-1, 1.7, 5000, device="cuda")],
                         state=E4M3)
    a, b = make(), make()
    for _ in range(3):
        a.step()
    b.params[0].copy_(a.params[0])
    b.load_state_dict({k: v.clone() if torch.is_tensor(v) else v for k, v in a.state_dict().items()})
    for _ in range(2):
        a.step()
        b.step()
    assert torch.equal(a.params[0], b.params[0]) and a.steps == b.steps == 5
    for x, y in ((a.m, b.m), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))

"""The training operators (layer norm and its gradients, global gradient norm,
AdamW) on the GPU, against their plain float64 forms in train_reference.py."""
import ctypes
import math

import pytest
import torch

from tests import train_reference as R

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def M():
    import top_routing_dispatch_gb300 as m
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rand(seed, *shape, std=1.0):
    return torch.randn(shape, generator=gen(seed)) * std


def f64(t):
    return t.detach().cpu().double()


def within(got, want, tol, dtype):
    """got (stored in dtype) is within tol, and its last rounding, of want."""
    got = f64(got)
    tol = tol + R.half_step(want.abs() + tol, dtype)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol.clamp(min=1e-300)).max()))


# ------------------------------------------------------------------- norm
# rows, length: every group size and kernel, lengths on both sides of each
# boundary, odd ones, one value, one row, rows longer than a CTA's registers
SIZES = [(1, 1), (3, 2), (1, 7), (130, 8), (17, 64), (33, 72), (9, 128), (65, 136), (5, 256), (7, 257),
         (129, 264), (31, 512), (6, 520), (40, 1024), (3, 1031), (12, 2048), (2, 2056), (301, 2048),
         (5, 4096), (3, 4104), (700, 1024), (4, 7168), (3, 8192), (2, 8200), (3, 16384), (2, 16392),
         (1, 32776), (2, 70001), (1, 70008), (2000, 40), (1000, 33)]


def norm_case(n, H, T, W, rms, bias, residual, seed=0, x=None):
    x = (rand(seed, n, H) * (0.5 + 2 * torch.rand((n, 1), generator=gen(seed + 1)))
         + rand(seed + 2, n, 1)).to(T) if x is None else x
    res = rand(seed + 3, n, H).to(T) if residual else None
    w = (1 + rand(seed + 4, H, std=0.3)).to(W)
    b = rand(seed + 5, H, std=0.2).to(W) if bias else None
    eps = 1e-6 if rms else 1e-5
    layer = M().LayerNorm(w.cuda(), None if b is None else b.cuda(), eps=eps, rms=rms, dtype=T)
    return layer, x, res, w, b, eps


def check_norm(layer, x, res, w, b, eps, rms, y, s, stats):
    T = x.dtype
    rows = x
    if res is not None:
        rows = (x.float() + res.float()).to(T)
        assert torch.equal(s.cpu(), rows)
    want, tol, mean, e_mean, r, e_r = R.norm(f64(rows), f64(w), None if b is None else f64(b), eps, rms)
    within(y, want, tol, T)
    if stats is not None:
        got = f64(stats)
        assert ((got[0] - mean).abs() <= e_mean).all()
        assert ((got[1] - r).abs() <= e_r * r).all()


@pytest.mark.parametrize("n,H", SIZES)
@pytest.mark.parametrize("form", [(F32, F32, False, True, False), (BF16, F32, False, True, True),
                                  (BF16, BF16, True, False, True), (F32, F32, True, False, True),
                                  (BF16, BF16, False, False, False)],
                         ids=["f32", "bf16-residual", "bf16-rms-residual", "f32-rms-residual", "bf16"])
def test_norm(n, H, form):
    T, W, rms, bias, residual = form
    layer, x, res, w, b, eps = norm_case(n, H, T, W, rms, bias, residual)
    stats = torch.empty((2, n), device="cuda")
    out = layer(x.cuda(), None if res is None else res.cuda(), stats=stats)
    y, s = out if residual else (out, None)
    check_norm(layer, x, res, w, b, eps, rms, y, s, stats)
    # without statistics the same
    out = layer(x.cuda(), None if res is None else res.cuda())
    assert torch.equal(out[0] if residual else out, y)


def rows_chain(n):
    """Longest chain of the sums over n rows: a range's rows, then its warps or
    groups, then the ranges one warp joins."""
    return n // 152 + 1 + 32 + 304 // 8 + 8 + 8


def check_backward(layer, dy, s, stats, w, ds, rms, out, bias):
    T = s.dtype
    st = f64(stats)
    want = R.norm_backward(f64(dy), f64(s), st[0], st[1], f64(w), None if ds is None else f64(ds), rms,
                           rows_chain(s.shape[0]))
    within(out[0], *want[0], T)
    within(out[1], *want[1], F32)
    if bias:
        within(out[2], *want[2], F32)
    else:
        assert out[2] is None


@pytest.mark.parametrize("n,H", SIZES)
@pytest.mark.parametrize("form", [(F32, F32, False, True, False), (BF16, F32, False, True, True),
                                  (BF16, BF16, True, False, True), (F32, F32, True, False, True),
                                  (BF16, BF16, False, False, False)],
                         ids=["f32", "bf16-ds", "bf16-rms-ds", "f32-rms-ds", "bf16"])
def test_norm_backward(n, H, form):
    T, W, rms, bias, with_ds = form
    layer, x, _, w, b, eps = norm_case(n, H, T, W, rms, bias, False, seed=20)
    stats = torch.empty((2, n), device="cuda")
    layer(x.cuda(), stats=stats)
    dy = rand(31, n, H).to(T)
    ds = rand(32, n, H).to(T) if with_ds else None
    args = (dy.cuda(), x.cuda(), stats)
    out = layer.backward(*args, ds=None if ds is None else ds.cuda())
    check_backward(layer, dy, x, stats, w, ds, rms, out, bias)
    again = layer.backward(*args, ds=None if ds is None else ds.cuda())
    assert all(a is None if b_ is None else torch.equal(a, b_) for a, b_ in zip(again, out))


# lengths of the groups between the powers of two, both ends of each, more than
# one turn of all groups
BETWEEN = [(900, 1025), (1600, 1529), (800, 2049), (470, 2553), (460, 2560), (310, 4089), (310, 4097),
           (330, 5113), (320, 5120), (310, 5128), (320, 6137), (310, 6144), (170, 6152), (160, 7161),
           (310, 7168), (160, 8185), (5000, 121), (5000, 249), (4999, 256)]


@pytest.mark.parametrize("n,H", BETWEEN)
@pytest.mark.parametrize("T,rms", [(F32, False), (BF16, False), (BF16, True)], ids=["f32", "bf16", "bf16-rms"])
def test_norm_groups_between_powers_of_two(n, H, T, rms):
    """Chains of a row: 16 values of a thread, five steps in a warp, five steps
    (or five warps) more: fewer than R.row_chain's."""
    layer, x, res, w, b, eps = norm_case(n, H, T, F32, rms, not rms, True, seed=50)
    stats = torch.empty((2, n), device="cuda")
    y, s = layer(x.cuda(), res.cuda(), stats=stats)
    check_norm(layer, x, res, w, b, eps, rms, y, s, stats)
    check_norm(layer, s.cpu(), None, w, b, eps, rms, layer(s), None, None)
    dy, s = rand(51, n, H).to(T), s.cpu()
    for ds in (None, res):
        out = layer.backward(dy.cuda(), s.cuda(), stats, None if ds is None else ds.cuda())
        check_backward(layer, dy, s, stats, w, ds, rms, out, not rms)


# rows of several CTAs: two to eight of them, a few rows and more than one turn
# of all clusters, odd lengths in every phase, both sides of the last length
CLUSTERS = [(1, 8200), (200, 8193), (170, 12296), (90, 16383), (161, 16384), (155, 16385), (7, 24576),
            (60, 24577), (1, 32769), (150, 32768), (9, 40003), (8, 57344), (41, 65528), (37, 65529),
            (40, 65536), (3, 65537)]


@pytest.mark.parametrize("n,H", CLUSTERS)
@pytest.mark.parametrize("T,rms", [(F32, False), (BF16, False), (BF16, True)], ids=["f32", "bf16", "bf16-rms"])
def test_norm_rows_of_several_ctas(n, H, T, rms):
    """Sums over a cluster have shorter chains than R.row_chain's: eight values
    of a thread, five steps in a warp, eight warps' sums, five steps.  A cluster
    takes at most n / 8 + 1 rows, and the sums of up to 76 of them are joined in
    chains of 3 + 5: fewer than rows_chain's."""
    layer, x, res, w, b, eps = norm_case(n, H, T, F32, rms, not rms, True, seed=40)
    stats = torch.empty((2, n), device="cuda")
    y, s = layer(x.cuda(), res.cuda(), stats=stats)
    check_norm(layer, x, res, w, b, eps, rms, y, s, stats)
    y2 = layer(s)
    check_norm(layer, s.cpu(), None, w, b, eps, rms, y2, None, None)
    dy, s = rand(41, n, H).to(T), s.cpu()
    for ds in (None, res):
        args = (dy.cuda(), s.cuda(), stats, None if ds is None else ds.cuda())
        out = layer.backward(*args)
        check_backward(layer, dy, s, stats, w, ds, rms, out, not rms)
        again = layer.backward(*args)
        assert all(p is None if q is None else torch.equal(p, q) for p, q in zip(again, out))


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("H", [64, 256, 2048])
def test_norm_rows_apart_and_off_alignment(T, H):
    """Rows inside a wider buffer, and rows that begin off 16 bytes: the values
    of contiguous, aligned ones (a vector and a scalar form may add in another
    order, so against the float64 form)."""
    n = 37
    for pad, off in ((64, 0), (8, 8), (3, 1), (0, 1), (0, 3)):
        wide = (rand(1, n * (H + pad) + off + 8)).to(T).cuda()
        x = wide[off:off + n * (H + pad)].view(n, H + pad)[:, :H]
        w_buf = (1 + rand(4, H + 8, std=0.3)).cuda()
        w, b = w_buf[off:off + H], w_buf[8 - off:8 - off + H].clone()
        layer = M().LayerNorm(w, b, dtype=T)
        stats = torch.empty((2, n), device="cuda")
        y, s = layer(x, x, stats=stats)
        check_norm(layer, x.cpu(), x.cpu(), w.cpu(), b.cpu(), 1e-5, False, y, s, stats)
        dy = rand(7, n, H + pad).to(T).cuda()[:, :H]
        out = layer.backward(dy, s, stats, ds=x)
        check_backward(layer, dy.cpu(), s.cpu(), stats, w.cpu(), x.cpu(), False, out, True)
        out2 = torch.empty(n * H + 8, dtype=T, device="cuda")[off:off + n * H].view(n, H)
        assert torch.equal(layer(x, x, y=out2)[0], out2)
        check_norm(layer, x.cpu(), x.cpu(), w.cpu(), b.cpu(), 1e-5, False, out2, s, None)


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("H", [33, 2048, 40000])
def test_norm_large_mean(T, H):
    """A mean far above the deviation: the deviations are taken before the squares."""
    x = (rand(1, 9, H) + 300.0).to(T)
    layer, x, _, w, b, eps = norm_case(9, H, T, F32, False, True, False, x=x)
    stats = torch.empty((2, 9), device="cuda")
    check_norm(layer, x, None, w, b, eps, False, layer(x.cuda(), stats=stats), None, stats)


def test_norm_constant_and_zero_rows():
    for rms in (False, True):
        for H in (8, 100, 2048, 20000):
            x = torch.zeros((3, H))
            x[1] = 5.0
            layer, x, _, w, b, eps = norm_case(3, H, F32, F32, rms, True, False, x=x)
            stats = torch.empty((2, 3), device="cuda")
            y = layer(x.cuda(), stats=stats)
            assert torch.isfinite(y).all()
            assert torch.equal(y[0].cpu(), b)
            check_norm(layer, x, None, w, b, eps, rms, y, None, stats)
            out = layer.backward(torch.ones_like(y), x.cuda(), stats)
            assert all(torch.isfinite(t).all() for t in out)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("H", [8, 64, 136, 1030, 2048, 20000])
def test_norm_keeps_a_bad_value_in_its_row(bad, H):
    for T in (F32, BF16):
        layer, x, _, w, b, eps = norm_case(50, H, T, F32, False, True, False)
        want = layer(x.cuda())
        x[11, H // 2] = bad
        got = layer(x.cuda())
        assert torch.isnan(got[11].float()).all()
        keep = torch.arange(50) != 11
        assert torch.equal(got[keep.cuda()], want[keep.cuda()])


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("H", [9, 121, 257, 1030, 2049, 4099, 5121, 7169, 8201, 16390])
def test_norm_bad_values_at_a_rows_ends(T, H):
    """NaN at both ends of a row, beside the neighbouring rows' ends: no other
    row's results change, with residual and in the gradients of the rows."""
    n = 400 if H < 3000 else 170
    layer, x, res, w, b, eps = norm_case(n, H, T, F32, False, True, True)
    dy, ds = rand(61, n, H).to(T), rand(62, n, H).to(T)
    stats = torch.empty((2, n), device="cuda")

    def run():
        y, s = layer(x.cuda(), res.cuda(), stats=stats)
        return y, s, layer.backward(dy.cuda(), s, stats, ds=ds.cuda())[0]

    want = run()
    keep = torch.ones(n, dtype=torch.bool)
    for row, t in ((0, x), (7, res), (n // 2, dy), (n // 2 + 3, ds), (n - 1, x)):
        t[row, 0] = t[row, -1] = math.nan
        keep[row] = False
    for got, clean in zip(run(), want):
        assert torch.equal(got[keep.cuda()], clean[keep.cuda()])


def test_norm_squares_beyond_float32():
    layer, x, _, w, b, eps = norm_case(3, 256, F32, F32, False, True, False)
    x[1] *= 1e25
    y = layer(x.cuda()).cpu()
    assert torch.equal(y[1], b) and torch.isfinite(y).all()


def test_norm_no_rows():
    layer, *_ = norm_case(2, 64, BF16, F32, False, True, False)
    x = torch.empty((0, 64), dtype=BF16, device="cuda")
    stats = torch.empty((2, 0), device="cuda")
    y, s = layer(x, x, stats=stats)
    assert y.shape == s.shape == (0, 64)
    dx, dw, db = layer.backward(x, x, stats, dweight=torch.ones(64, device="cuda"),
                                dbias=torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_norm_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31 of the first one."""
    n, H = 2 ** 31 // 4096 + 9, 4096
    x = torch.zeros((n, H), dtype=BF16, device="cuda")
    last = rand(1, 7, H).to(BF16)
    x[-7:] = last.cuda()
    layer = M().LayerNorm(torch.ones(H, device="cuda"), dtype=BF16)
    stats = torch.empty((2, n), device="cuda")
    y = layer(x, stats=stats)
    small = torch.empty((2, 7), device="cuda")
    assert torch.equal(y[-7:], layer(last.cuda(), stats=small))
    assert torch.equal(stats[:, -7:], small) and not y[0].any()
    dy = torch.zeros_like(x)
    dy[-7:] = rand(2, 7, H).to(BF16).cuda()
    dx, dw, _ = layer.backward(dy, x, stats, dx=y)
    want = layer.backward(dy[-7:], last.cuda(), small)
    assert torch.equal(dx[-7:], want[0])
    # the same terms, spread over the ranges in another way
    tol = 2 * 20 * R.U32 * (f64(dy[-7:]) * ((f64(last) - f64(small)[0][:, None]) * f64(small)[1][:, None])).abs().sum(0)
    assert ((f64(dw) - f64(want[1])).abs() <= tol).all()


def test_norm_gradients_against_differences():
    """Through the kernels alone: central differences of L = <y, dy> along a
    random direction of each argument, step h.  L's float32 error is within
    u sum|y dy| * 8 at either end; the third derivative of a norm of rows of
    unit size is of the order of one times the direction's cubed size per row,
    so h^2 times sum over rows of |dy| |direction|^3 / sqrt(H) bounds the rest."""
    n, H, h = 40, 256, 2.0 ** -8
    for rms in (False, True):
        layer, x, _, w, b, eps = norm_case(n, H, F32, F32, rms, True, False, x=rand(8, n, H))
        dy = rand(9, n, H)
        stats = torch.empty((2, n), device="cuda")
        y = layer(x.cuda(), stats=stats)
        dx, dw, db = layer.backward(dy.cuda(), x.cuda(), stats)
        noise = 2 * 8 * R.U32 * float((f64(y) * dy.double()).abs().sum()) / (2 * h)
        for arg, grad in ((x, dx), (w, dw), (b, db)):
            way = torch.randn(arg.shape, generator=gen(10))
            ends = []
            for sign in (h, -h):
                at = [(a + sign * way if a is arg else a) for a in (x, w, b)]
                moved = M().LayerNorm(at[1].cuda(), at[2].cuda(), eps=eps, rms=rms)
                ends.append(float((f64(moved(at[0].cuda())) * dy.double()).sum()))
            want = float((f64(grad) * way.double()).sum())
            # the moved arguments are themselves rounded: u of their size against h
            moves = float((f64(grad).abs() * arg.double().abs()).sum()) * R.U32 / h
            curve = h * h * float(dy.double().norm(dim=1).sum()) * 8 if arg is x else 0.0
            assert abs((ends[0] - ends[1]) / (2 * h) - want) <= noise + moves + curve


# ----------------------------------------------------------- gradient norm
@pytest.mark.parametrize("sizes", [(1,), (5, 0, 2049), (2048, 4096, 3), tuple(range(1, 60)),
                                   tuple(37 * i % 3001 for i in range(1300)), tuple(range(1, 130)), (3_000_001, 7, 500_000),
                                   (0, 0)])
def test_grad_norm(sizes):
    line = rand(1, sum(sizes) + 1, std=3.0).cuda()[1:]  # views at any element
    grads = [t if i % 3 else t.to(BF16) for i, t in enumerate(line.split(list(sizes)))]
    total = math.sqrt(sum(float(f64(t).square().sum()) for t in grads))
    for most in (math.inf, 1.0, total * 2 + 1):
        norm, factor = M().GradNorm(grads)(most)
        # nine roundings of a term and its short sum, the rest in double; a root halves them
        assert abs(float(norm) - total) <= (4.5 + 1) * R.U32 * total
        want = min(1.0, most / (total + 1e-6))
        assert abs(float(factor) - want) <= (5.5 + 4) * R.U32 * want


def test_grad_norm_bad_values():
    g = [torch.ones(5000, device="cuda"), torch.ones(3, device="cuda")]
    call = M().GradNorm(g)
    g[0][17] = math.inf
    assert [float(t) for t in call(1.0)] == [math.inf, 0.0]
    g[0][17] = 1e25  # its square is beyond float32
    assert [float(t) for t in call(1.0)] == [math.inf, 0.0]
    g[1][2] = math.nan
    assert all(math.isnan(float(t)) for t in call(1.0))


# ------------------------------------------------------------------- AdamW
B1, B2, EPS, LR, WD = 0.9, 0.95, 1e-8, 3e-3, 0.1


class Plain:
    """The same step on CPU copies: moments in float32, in the
    interface's operations;
    parameters in float64 with their bound."""

    def __init__(self, opt, state):
        n = [p.numel() for p in opt.params]
        self.state, self.n = state, n
        self.p = [f64(p if w is None else w) for p, w in zip(opt.params, opt.masters)]
        self.err = [torch.zeros_like(p) for p in self.p]
        self.m = [torch.zeros(R.blocks(p.float()).shape) for p in self.p]
        self.v = [t.clone() for t in self.m]
        self.ms = [torch.zeros(len(t)) for t in self.m]
        self.vs = [torch.zeros(len(t)) for t in self.m]

    def step(self, t, grads, lr, decay, factor):
        for i, g in enumerate(grads):
            g = R.blocks(g.detach().cpu().float())
            if factor is not None:
                g = g * torch.tensor(factor, dtype=F32)
            m, v = self.m[i], self.v[i]
            if self.state == E4M3:
                m, v = R.decode(m, self.ms[i]), R.decode(v, self.vs[i])
                v = v * v
            m, v, root = R.adamw_moments(g, m, v, B1, B2)
            shape, k = self.p[i].shape, self.n[i]
            flat = lambda x: x.reshape(-1)[:k].view(shape)  # noqa: E731
            self.p[i], tol = R.adamw_param(self.p[i], flat(m), flat(v), lr, decay[i], B1, B2, EPS, t)
            self.err[i] = self.err[i] * (1 + 1e-3) + tol
            if self.state == E4M3:
                (m, self.ms[i]), (v, self.vs[i]) = R.encode(m, False), R.encode(root, True)
            self.m[i], self.v[i] = m, v

    def check(self, opt):
        for i, (p, w) in enumerate(zip(opt.params, opt.masters)):
            if self.n[i] == 0:
                continue
            b, e = opt.offsets[i], opt.offsets[i] + len(self.m[i])
            live = torch.arange(256 * len(self.m[i])).view(-1, 256) < self.n[i]
            for name, want in (("m", self.m[i]), ("v", self.v[i])):
                got = getattr(opt, name)[b:e].cpu().float()
                assert not got[~live].any()
                assert torch.equal(torch.nan_to_num(got[live], 7e30), torch.nan_to_num(want.float()[live], 7e30)), (i, name)
            if self.state == E4M3:
                assert torch.equal(opt.m_scale[b:e].cpu(), self.ms[i])
                assert torch.equal(opt.v_scale[b:e].cpu(), self.vs[i])
            if w is not None:
                within(w, self.p[i], self.err[i], F32)
                assert torch.equal(p, w.to(p.dtype))
            else:
                within(p, self.p[i], self.err[i], p.dtype)


SHAPES = [(1,), (255,), (256,), (257,), (3, 5, 7), (2048,), (2049,), (100, 33), (7, 4096), (30011,)]


def adamw_case(state, dtype, grad, masters, shapes=SHAPES, off=0, decay=WD):
    def make(i, s, dt, std):
        n = math.prod(s)
        buf = torch.empty(n + off, dtype=dt, device="cuda")
        buf[off:] = rand(i, n, std=std).to(dt).cuda()
        return buf[off:].view(s)
    params = [make(i, s, dtype, 0.02) for i, s in enumerate(shapes)]
    grads = [make(50 + i, s, grad, 10.0 ** -(i % 5)) for i, s in enumerate(shapes)]
    grads[-1].view(-1)[-700:] = 0  # never any gradient
    return M().AdamW(params, grads, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay, state=state,
                     masters=masters)


@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
@pytest.mark.parametrize("kind", [(F32, F32, None, 0), (BF16, F32, True, 0), (BF16, BF16, None, 0),
                                  (F32, BF16, None, 1), (BF16, F32, True, 3)],
                         ids=["f32", "master", "bf16", "bf16-grad-off", "master-off"])
def test_adamw_steps(state, kind):
    """Three steps with gradients of their own.  A parameter held in bf16 is
    compared after each step from its own rounded value."""
    dtype, grad, masters, off = kind
    opt = adamw_case(state, dtype, grad, masters, off=off, decay=[0.0, 0.1] * 5)
    plain = Plain(opt, state)
    for t in (1, 2, 3):
        factor = None if t == 2 else torch.tensor([0.37], device="cuda")
        lr = LR if t < 3 else 2 * LR
        opt.step(lr=lr, grad_scale=factor)
        plain.step(t, opt.grads, lr, [0.0, 0.1] * 5, None if t == 2 else 0.37)
        plain.check(opt)
        assert opt.steps == t
        if masters is None and dtype == BF16:
            plain.p = [f64(p) for p in opt.params]
            plain.err = [torch.zeros_like(p) for p in plain.p]
        for i, g in enumerate(opt.grads):
            g.copy_(rand(100 * t + i, *g.shape, std=10.0 ** -(i % 4)))


@pytest.mark.parametrize("count", [47, 48, 49, 384, 385, 900])
@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
def test_adamw_many_tensors(count, state):
    """More tensors than one launch takes, empty ones among them."""
    shapes = [(0,) if i % 13 == 5 else (1 + 37 * i % 700,) for i in range(count)]
    shapes[-1] = (900,)
    opt = adamw_case(state, F32, F32, None, shapes)
    plain = Plain(opt, state)
    for t in (1, 2):
        opt.step()
        plain.step(t, opt.grads, LR, [WD] * count, None)
    plain.check(opt)
    assert opt.steps == 2


@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
def test_adamw_all_empty_counts_a_step(state):
    opt = adamw_case(state, F32, F32, None, [(700,)])
    empty = M().AdamW([torch.empty(0, device="cuda")], [torch.empty(0, device="cuda")], state=state)
    empty.step()
    assert empty.steps == 1 and opt.steps == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
def test_adamw_keeps_a_bad_gradient_where_it_is(state, bad):
    opt, good = (adamw_case(state, F32, F32, None, [(700,)]) for _ in range(2))
    opt.grads[0][300] = bad
    good.grads[0][300] = 0
    for _ in range(2):
        opt.step()
        good.step()
    other = (torch.arange(700) != 300).cuda()
    assert torch.equal(opt.params[0][other], good.params[0][other])
    if state == E4M3:
        code = opt.m.float().view(-1)
        assert torch.isnan(code[300]) and torch.isnan(opt.v.float().view(-1)[300])
        assert torch.equal(code[:700][other], good.m.float().view(-1)[:700][other])
        assert torch.equal(opt.m_scale, good.m_scale) and torch.equal(opt.v_scale, good.v_scale)


def test_adamw_small_roots_keep_a_code():
    """Second moments far below their block's largest do not become zero."""
    g = torch.full((256,), 1e-7)
    g[0] = 1e3
    opt = M().AdamW([torch.zeros(256, device="cuda")], [g.cuda()], state=E4M3)
    opt.step()
    assert (opt.v.float() > 0).all() and not opt.m.float()[0, 1:].any()
    opt.step()
    assert torch.isfinite(opt.params[0]).all()


def test_adamw_far_steps():
    """The bias correction of late steps, and of betas of zero."""
    for steps in (1, 1000, 10 ** 7):
        opt = adamw_case(F32, F32, F32, None, [(500,)])
        opt.load_state_dict({"steps": steps, "m": opt.m, "v": opt.v, "m_scale": None, "v_scale": None})
        plain = Plain(opt, F32)
        for t in (1, 2):
            opt.step()
            plain.step(steps + t, opt.grads, LR, [WD], None)
        plain.check(opt)
        assert opt.steps == steps + 2
    p, g = torch.ones(300, device="cuda"), torch.full((300,), -2.0, device="cuda")
    opt = M().AdamW([p], [g], lr=0.5, betas=(0.0, 0.0), weight_decay=0.0)
    opt.step()
    # m = g, v = g^2: one step of lr against the sign
    assert ((p - 1.5).abs() <= 8 * R.U32 * 1.5 + 1e-8).all()


def test_adamw_resumes():
    a, b = (adamw_case(E4M3, BF16, F32, True) for _ in range(2))
    for _ in range(3):
        a.step()
    d = a.state_dict()
    for to, src in zip(b.params, a.params):
        to.copy_(src)
    b.load_state_dict(d)
    a.step()
    b.step()
    assert a.steps == b.steps == 4
    for x, y in zip([*a.params, *a.masters, a.m_scale, a.v_scale], [*b.params, *b.masters, b.m_scale, b.v_scale]):
        assert torch.equal(x, y)
    assert torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))
    with pytest.raises(ValueError):
        adamw_case(F32, BF16, F32, True).load_state_dict(d)


@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
def test_adamw_past_32_bits(state):
    """A tensor of more than 2^31 values: the last ones as in a small tensor."""
    n = 2 ** 31 + 256 * 9 + 5
    tail = 256 + 5
    p, g = (torch.zeros(n, dtype=BF16, device="cuda") for _ in range(2))
    sp, sg = (rand(i, tail, std=0.1).to(BF16).cuda() for i in (1, 2))
    p[-tail:], g[-tail:] = sp, sg
    big, small = M().AdamW([p], [g], state=state), M().AdamW([sp], [sg], state=state)
    for _ in range(2):
        big.step()
        small.step()
    assert torch.equal(p[-tail:], sp) and not p[:1000].any()
    assert torch.equal(big.m[-2:].view(torch.uint8), small.m.view(torch.uint8))
    norm, _ = M().GradNorm([g])()
    assert abs(float(norm) - float(f64(sg).norm())) <= 6 * R.U32 * float(norm)


# ------------------------------------------------------- streams and graphs
def test_calls_on_other_streams():
    layer, x, res, w, b, eps = norm_case(300, 520, BF16, F32, False, True, True)
    x, res = x.cuda(), res.cuda()
    stats = torch.empty((2, 300), device="cuda")
    y, s = layer(x, res, stats=stats)
    want = (y, s, *layer.backward(x, s, stats, ds=res))
    grads = [want[3], want[4]]
    norm = M().GradNorm(grads)
    first = norm(1.0)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for st in streams:
            y, s = layer(x, res, stream=st)
            got.append((y, s, *layer.backward(x, want[1], stats, ds=res, stream=st), *norm(1.0, stream=st)))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b_) for a, b_ in zip(g, (*want, *first)))


def test_an_optimizer_made_on_a_side_stream():
    side = torch.cuda.Stream()
    a = adamw_case(E4M3, BF16, F32, True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b = adamw_case(E4M3, BF16, F32, True)
    torch.cuda.current_stream().wait_stream(side)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    a.step()
    b.step(stream=other)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params)) and b.steps == 1


def test_a_captured_step_counts_on():
    """Norm, backward, clipping and step as one graph: each replay is one more
    step, with the learning rate and the inputs that its buffers then hold."""
    def make():
        layer, x, _, w, b, eps = norm_case(70, 264, BF16, F32, False, True, False)
        bufs = dict(dw=torch.zeros(264, device="cuda"), db=torch.zeros(264, device="cuda"))
        opt = M().AdamW([layer.weight, layer.bias], [bufs["dw"], bufs["db"]], lr=9.0, state=E4M3)
        return layer, x.cuda(), bufs, opt, M().GradNorm([bufs["dw"], bufs["db"]]), torch.full((1,), LR, device="cuda")

    def step(layer, x, bufs, opt, norm, lr):
        stats = torch.empty((2, 70), device="cuda")
        y = layer(x, stats=stats)
        layer.backward(y, x, stats, dweight=bufs["dw"], dbias=bufs["db"])
        opt.step(lr=lr, grad_scale=norm(0.5)[1])
    eager, captured = make(), make()
    step(*eager)
    step(*captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured)
    assert captured[3].steps == 1
    for i in range(3):
        for side in (eager, captured):
            side[5].fill_(LR * (i + 1))
            side[1].copy_(rand(60 + i, 70, 264))
        step(*eager)
        graph.replay()
    assert captured[3].steps == eager[3].steps == 4
    for a, b in zip(eager[3].params, captured[3].params):
        assert torch.equal(a, b)


def test_two_graphs_of_one_object():
    """Two captured backwards of one norm hold scratch of their own."""
    layer, x, _, w, b, eps = norm_case(400, 1024, BF16, F32, False, True, False)
    xs = [x.cuda(), (2 * x.float() + 1).to(BF16).cuda()]
    stats = [torch.empty((2, 400), device="cuda") for _ in xs]
    for a, s in zip(xs, stats):
        layer(a, stats=s)
    want = [layer.backward(a, a, s) for a, s in zip(xs, stats)]
    graphs, outs = [], []
    for a, s in zip(xs, stats):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.backward(a, a, s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, wnt in zip(outs, want):
        assert all(torch.equal(a, c) for a, c in zip(o, wnt))


def test_c_calls_with_plain_pointers():
    """The C interface as a C program uses it: scratch and results of the caller."""
    m, lib = M(), M()._lib.load()
    n, H = 5, 96
    x, w = rand(1, n, H).cuda(), torch.ones(H, device="cuda")
    y, stats = torch.empty_like(x), torch.empty((2, n), device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    d = m._lib.NormDesc(n, H, 0, 0, 1, 1e-6)
    assert lib.moe_layer_norm(ctypes.byref(d), x.data_ptr(), H, None, 0, w.data_ptr(), None, None,
                              y.data_ptr(), stats.data_ptr(), stream) == 0
    ws = torch.full((lib.moe_layer_norm_backward_workspace_size(ctypes.byref(d)),), 0xff,
                    dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    assert lib.moe_layer_norm_backward(ctypes.byref(d), y.data_ptr(), H, x.data_ptr(), H,
                                       stats.data_ptr(), w.data_ptr(), None, 0, dx.data_ptr(),
                                       dw.data_ptr(), None, ws.data_ptr(), ws.numel(), stream) == 0
    layer = m.LayerNorm(w, eps=1e-6, rms=True)
    assert torch.equal(y, layer(x))
    got = layer.backward(y, x, stats)
    assert torch.equal(dx, got[0]) and torch.equal(dw, got[1])


# ------------------------------------------------- rows of every phase
@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("n,H", [(1, 3), (2, 1), (9, 5), (400, 7), (1300, 9), (153, 121), (1217, 127), (1200, 130),
                                 (161, 1025), (305, 2050), (160, 4093), (310, 8186), (153, 8189), (155, 16379)])
def test_norm_odd_rows_in_many_rounds(n, H, T):
    """Rows that begin at every place within 16 bytes, several to a group, in a
    buffer with nothing behind its last row."""
    layer, x, res, w, b, eps = norm_case(n, H, T, F32, False, True, True, seed=40)
    x, res = x.cuda(), res.cuda()
    stats = torch.empty((2, n), device="cuda")
    y, s = layer(x, res, stats=stats)
    check_norm(layer, x.cpu(), res.cpu(), w, b, eps, False, y, s, stats)
    y, s = layer(x, res[:, :].clone(), stats=stats)
    dy = rand(41, n, H).to(T).cuda()
    out = layer.backward(dy, s, stats, ds=res)
    check_backward(layer, dy.cpu(), s.cpu(), stats, w, res.cpu(), False, out, True)


def test_norm_row_strides_of_unequal_phase():
    """x in a buffer of odd row stride, the result contiguous; and strides of
    one odd phase that are not the length."""
    for T in (F32, BF16):
        for H, strides in ((40, (41, 41)), (40, (41, 48)), (41, (49, 57)), (41, (41, 49)), (33, (35, 35))):
            n = 700
            x, res = (rand(i, n, st).to(T).cuda()[:, :H] for i, st in enumerate(strides))
            layer, _, _, w, b, eps = norm_case(2, H, T, F32, False, True, True)
            stats = torch.empty((2, n), device="cuda")
            y, s = layer(x, res, stats=stats)
            check_norm(layer, x.cpu(), res.cpu(), w, b, eps, False, y, s, stats)
            out = layer.backward(x, s, stats, ds=res)
            check_backward(layer, x.cpu(), s.cpu(), stats, w, res.cpu(), False, out, True)


# ------------------------------------------------------------------ scratch
def test_calls_of_threads_on_one_stream():
    """Threads' backward calls and gradient norms, of unequal sizes, share a
    stream's scratch memory."""
    import threading
    work = []
    for i, (n, H) in enumerate(((400, 2048), (3, 40), (1200, 136), (90, 1031))):
        layer, x, _, w, b, eps = norm_case(n, H, BF16, F32, False, True, False, seed=70 + i)
        x, stats = x.cuda(), torch.empty((2, n), device="cuda")
        layer(x, stats=stats)
        norm = M().GradNorm([x, stats])
        work.append((layer, x, stats, norm, layer.backward(x, x, stats) + norm(1.0), []))
    torch.cuda.synchronize()

    def calls(layer, x, stats, norm, want, got):
        for _ in range(25):
            got.append(layer.backward(x, x, stats) + norm(1.0))
    threads = [threading.Thread(target=calls, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for *_, want, got in work:
        assert len(got) == 25
        assert all(torch.equal(a, c) for g in got for a, c in zip(g, want))


def test_scratch_grows_between_calls():
    """A larger call behind a smaller one on the same streams, eager and captured."""
    small, large = ((norm_case(n, H, BF16, F32, False, True, False)) for n, H in ((2, 64), (700, 8192)))
    want = []
    for layer, x, *_ in (small, large):
        x = x.cuda()
        stats = torch.empty((2, len(x)), device="cuda")
        layer(x, stats=stats)
        want.append((layer, x, stats, layer.backward(x, x, stats)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for layer, x, stats, out in want + want[::-1]:
            got = layer.backward(x, x, stats, stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(got, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [layer.backward(x, x, stats) for layer, x, stats, _ in want]
    for _ in range(2):
        graph.replay()
        want[1][0].backward(*want[1][1:2] * 2, want[1][2])
    torch.cuda.synchronize()
    for got, (*_, out) in zip(outs, want):
        assert all(torch.equal(a, c) for a, c in zip(got, out))


# ------------------------------------------------- mixed lists of parameters
@pytest.mark.parametrize("state", [F32, E4M3], ids=["f32", "e4m3"])
def test_adamw_mixed_kinds(state):
    """Parameters and gradients of every pair of types in one optimizer, with
    masters for some of either type, more of one kind than a launch takes, and
    tensors off 16 bytes beside aligned ones."""
    kinds = [(F32, F32, False), (BF16, F32, True), (BF16, BF16, False), (F32, BF16, True), (BF16, BF16, True),
             (BF16, F32, False), (F32, F32, True), (F32, BF16, False)] + [(BF16, F32, True)] * 60
    params, grads, masters = [], [], []
    for i, (pt, gt, has) in enumerate(kinds):
        n, off = 1 + 613 * i % 2900, i % 3
        p = torch.empty(n + off, dtype=pt, device="cuda")[off:]
        p.copy_(rand(i, n, std=0.05))
        params.append(p)
        grads.append(rand(100 + i, n).to(gt).cuda())
        masters.append(p.clone().float() if has else None)
    opt = M().AdamW(params, grads, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, state=state, masters=masters)
    plain = Plain(opt, state)
    for t in (1, 2):
        for i, (p, w) in enumerate(zip(params, masters)):
            if w is None and p.dtype == BF16:
                plain.p[i], plain.err[i] = f64(p), torch.zeros(p.shape, dtype=torch.float64)
        opt.step()
        plain.step(t, grads, LR, [WD] * len(kinds), None)
        plain.check(opt)
    assert opt.steps == 2


def test_adamw_leaves_what_lies_between_tensors():
    """Parameters, gradients and masters as parts of larger buffers."""
    for state in (F32, E4M3):
        line = torch.full((3, 2000), 7.0, device="cuda")
        parts = [slice(3, 4), slice(10, 700), slice(701, 1999)]
        params, grads = [line[0, p] for p in parts], [line[1, p] for p in parts]
        opt = M().AdamW(params, grads, state=state)
        opt.step()
        touched = torch.zeros(2000, dtype=torch.bool)
        for p in parts:
            touched[p] = True
        assert (line[0].cpu()[~touched] == 7).all() and (line[0].cpu()[touched] != 7).all()
        assert (line[1:] == 7).all()


@pytest.mark.parametrize("T", [F32, BF16])
def test_norm_gaps_between_rows(T):
    """What lies between rows does not reach the results, NaN included, and
    stays as it was where a result lies in a larger buffer."""
    for H, pad in ((40, 8), (41, 8), (1031, 5), (2048, 16), (8190, 3), (5, 3)):
        n = 170
        wide = torch.full((n, H + pad), math.nan)
        wide[:, :H] = rand(1, n, H)
        x = wide.to(T).cuda()[:, :H]
        layer, _, _, w, b, eps = norm_case(2, H, T, F32, False, True, True)
        stats = torch.empty((2, n), device="cuda")
        buf = torch.full((n * H + 16,), 7.0, dtype=T, device="cuda")
        y, s = layer(x, x, y=buf[8:8 + n * H].view(n, H), stats=stats)
        assert (buf[:8] == 7).all() and (buf[8 + n * H:] == 7).all()
        check_norm(layer, x.cpu(), x.cpu(), w, b, eps, False, y, s, stats)
        out = layer.backward(x, s, stats, ds=x, dx=buf[8:8 + n * H].view(n, H))
        assert (buf[:8] == 7).all() and (buf[8 + n * H:] == 7).all()
        check_backward(layer, x.cpu(), s.cpu(), stats, w, x.cpu(), False, out, True)


def test_optimizer_takes_leaf_parameters():
    """Parameters of a module: written in place, no graph kept."""
    p = torch.nn.Parameter(torch.ones(300, device="cuda", dtype=BF16))
    opt = M().AdamW([p], [torch.ones(300, device="cuda")], lr=0.25, weight_decay=0.0, masters=True)
    opt.step()
    assert not opt.masters[0].requires_grad and torch.equal(p.detach(), torch.full_like(p, 0.75))

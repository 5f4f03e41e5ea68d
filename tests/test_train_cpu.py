"""Refusals of the training calls and the plain forms' own pins, without a GPU:
every bad argument is answered before any CUDA call, through the C ABI (fake
pointers, never dereferenced) and through the Python classes (CPU tensors)."""
import ctypes
import math
import os
import shutil

import pytest
import torch

from tests import train_reference as R

pytestmark = pytest.mark.skipif(
    not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")),
    reason="CUDA toolkit not installed")

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 1 << 20          # a fake, well aligned pointer
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from top_routing_dispatch_gb300 import build as B
    B.build()
    from top_routing_dispatch_gb300 import _lib
    return _lib.load()


# ------------------------------------------------------------------- norm
def desc(**kw):
    from top_routing_dispatch_gb300._lib import NormDesc
    return NormDesc(**{**dict(n=4, H=64, dtype=1, weight_dtype=0, rms=0, eps=1e-5), **kw})


def forward(lib, d=None, x=P, xs=64, res=None, rs=64, w=P, b=None, s=None, y=P, stats=None):
    return lib.moe_layer_norm(ctypes.byref(desc() if d is None else d), x, xs, res, rs, w, b, s, y,
                              stats, None)


def backward(lib, d=None, dy=P, dys=64, s=P, ss=64, stats=P, w=P, ds=None, dss=64, dx=P, dw=P,
             db=None, ws=P, nbytes=1 << 40):
    return lib.moe_layer_norm_backward(ctypes.byref(desc() if d is None else d), dy, dys, s, ss,
                                       stats, w, ds, dss, dx, dw, db, ws, nbytes, None)


BAD_NORMS = [
    (dict(n=-1), INVALID), (dict(H=0), INVALID), (dict(H=-8), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=7), INVALID), (dict(weight_dtype=2), INVALID),
    (dict(dtype=0, weight_dtype=1), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(H=(1 << 20) + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", BAD_NORMS, ids=str)
def test_bad_norm_descriptions(lib, bad, code):
    d = desc(**bad)
    assert forward(lib, d) == code and backward(lib, d) == code
    assert lib.moe_layer_norm_backward_workspace_size(ctypes.byref(d)) == 0


def test_null_norm_description(lib):
    null = ctypes.POINTER(type(desc()))()
    assert lib.moe_layer_norm(null, P, 0, None, 0, P, None, None, P, None, None) == INVALID
    assert lib.moe_layer_norm_backward(null, P, 0, P, 0, P, P, None, 0, P, P, None, P, 1, None) == INVALID
    assert lib.moe_layer_norm_backward_workspace_size(null) == 0


def test_norm_refusals(lib):
    for kw in (dict(x=None), dict(y=None), dict(w=None), dict(x=P + 1), dict(y=P + 1), dict(w=P + 2),
               dict(b=P + 2), dict(stats=P + 2), dict(xs=63), dict(xs=0), dict(xs=-64),
               dict(res=P), dict(s=P), dict(res=P, s=P + 1), dict(res=P + 1, s=P),
               dict(res=P, s=P, rs=32)):
        assert forward(lib, **kw) == INVALID, kw
    assert forward(lib, desc(dtype=0, weight_dtype=0), x=P + 2) == INVALID
    assert forward(lib, desc(n=0), x=None, y=None, w=None) == 0


def test_norm_backward_refusals(lib):
    need = lib.moe_layer_norm_backward_workspace_size(ctypes.byref(desc()))
    assert need > 0
    assert backward(lib, nbytes=need - 1) == WORKSPACE
    for kw in (dict(dy=None), dict(s=None), dict(stats=None), dict(w=None), dict(dx=None),
               dict(dw=None), dict(ws=None), dict(dy=P + 1), dict(s=P + 1), dict(stats=P + 2),
               dict(w=P + 2), dict(ds=P + 1), dict(dx=P + 1), dict(dw=P + 2), dict(db=P + 2),
               dict(ws=P + 8), dict(dys=63), dict(ss=0), dict(ds=P, dss=10)):
        assert backward(lib, **kw) == INVALID, kw
    # the gradients are written even without rows
    assert backward(lib, desc(n=0), dw=None) == INVALID


# -------------------------------------------------------- norm of gradients
def tensors(*items):
    from top_routing_dispatch_gb300._lib import TensorDesc
    return (TensorDesc * len(items))(*[TensorDesc(*i) for i in items])


def grad_norm(lib, t=((P, 10, 0), (P, 10, 1)), count=None, most=1.0, norm=P, factor=P, ws=P,
              nbytes=1 << 40):
    return lib.moe_grad_norm(tensors(*t) if t else None, len(t) if count is None else count, most,
                             norm, factor, ws, nbytes, None)


def test_grad_norm_refusals(lib):
    assert lib.moe_grad_norm_workspace_size(-1) == 0
    assert lib.moe_grad_norm_workspace_size(65537) == 0
    need = lib.moe_grad_norm_workspace_size(2)
    assert 0 < need <= lib.moe_grad_norm_workspace_size(65536)
    assert grad_norm(lib, nbytes=need - 1) == WORKSPACE
    for t in (((None, 10, 0),), ((P + 2, 10, 0),), ((P + 1, 10, 1),), ((P, -1, 0),), ((P, 10, 2),)):
        assert grad_norm(lib, t) == INVALID, t
    for kw in (dict(t=(), count=1), dict(count=-1), dict(most=0.0), dict(most=-1.0),
               dict(most=math.nan), dict(norm=None), dict(factor=None), dict(norm=P + 2),
               dict(factor=P + 1), dict(ws=None), dict(ws=P + 16)):
        assert grad_norm(lib, **kw) == INVALID, kw
    assert grad_norm(lib, ((P, (1 << 40) + 1, 0),)) == UNSUPPORTED
    assert grad_norm(lib, ((P, 1 << 40, 0), (P, 1, 0))) == UNSUPPORTED
    assert grad_norm(lib, ((P, 4, 0),), count=65537) == UNSUPPORTED


# ------------------------------------------------------------------- AdamW
def opt(**kw):
    from top_routing_dispatch_gb300._lib import AdamWDesc
    return AdamWDesc(**{**dict(state_dtype=0, lr=1e-3, lr_device=None, grad_scale=None, beta1=0.9,
                               beta2=0.99, eps=1e-8), **kw})


def tensor(**kw):
    from top_routing_dispatch_gb300._lib import AdamWTensor
    return AdamWTensor(**{**dict(param=P, master=None, grad=P, m=P, v=P, m_scale=None, v_scale=None,
                                 numel=300, dtype=0, grad_dtype=0, weight_decay=0.1), **kw})


def step(lib, o=None, t=None, count=1, state=P):
    t = tensor() if t is None else t
    return lib.moe_adamw_step(ctypes.byref(opt() if o is None else o), ctypes.byref(t), count,
                              state, None)


def test_adamw_refusals(lib):
    for kw in (dict(state_dtype=1), dict(state_dtype=3), dict(lr=-1e-3), dict(lr=math.nan),
               dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
               dict(beta2=math.nan), dict(eps=0.0), dict(eps=1e-39), dict(eps=-1e-8), dict(eps=math.inf),
               dict(lr_device=P + 2), dict(grad_scale=P + 1)):
        assert step(lib, opt(**kw)) == INVALID, kw
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(numel=-1),
               dict(dtype=2), dict(grad_dtype=2), dict(weight_decay=-0.1),
               dict(weight_decay=math.nan), dict(param=P + 2), dict(master=P + 2), dict(grad=P + 2),
               dict(m=P + 1), dict(v=P + 2), dict(m_scale=P), dict(v_scale=P)):
        assert step(lib, t=tensor(**kw)) == INVALID, kw
    e = opt(state_dtype=2)
    for kw in (dict(), dict(m_scale=P), dict(v_scale=P), dict(m_scale=P, v_scale=P + 2),
               dict(m_scale=P, v_scale=P, m=None)):
        assert step(lib, e, tensor(**kw)) == INVALID, kw
    assert step(lib, state=None) == INVALID and step(lib, state=P + 8) == INVALID
    assert step(lib, count=-1) == INVALID
    assert lib.moe_adamw_step(ctypes.byref(opt()), None, 1, P, None) == INVALID
    assert lib.moe_adamw_step(None, ctypes.byref(tensor()), 1, P, None) == INVALID
    assert step(lib, t=tensor(numel=(1 << 40) + 1)) == UNSUPPORTED
    assert step(lib, count=65537) == UNSUPPORTED
    for b1, b2, n, s in ((1.0, 0.9, 0, P), (0.9, -1.0, 0, P), (0.9, 0.9, -1, P), (0.9, 0.9, 0, None),
                         (0.9, 0.9, 0, P + 4)):
        assert lib.moe_adamw_set_steps(b1, b2, n, s, None) == INVALID


# ------------------------------------------------------------ Python classes
def test_layer_norm_refusals(lib):
    import top_routing_dispatch_gb300 as M
    w = torch.ones(64)
    for kw in (dict(weight=w[None]), dict(weight=w.half()), dict(weight=torch.ones(128)[::2]),
               dict(bias=torch.ones(32)), dict(bias=w.to(BF16)), dict(dtype=torch.float16),
               dict(bias=torch.ones(128)[::2])):
        with pytest.raises(ValueError):
            M.LayerNorm(**{**dict(weight=w), **kw})
    for kw in (dict(weight=w.to(BF16), dtype=F32), dict(eps=-1.0), dict(eps=math.nan),
               dict(weight=torch.ones(0)), dict(weight=torch.ones((1 << 20) + 1))):
        with pytest.raises(M.MoEError):
            M.LayerNorm(**{**dict(weight=w), **kw})
    norm = M.LayerNorm(w, dtype=BF16)
    x, stats = torch.zeros((3, 64), dtype=BF16), torch.zeros((2, 3))
    for kw in (dict(x=x.float()), dict(x=x[0]), dict(x=x[:, :32]), dict(x=x.t().contiguous().t()),
               dict(s=x)):
        with pytest.raises(ValueError):
            norm(**{**dict(x=x), **kw})
    for kw in (dict(dy=x.float()), dict(dy=x[:2]), dict(s=x[:, :32]), dict(ds=x.float()),
               dict(dy=x[0])):
        with pytest.raises(ValueError):
            norm.backward(**{**dict(dy=x, s=x, stats=stats), **kw})


def test_layer_norm_result_refusals(lib, monkeypatch):
    """Given results of another shape, type or order."""
    import top_routing_dispatch_gb300 as M
    from top_routing_dispatch_gb300 import train
    monkeypatch.setattr(train, "_here", lambda *a: None)
    norm = M.LayerNorm(torch.ones(64), torch.ones(64), dtype=BF16)
    plain = M.LayerNorm(torch.ones(64), dtype=BF16)
    x, stats, vec = torch.zeros((3, 64), dtype=BF16), torch.zeros((2, 3)), torch.zeros(64)
    wide = torch.zeros((3, 128), dtype=BF16)[:, :64]
    for kw in (dict(y=x.float()), dict(y=x[:2]), dict(y=wide), dict(residual=x, s=wide),
               dict(residual=x, s=x.float()), dict(residual=x.float()), dict(residual=x[:2]),
               dict(stats=stats.t().contiguous()), dict(stats=stats.double())):
        with pytest.raises(ValueError):
            norm(**{**dict(x=x), **kw})
    for kw in (dict(stats=stats[0]), dict(dx=x.float()), dict(dx=wide), dict(dweight=vec[:32]),
               dict(dweight=vec.to(BF16)), dict(dbias=vec[:32])):
        with pytest.raises(ValueError):
            norm.backward(**{**dict(dy=x, s=x, stats=stats), **kw})
    with pytest.raises(ValueError):
        plain.backward(x, x, stats, dbias=vec)


def test_grad_norm_and_adamw_constructor_refusals(lib):
    import top_routing_dispatch_gb300 as M
    t = torch.zeros((4, 6))
    for bad in ([], [t.half()], [t.t()], [t.double()]):
        with pytest.raises(ValueError):
            M.GradNorm(bad)
    p, g = [torch.zeros(300), torch.zeros((2, 5), dtype=BF16)], [torch.zeros(300), torch.zeros((2, 5))]
    for kw in (dict(params=[]), dict(params=p[:1]), dict(params=[p[0].half(), p[1]]),
               dict(grads=[g[0], g[1].t()]), dict(grads=[g[0], torch.zeros(10)]),
               dict(grads=[g[0][:299], g[1]]), dict(state=BF16), dict(weight_decay=[0.1]),
               dict(weight_decay=-0.1), dict(weight_decay=math.inf), dict(lr=-1.0),
               dict(lr=math.nan), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0),
               dict(masters=[None]), dict(masters=[None, torch.zeros((2, 5), dtype=BF16)]),
               dict(masters=[None, torch.zeros(10)]), dict(params=[p[0], p[0][:10].view(2, 5)]),
               dict(params=[p[0], p[1]], masters=[p[0], None])):
        with pytest.raises(ValueError):
            M.AdamW(**{**dict(params=p, grads=g), **kw})


def calls():
    import top_routing_dispatch_gb300 as M
    norm = M.LayerNorm(torch.ones(64), dtype=BF16)
    x, stats = torch.zeros((3, 64), dtype=BF16), torch.zeros((2, 3))
    one = torch.zeros(1)
    return {
        "norm": lambda: norm(x, y=x.clone()),
        "backward": lambda: norm.backward(x, x, stats, dx=x.clone(), dweight=torch.zeros(64)),
        "grad_norm": lambda: M.GradNorm([torch.zeros(5)])(1.0, norm=one, factor=one.clone()),
        "adamw": lambda: M.AdamW([torch.zeros(5)], [torch.zeros(5)]),
    }


@pytest.mark.parametrize("name", ["norm", "backward", "grad_norm", "adamw"])
def test_calls_refuse_tensors_that_are_not_on_a_gpu(lib, name):
    with pytest.raises(ValueError, match="CUDA"):
        calls()[name]()


@pytest.mark.parametrize("name", ["norm", "backward", "grad_norm", "adamw"])
def test_calls_ask_for_their_device(lib, monkeypatch, name):
    """The library launches on the current device."""
    from top_routing_dispatch_gb300 import decode

    class Reached(Exception):
        pass

    def ready(device):
        raise Reached
    monkeypatch.setattr(decode, "_ready", ready)
    with pytest.raises(Reached):
        calls()[name]()


# ------------------------------------------------ the plain forms themselves
@pytest.mark.parametrize("rms", [False, True])
def test_plain_norm_gradients_against_differences(rms):
    """Central differences of the float64 norm, on every argument: their error
    is of the order of h^2."""
    g = torch.Generator()
    g.manual_seed(3)
    s, w, b, dy, ds = (torch.randn(sh, generator=g, dtype=torch.float64)
                       for sh in ((5, 17), (17,), (17,), (5, 17), (5, 17)))
    eps, h = 1e-3, 1e-5

    def loss(s, w, b):
        return float((R.norm(s, w, b, eps, rms)[0] * dy).sum() + (s * ds).sum())
    _, _, mean, _, r, _ = R.norm(s, w, b, eps, rms)
    got = R.norm_backward(dy, s, mean, r, w, ds, rms, 10)
    for i, (arg, (grad, _)) in enumerate(zip((s, w, b), got)):
        for at in range(arg.numel()):
            ends = []
            for sign in (1, -1):
                moved = arg.clone()
                moved.view(-1)[at] += sign * h
                ends.append(loss(*[moved if j == i else a for j, a in enumerate((s, w, b))]))
            assert abs((ends[0] - ends[1]) / (2 * h) - float(grad.reshape(-1)[at])) < 1e-6


def test_plain_codes_are_within_half_a_step():
    g = torch.Generator()
    g.manual_seed(4)
    x = torch.randn((40, 256), generator=g) * torch.logspace(-30, 20, 40)[:, None]
    x[3] = 0
    x[5, 7] = math.inf
    x[6, 8] = math.nan
    code, scale = R.encode(x, False)
    back = R.decode(code, scale)
    ok = torch.isfinite(x)
    assert torch.isnan(back[~ok]).all() and (back[3] == 0).all()
    top = torch.where(ok, x, torch.zeros(())).abs().amax(1, keepdim=True)
    # half a step of three mantissa bits, or of the smallest code; scale and quotient in float32
    tol = x.abs() * 2.0 ** -4 * (1 + 1e-5) + top / 448 * 2.0 ** -10 * (1 + 1e-5)
    assert ((back - x).abs() <= tol)[ok].all()
    code, scale = R.encode(x.abs(), True)
    assert (code.float()[ok & (x != 0)] > 0).all() and (code.float()[3] == 0).all()

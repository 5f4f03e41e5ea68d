"""The training calls without a GPU, beside test_train_cpu.py: the rounding of
8-bit states, and how calls handle their arguments and memory."""
import ctypes
import math
import os
import shutil

import pytest
import torch

from tests import train_random_reference as Q
from tests import train_reference as R

pytestmark = pytest.mark.skipif(
    not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")),
    reason="CUDA toolkit not installed")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
P = 1 << 20  # a fake, well aligned pointer


# ------------------------------------------------------- rounding of 8-bit states
def test_rounding_refusals():
    import top_routing_dispatch_gb300 as M
    from top_routing_dispatch_gb300 import _lib
    from top_routing_dispatch_gb300 import build as B
    B.build()
    lib = _lib.load()
    t = _lib.AdamWTensor(param=P, grad=P, m=P, v=P, m_scale=P, v_scale=P, numel=300, weight_decay=0.1)
    for state in (0, 2):
        for rounding in (-1, 3):
            o = _lib.AdamWDesc(state_dtype=state, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, rounding=rounding)
            assert lib.moe_adamw_step(ctypes.byref(o), ctypes.byref(t), 1, P, None) == 1
    p, g = [torch.zeros(300)], [torch.zeros(300)]
    for kw in (dict(state=E4M3, rounding="up"), dict(state=E4M3, rounding=True), dict(rounding="random"),
               dict(rounding="nearest")):
        with pytest.raises(ValueError, match="rounding"):
            M.AdamW(p, g, **kw)


def test_plain_random_codes_are_neighbours():
    """A code stays, a value between two codes becomes one of them, and what is
    past the largest becomes the largest."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).float()  # 0 to 448
    chance = torch.arange(0, 1 << 32, 0xFFFFF7)[:, None]
    for f in (Q.random_code, Q.random_root):
        assert torch.equal(f(codes.expand(len(chance), -1), chance), codes.expand(len(chance), -1))
        lo, hi = codes[:-1], codes[1:]
        for part in (0.01, 0.3, 0.5, 0.99):
            got = f((lo + (hi - lo) * part).expand(len(chance), -1), chance)
            assert ((got == lo) | (got == hi)).all() and (got != got[:1]).any(0).all()
    for f in (Q.random_code, Q.random_root):
        assert (f(torch.full((len(chance),), 448 * (1 + 2.0 ** -22)), chance[:, 0]) == 448).all()
    x = torch.linspace(-40, 40, 1000)
    assert torch.equal(Q.random_code(-x, chance[:50]), -Q.random_code(x, chance[:50]))


def test_plain_random_codes_are_unbiased():
    """Over every chance of 20 bits: the mean code is y (below 2^-6 rounded once
    more, by 2^-30 at most); over chances 2^-18 apart: the mean square of a
    root's code is y^2 within that of the gap's (and float32)."""
    y = torch.cat([torch.logspace(-4.2, 2.64, 60), torch.tensor([2.0 ** -6 * (1 - 2.0 ** -24), 2.0 ** -9, 447.9999, 3e-9])])
    every, some = torch.arange(1 << 20) << 12, (torch.arange(1 << 18) << 14) + (1 << 13)
    for v in y:
        lo, hi = (t.double() for t in Q.neighbours(v.view(1)))
        got = Q.random_code(v.expand(1 << 20), every).double().mean()
        assert abs(got - v.double()) <= 2.0 ** -30 + 1e-12 * v
        got = Q.random_root(v.expand(1 << 18), some).double().square().mean()
        assert abs(got - v.double() ** 2) <= (hi ** 2 - lo ** 2) * (2.0 ** -18 + 2.0 ** -20)


def test_plain_hash_looks_random():
    """Over steps, places and values: each of the codes' chances is spread
    evenly (deviations of a mean of N: six times sqrt(1 / 12 / N)), and those of
    neighbouring steps, places and values are not correlated (six over sqrt N)."""
    v = torch.full((64, 256), 0.37) * (1 + torch.arange(64)[:, None] * 2.0 ** -23)
    pairs = [Q.chances(v, s) for s in [*range(64), *range(2 ** 33, 2 ** 33 + 64)]]
    both = [(torch.stack([p[i] for p in pairs]).double() + 0.5) / 2 ** 32 - 0.5 for i in (0, 1)]
    assert abs((both[0] * both[1]).mean()) * 12 <= 6 / math.sqrt(both[0].numel())
    for u in both:
        n = u.numel()
        assert abs(u.mean()) <= 6 * math.sqrt(1 / 12 / n)
        assert abs(u.square().mean() - 1 / 12) <= 6 * math.sqrt(1 / 180 / n)
        for axis in range(3):
            a, b = u.narrow(axis, 0, u.shape[axis] - 1), u.narrow(axis, 1, u.shape[axis] - 1)
            assert abs((a * b).mean()) * 12 <= 6 / math.sqrt(a.numel())
        for axis in range(3):  # the mean along each line
            line = u.mean(axis)
            assert line.abs().max() <= 7 * math.sqrt(1 / 12 / u.shape[axis])


@pytest.mark.parametrize("random", [False, True])
def test_plain_states_over_many_steps(random):
    """Constant gradients, a quarter 100 times smaller after 100 steps, beta2
    0.98: what the codes hold after 700 more (float32: v of the quarter within
    0.02 of 1e-4 of the others').  At random it is there within the chance of
    64 * 4 values (0.4 / 0.6 of v^2 and more in small steps: one deviation
    below 1, six of the mean 0.38); to nearest it has not moved."""
    b1, b2 = 0.9, 0.98
    g = torch.ones(4, 256)
    zeros = lambda: (torch.zeros(4, 256), torch.zeros(4))  # noqa: E731
    m, ms, r, rs = *zeros(), *zeros()
    for t in range(800):
        if t == 100:
            g[:, :64] = 0.01
        if random:
            (m, ms, r, rs), _, _ = Q.step(g, (m, ms, r, rs), t, b1, b2)
        else:
            root = R.decode(r, rs)
            mm, v, root = R.adamw_moments(g, R.decode(m, ms), root * root, b1, b2)
            (m, ms), (r, rs) = R.encode(mm, False), R.encode(root, True)
    v = R.decode(r, rs).double().square()
    ratio = float(v[:, :64].mean() / (1e-4 * v[:, 64:].mean()))
    assert abs(ratio - 1) <= 0.4 if random else ratio > 5000


# -------------------------------------------------------------- scratch memory
def scratch(monkeypatch, capturing=False):
    """_scratch_for with what it asks of torch recorded, not done."""
    import contextlib

    from top_routing_dispatch_gb300 import train
    made = []

    def empty(nbytes, dtype, device, stream):
        made.append((nbytes, stream))
        return torch.empty(nbytes, dtype=dtype)
    monkeypatch.setattr(train, "_empty", empty)
    monkeypatch.setattr(train, "_scratch", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: 0)
    ask = lambda nbytes, handle, stream=None: train._scratch_for(  # noqa: E731
        nbytes, torch.device("cpu"), 0, stream, handle)
    return train, made, ask


def test_scratch_is_kept_for_a_stream(monkeypatch):
    train, made, ask = scratch(monkeypatch)
    a = ask(1000, 7)
    assert ask(1 << 20, 7) is a and ask(500, 7, 7) is a and len(made) == 1
    b = ask(1000, 8, 8)
    assert b is not a and b.data_ptr() != a.data_ptr()
    big = ask(3 << 20, 7)
    assert ask(10, 7) is big and big.numel() == 3 << 20


def test_large_scratch_is_not_kept(monkeypatch):
    train, made, ask = scratch(monkeypatch)
    kept = ask(32 << 20, 7)
    assert ask(5, 7) is kept
    for stream in (None, 7):
        t = ask((32 << 20) + 1, 7, stream)
        assert t is not kept and t.numel() == (32 << 20) + 1 and made[-1] == (t.numel(), stream)
    assert list(train._scratch.values()) == [kept] and ask(5, 7) is kept


@pytest.mark.parametrize("stream", [None, 2])
def test_threads_streams_of_one_handle_share_no_scratch(monkeypatch, stream):
    """The per-thread default stream has the handle 2 in every thread."""
    train, made, ask = scratch(monkeypatch)
    a, b = ask(1000, 2, stream), ask(1000, 2, stream)
    assert a.data_ptr() != b.data_ptr() and not train._scratch
    assert made == [(1000, 2)] * 2


def test_scratch_of_a_capture_is_the_graphs(monkeypatch):
    train, made, ask = scratch(monkeypatch, capturing=True)
    for handle, stream in ((7, None), (7, 7), (2, 2)):
        a, b = ask(1000, handle, stream), ask(1000, handle, stream)
        assert a.data_ptr() != b.data_ptr()
    assert not train._scratch


def test_workspaces_of_the_threads_own_streams(monkeypatch):
    """One workspace for each thread's default stream, although it has one handle."""
    import contextlib
    import threading

    from top_routing_dispatch_gb300 import decode
    waits = []

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

        def wait_event(self, event):
            waits.append(("event", self.cuda_stream))

        def wait_stream(self, other):
            waits.append(("stream", self.cuda_stream, other.cuda_stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(0))
    ws = decode._Workspaces(torch.device("cpu"), lambda: torch.zeros(8), [])
    got = {}

    def ask(i):
        got[i] = [ws.add(2) for _ in range(3)]
    for i in range(2):
        t = threading.Thread(target=ask, args=(i,))
        t.start()
        t.join()
    ask(2)
    assert all(len(set(p)) == 1 for p in got.values()) and len({p[0] for p in got.values()}) == 3
    assert waits == [("event", 2), ("stream", 2, 0)] * 3 and 2 not in ws.pointers
    a = ws.add(5)
    assert ws.pointers[5] == a and len(ws.all) == 5


# ----------------------------------------------------------- refused before work
def test_a_refused_state_changes_nothing(monkeypatch):
    """Every entry is checked before the first one is copied."""
    from top_routing_dispatch_gb300 import train
    opt = train.AdamW.__new__(train.AdamW)
    taken = []
    monkeypatch.setattr(train.AdamW, "_set_steps", lambda self, steps: taken.append(steps))
    opt.m, opt.v = torch.zeros(2, 256), torch.zeros(2, 256)
    opt.m_scale = opt.v_scale = None
    opt.masters = [torch.zeros(300), None]
    good = dict(steps=7, m=torch.ones(2, 256), v=torch.ones(2, 256), m_scale=None, v_scale=None,
                masters=[torch.ones(300), None])
    for kw in (dict(steps=-1), dict(steps="x"), dict(steps=2 ** 63), dict(m=torch.ones(3, 256)), dict(v=torch.ones(2, 256).double()),
               dict(v_scale=torch.ones(2)), dict(masters=[torch.ones(300)]), dict(masters=[None, None]),
               dict(masters=[torch.ones(299), None])):
        with pytest.raises(ValueError):
            opt.load_state_dict({**good, **kw})
        assert not opt.m.any() and not opt.v.any() and not opt.masters[0].any() and not taken
    for name in ("steps", "m", "v", "m_scale", "v_scale"):
        with pytest.raises(KeyError):
            opt.load_state_dict({k: v for k, v in good.items() if k != name})
        assert not opt.m.any() and not taken
    opt.load_state_dict(good)
    assert opt.m.all() and opt.v.all() and opt.masters[0].all() and taken == [7]


def test_gradients_in_the_memory_of_parameters_are_refused():
    """A step reads gradients and writes parameters and masters in no order."""
    import top_routing_dispatch_gb300 as M
    line = torch.zeros(2000)
    p, g = [line[:300], line[300:700]], [torch.zeros(300), torch.zeros(400)]
    masters = [None, torch.zeros(400)]
    bf = [torch.zeros(300), torch.zeros(400, dtype=BF16)]
    for kw in (dict(grads=[line[:300], g[1]]), dict(grads=[g[0], line[299:699]]), dict(grads=[line[699:999], g[1]]),
               dict(params=bf, masters=masters, grads=[g[0], masters[1]])):
        with pytest.raises(ValueError, match="memory"):
            M.AdamW(**{**dict(params=p, grads=g), **kw})
    # beside them, and one gradient of two parameters, are taken (and refused for the device)
    for grads in ([line[700:1000], line[1000:1400]], [line[1000:1300], line[900:1300]]):
        with pytest.raises(ValueError, match="CUDA"):
            M.AdamW(p, grads)

"""The training operators together: a residual block's gradients against the
float64 oracle, a stack of blocks against the single calls, and the example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import moe_backward as OB
from oracle import moe_oracle as O
from tests import train_reference as R
from tests.gpu_helpers import NEAR_TIE_GAP

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = torch.float32, torch.bfloat16


def example():
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().double()


def make_block(n, rms, bias, seed=3, H=256, I=128, E=8, K=2):
    import top_routing_dispatch_gb300 as M
    g = torch.Generator()
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    norm = M.LayerNorm((1 + 0.2 * rand(H)).cuda(), None if rms else (0.1 * rand(H)).cuda(), rms=rms, dtype=BF16)
    block = M.MoEBlock(M.make_desc(n, H, I, E, K, BF16, True), norm, (0.05 * rand(H, E)).to(BF16).cuda(),
                       (0.1 * rand(E)).cuda() if bias else None, (rand(E, H, 2 * I) / H ** 0.5).to(BF16).cuda(),
                       (rand(E, I, H) / I ** 0.5).to(BF16).cuda())
    x, r, dout, ds = (rand(n, H).to(BF16).cuda() for _ in range(4))
    return block, x, r, dout, ds


@pytest.mark.parametrize("n", [1, 300])
@pytest.mark.parametrize("rms,bias", [(False, True), (True, False)])
def test_block_gradients_against_the_oracle(n, rms, bias):
    """Expert and router gradients within the 2e-2 (relative Frobenius) that
    moe_backward has; dx through the norm's gradient, which multiplies a row's
    error by at most r max|w|, plus dx's own rounding; the norm's weight
    gradient likewise, sum |d(dy)| |xh| (Cauchy-Schwarz over rows)."""
    block, x, r, dout, ds = make_block(n, rms, bias)
    out, s = block.forward(x, r)
    dx = block.backward(dout, ds)
    block.check()
    assert torch.equal(s, (x.float() + r.float()).to(BF16))
    norm = block.norm
    b64 = None if norm.bias is None else f64(norm.bias)
    want, _, mean, _, rstd, _ = R.norm(f64(s), f64(norm.weight), b64, 1e-5, rms)
    h_in = f64(block.h_in)
    assert ((h_in - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
    wg, b = f64(block.w_gate).numpy(), None if block.bias is None else f64(block.bias).numpy()
    near = O.near_tie_tokens(O.router_logits(h_in.numpy(), wg, b), 2, NEAR_TIE_GAP)
    forced = (np.where(near)[0], block.topk_idx.cpu().numpy()[near])
    w13, w2 = f64(block.w13).numpy(), f64(block.w2).numpy()
    y = O.moe_forward(h_in.numpy(), wg, b, w13, w2, 2, True, forced=forced)["y"]
    rel = lambda a, c: float(np.linalg.norm(a - c) / max(np.linalg.norm(c), 1e-30))  # noqa: E731
    assert rel(f64(out).numpy(), y) <= 1e-2
    o = OB.moe_backward(h_in.numpy(), wg, b, w13, w2, 2, True, f64(dout).numpy(), forced=forced)
    g = block._grads
    for name, key in (("w_gate", "dw_gate"), ("w13", "dw13"), ("w2", "dw2")):
        assert rel(f64(g[name]).numpy(), o[key]) <= 2e-2, name
    if bias:
        assert rel(f64(g["bias"]).numpy(), o["dbias"]) <= 2e-2
    dh = torch.from_numpy(o["dx"])
    off = 2e-2 * float(dh.norm())
    (wdx, _), (wdw, _), (wdb, _) = R.norm_backward(dh, f64(s), mean, rstd, f64(norm.weight), f64(ds), rms, n)
    gain = float(rstd.max()) * float(f64(norm.weight).abs().max())
    assert float((f64(dx) - wdx).norm()) <= gain * off + 2.0 ** -8 * float(wdx.norm())
    xh = (f64(s) - mean[:, None]) * rstd[:, None]
    assert float((f64(g["norm"]) - wdw).abs().max()) <= off * float(xh.norm(dim=0).max()) * (1 + 1e-3)
    if not rms:
        assert float((f64(g["norm_bias"]) - wdb).abs().max()) <= off * n ** 0.5 * (1 + 1e-3)


def test_block_without_residual_and_on_another_stream():
    block, x, _, dout, _ = make_block(130, False, True)
    out, s = block.forward(x)
    assert s is x
    dx = block.backward(dout)
    want = [out, dx] + [g.clone() for g in block.grads]
    other, side = make_block(130, False, True)[0], torch.cuda.Stream()
    torch.cuda.synchronize()
    out, _ = other.forward(x, stream=side)
    dx = other.backward(dout, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [out, dx] + other.grads))


def test_block_refusals():
    import top_routing_dispatch_gb300 as M
    block, x, r, dout, ds = make_block(20, False, True)
    with pytest.raises(ValueError):
        block.backward(dout)
    block.forward(x, r)
    for kw in (dict(dout=dout.float()), dict(dout=dout[:5]), dict(dout=dout, ds=ds.float()),
               dict(dout=dout, dx=dout[:5])):
        with pytest.raises(ValueError):
            block.backward(**kw)
    for kw in (dict(x=x.float()), dict(x=x, residual=r[:5]), dict(x=x, out=r.float())):
        with pytest.raises(ValueError):
            block.forward(**kw)
    args = [block.desc, block.norm, block.w_gate, block.bias, block.w13, block.w2]
    tiled = M.make_desc(20, 256, 128, 8, 2, BF16, True, tiled=True)
    f32norm = M.LayerNorm(torch.ones(256, device="cuda"))
    for i, bad in ((0, tiled), (0, M.make_desc(20, 128, 128, 8, 2, "f32", True)), (1, f32norm), (2, block.w_gate.float()),
                   (3, block.bias.to(BF16)), (4, block.w13[:4]), (5, block.w2.float())):
        with pytest.raises(ValueError):
            M.MoEBlock(*[bad if j == i else a for j, a in enumerate(args)])


def test_a_refused_forward_leaves_the_last_one():
    """A forward that is refused has not touched what the last one left for its
    backward; one that fails on the way leaves nothing to go back from."""
    block, x, r, dout, ds = make_block(40, False, True)
    block.forward(x, r)
    want = [block.backward(dout, ds)] + [g.clone() for g in block.grads]
    for kw in (dict(x=r, residual=x, out=torch.empty(40, 512, dtype=BF16, device="cuda")[:, ::2]),
               dict(x=r, out=r.float()), dict(x=r, residual=x[:5])):
        with pytest.raises(ValueError):
            block.forward(**kw)
    got = [block.backward(dout, ds)] + block.grads
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    w13, block.w13 = block.w13, None
    with pytest.raises(Exception):
        block.forward(r, x)
    with pytest.raises(ValueError):
        block.backward(dout, ds)
    block.w13 = w13
    block.forward(x, r)
    assert torch.equal(block.backward(dout, ds), want[0])


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_stack_step_is_its_single_calls(state):
    """A step of the example's stack: gradients clipped by the norm of them all,
    and every parameter moved as the plain step says."""
    ex = example()
    a, b = (ex.Stack(2, 70, state=state, max_norm=0.01) for _ in range(2))
    a.step()
    e = b.forward() - b.target
    b.backward(e / e.numel())
    assert all(torch.equal(p, q) for p, q in zip(a.grads, b.grads))
    total = float(torch.stack([f64(g).square().sum() for g in b.grads]).sum().sqrt())
    assert total > 0.01
    factor = torch.tensor(0.01 / (total + 1e-6), dtype=F32)
    before = [p.clone() for p in b.params]
    for i, (p, w, g, p0) in enumerate(zip(a.params, a.optimizer.masters, a.grads, before)):
        m, v, _ = R.adamw_moments(g.cpu() * factor, torch.zeros(g.shape), torch.zeros(g.shape), 0.9, 0.999)
        decay = 0.1 if p.dim() > 1 else 0.0
        want, tol = R.adamw_param(p0.cpu(), m, v, 1e-3, decay, 0.9, 0.999, 1e-8, 1)
        # the factor and with it m and the root of v are off by at most 10 u, which cancels but for eps
        tol = tol + 1e-3 * 20 * R.U32
        got = f64(w if w is not None else p)
        assert ((got - want).abs() <= tol + R.half_step(want, F32)).all(), i
        if w is not None:
            assert torch.equal(p, w.to(BF16))
    a.check()


def test_the_command_runs(capsys, monkeypatch):
    ex = example()
    for argv in (["--tokens", "100", "--steps", "5"], ["--tokens", "64", "--steps", "5", "--graph"],
                 ["--tokens", "100", "--steps", "4", "--state", "e4m3", "--blocks", "3", "--graph"]):
        monkeypatch.setattr("sys.argv", ["train_step.py"] + argv)
        ex.main()
        out = capsys.readouterr().out
        assert "us a step" in out and "nan" not in out


def test_a_graph_of_steps_is_the_eager_steps():
    """Replays of a captured step, one after another, against the same steps
    called one by one."""
    ex = example()
    eager, captured = ex.Stack(2, 96, state="e4m3"), ex.Stack(2, 96, state="e4m3")
    for s in (eager, captured):
        s.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for _ in range(3):
        eager.step()
        graph.replay()
    assert eager.optimizer.steps == captured.optimizer.steps == 4
    assert all(torch.equal(a, b) for a, b in zip(eager.params, captured.params))

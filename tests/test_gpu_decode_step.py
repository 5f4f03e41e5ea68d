"""The serving example against a float64 decoder layer: cache, attention,
router and experts together over several steps."""
import importlib.util
import math
import os

import pytest
import torch

from tests import decode_reference as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm64(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_steps_follow_the_float64_layer(cache):
    """Each step's output is within the roundings of its bf16 intermediates.

    x, the projections, q, attention, norms and the experts' output are rounded
    to bf16, each by at most 2^-8 of its value: about ten roundings of terms no
    larger than the output's own size, so 10 * 2^-8 in the relative norm.  An
    8-bit cache rounds keys and values by up to 2^-4; scores of deviation about
    1 and averages over values then move by at most 2 * 2^-4 of the attention
    term, one of the three terms of comparable size that the output adds."""
    ex = example()
    seqs, steps, page = 3, 21, 16
    L = ex.DecoderLayer(seqs, steps, hidden=256, q_heads=4, kv_heads=2, head_dim=64,
                        intermediate=128, experts=8, top_k=2, group=32, page=page, cache=cache)
    f = lambda t: t.detach().float().cpu().double()  # noqa: E731
    w13, w2 = R.unpack_w4(L.codes[0].cpu(), f(L.codes[1])), R.unpack_w4(L.codes[2].cpu(), f(L.codes[3]))
    wq, wo = f(L.w_qkv), f(L.w_out)
    rope = L.cache.rope.cpu().double()
    keys, vals = [], []
    g = torch.Generator()
    g.manual_seed(5)
    tol = 10 * 2.0 ** -8 + (2 * 2.0 ** -4 if cache == "e4m3" else 0)
    for t in range(steps):
        x = torch.randn((seqs, 256), generator=g).bfloat16()
        L.grow()
        y = f(L.step(x.cuda()))
        L.check()
        x = x.double()
        q, k, v = (z.unflatten(1, (-1, 64)) for z in (norm64(x) @ wq).split([256, 128, 128], 1))
        pos = [t] * seqs
        q, _ = R.rotate(q, rope, pos, False)
        k, _ = R.rotate(k, rope, pos, False)
        keys.append(k), vals.append(v)
        K, V = torch.stack(keys, 2), torch.stack(vals, 2)  # (seqs, kv_heads, t + 1, 64)
        s = torch.einsum("bhgd,bhtd->bhgt", q.view(seqs, 2, 2, 64), K) / math.sqrt(64)
        a = torch.einsum("bhgt,bhtd->bhgd", torch.softmax(s, -1), V).reshape(seqs, 256)
        x = x + a @ wo
        # the router's choice is the layer's own (ties aside, tested elsewhere)
        e, _ = R.experts(norm64(x), L.idx.cpu(), L.weights.cpu().double(), w13, w2)
        want = x + e
        assert float((y - want).norm() / want.norm()) <= tol, t


def test_the_command_runs(capsys, monkeypatch):
    ex = example()
    for argv in (["--seqs", "3", "--steps", "20"], ["--seqs", "2", "--steps", "20", "--graph"],
                 ["--seqs", "2", "--steps", "5", "--cache", "e4m3"]):
        monkeypatch.setattr("sys.argv", ["decode_step.py"] + argv)
        ex.main()
        assert "us a step" in capsys.readouterr().out

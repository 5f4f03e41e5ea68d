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

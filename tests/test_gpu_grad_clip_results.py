"""What a flat shard's step with a clip leaves to be read: finish_step(), and a loss scale that follows norm_buf."""
import math

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu

SIZES = [300, 1, 70001, 0, 255]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def grads(step, scale=1.0):
    return [(torch.randn(n, generator=gen(10 * step + i)) * 0.02 * scale).half().cuda() for i, n in enumerate(SIZES)]


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("capturable", [False, True])
def test_launch_clip_and_finish_step(capturable, side):
    kw = dict(lr=1e-2, device="cuda", capturable=capturable)
    a, b = (pkg.FlatShardAdamW(SIZES, **kw) for _ in range(2))
    ca, cb = (o.grad_clip(group_of=[0, 1, 0, 1, 1], max_norm=[0.1, 0.2]) for o in (a, b))
    stream = torch.cuda.Stream() if side else None
    for step in range(4):
        xs = grads(step)
        if step == 1:
            xs[2][70000] = math.inf
        for o in (a, b):
            o.flatten(xs, accumulate=False)
        torch.cuda.synchronize()
        a.launch_clip(ca, stream=stream)
        r = a.finish_step(stream)
        assert r == b.step(clip=cb) or (step == 1 and not r.finite)
        assert r.finite == (step != 1) and r.clip_coef == 1.0 and a.t == b.t == step + (step == 0)
        assert torch.equal(a.master, b.master) and torch.equal(a.exp_avg_sq, b.exp_avg_sq)
        assert torch.equal(a.norm_buf, ca.result)
    # and a step by the scalar limit after it
    for o in (a, b):
        assert o.step().finite
    assert torch.equal(a.norm_buf, b.norm_buf) and torch.equal(a.master, b.master)


@pytest.mark.parametrize("captured", [False, True])
def test_a_loss_scale_follows_steps_with_a_clip(captured):
    """It grows after good steps and backs off after the overflowed one; a scale that read another result would part."""
    o = pkg.FlatShardAdamW(SIZES, lr=1e-2, device="cuda", capturable=captured)
    clip = o.grad_clip(max_norm=0.1)
    scaler = pkg.DeviceLossScale("cuda", init_scale=2.0 ** 8, growth_interval=2)
    xs = grads(0)
    o.register_grads(xs)

    def step():
        o.flatten(accumulate=False, loss_scale=scaler)
        o.launch_clip(clip)
        scaler.launch_update(o.norm_buf)

    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    scale, good = 2.0 ** 8, 0
    for k in range(7):
        for x, y in zip(xs, grads(k, scale)):
            x.copy_(y)
        if k == 3:
            xs[0][5] = math.nan
        graph.replay() if captured else step()
        assert o.finish_step().finite == (k != 3)
        good = good + 1 if k != 3 else 0
        scale *= 0.5 if k == 3 else 2.0 if good == 2 else 1.0
        good %= 2
        assert scaler.scale == scale, k
    assert o.t == 6

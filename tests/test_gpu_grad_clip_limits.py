"""Limits changed while launches on another stream still wait there."""
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu

N = 1 << 16


@pytest.mark.parametrize("there", [False, True])
def test_each_launch_has_the_limits_of_its_time(there):
    side = torch.cuda.Stream()
    x, ys = torch.full((N,), 2.0, device="cuda"), [torch.zeros(N, device="cuda") for _ in range(3)]
    clips = [pkg.GradClip([N], max_norm=1e9) for _ in range(2)]
    clips[1].launch([x], out=[ys[0]], scale=1.0)  # its kernels are loaded
    c = clips[0]
    torch.cuda.synchronize()
    limits = [256.0, 128.0, 64.0]
    for limit, y in zip(limits, ys):
        c.set_max_norm(limit, stream=side if there else None)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        c.launch([x], out=[y], stream=side)
    c.set_max_norm(1e9, stream=side if there else None)
    side.synchronize()
    # the norm is 512: coefficients of 1/2, 1/4 and 1/8 but for the 1e-6 beside it
    for limit, y in zip(limits, ys):
        assert torch.allclose(y, torch.full_like(y, 2.0 * limit / 512.0), rtol=1e-6, atol=0)


def test_a_list_steps_limits_change_in_order():
    """TensorListAdamW launched on another stream, its limits changed on the current one at each step."""
    side = torch.cuda.Stream()
    masters = [[torch.ones(300, device="cuda"), torch.ones(70001, device="cuda")] for _ in range(2)]
    a, b = (pkg.TensorListAdamW(m, groups=[{}, {}], group_of=[0, 1], max_norm=[1.0, 1.0], lr=1e-2) for m in masters)
    xs = [torch.full((300,), 0.5, device="cuda"), torch.full((70001,), 0.25, device="cuda")]
    torch.cuda.synchronize()
    for k in range(3):
        a.clip.set_max_norm([0.5 ** k, 0.25])
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        a.launch_step(xs, stream=side)
        a.clip.set_max_norm([1e-9, 1e-9])  # behind that launch
        assert a.finish_step(side).finite
        b.clip.set_max_norm([0.5 ** k, 0.25])
        assert b.step(xs).finite
        for p, q in zip(a.exp_avg.split(256), b.exp_avg.split(256)):
            assert torch.equal(p, q)
    assert all(torch.equal(p, q) for p, q in zip(*masters))

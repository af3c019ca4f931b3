"""8-bit moments near the lower end of binary32, on the GPU."""
import numpy as np
import pytest
import torch

import _ref8 as R
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs
from test_gpu_state8 import HP, check_step, codes_view, f64, gen, host

pytestmark = pytest.mark.gpu


def state(n, power_m, power_r, g):
    """Any codes above zero at one power of two each."""
    nb = zs.state8_blocks(n)
    q = zs.State8(codes_view(n), torch.full((nb,), 2.0 ** power_m, device="cuda"), codes_view(n),
                  torch.full((nb,), 2.0 ** power_r, device="cuda"))
    for t in (q.exp_avg, q.root):
        t.view(torch.uint8).copy_(torch.randint(1, 127, (n,), generator=g))
    return q


def call(p, q, x, hp=HP, seed=None):
    table = zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda")
    zs.zero_adamw_step8_tensors(p, q, table, 1, x.numel(), x.dtype, 0, 1.0, None, hp["lr"], hp["b1"], hp["b2"], hp["eps"],
                                hp["wd"], 3, rounding_seed=seed)


def one_step(n, q, x, hp=HP, seed=None, p=None):
    p = torch.randn(n, generator=gen(3)).cuda() if p is None else p
    p0, old = f64(p), host(q)
    call(p, q, x.cuda(), hp, seed)
    check_step(p0, old, *R.grad(f64(x)), p, None, q, hp=hp, seed=seed)
    return p


@pytest.mark.parametrize("seed", [None, 5])
@pytest.mark.parametrize("power", [-48, -50, -54, -60, -71, -74, -76, -80, -83])
def test_zero_grads_let_a_small_exp_avg_sq_decay(power, seed):
    n = 3000
    q = state(n, power, power, gen(1))
    one_step(n, q, torch.zeros(n), seed=seed)
    assert (q.root.view(torch.uint8) > 0).all()


@pytest.mark.parametrize("seed", [None, 5])
@pytest.mark.parametrize("power", [-40, -52, -60, -66, -72, -80])
def test_small_grads(power, seed):
    # roots over 20 octaves of a block: exp_avg_sq from normal numbers down past the subnormal ones
    n, g = 3000, gen(2)
    x = torch.randn(n, generator=g) * torch.exp2(power - 20 * torch.rand(n, generator=g))
    one_step(n, state(n, power - 4, power - 6, g), x, seed=seed)
    one_step(n, zs.new_state8(n, "cuda"), x, seed=seed)


@pytest.mark.parametrize("b2", [0.0, 2.0 ** -20, 0.05])
def test_small_beta2(b2):
    n, g = 2048, gen(4)
    for power in (-70, -45, 0, 30):
        x = torch.randn(n, generator=g) * 2.0 ** -66
        one_step(n, state(n, -66, power, g), x, hp={**HP, "b2": b2})


@pytest.mark.parametrize("eps", [1e-12, 1e-20, 1e-30])
def test_a_small_eps_shows_the_root(eps):
    # single small elements in blocks of large ones: their exp_avg_sq is under 2^-126, their update around lr
    n, g = 4096, gen(5)
    x = torch.randn(n, generator=g)
    x[1::2] *= 2.0 ** -65
    q = state(n, 0, 0, g)
    for t in (q.exp_avg, q.root):
        t.view(torch.uint8)[1::2] = 0
    p = one_step(n, q, x, hp={**HP, "eps": eps, "wd": 0.0}, p=torch.zeros(n, device="cuda"))
    assert (p[1::2].abs() < 10 * HP["lr"]).all() and (p[1::2] != 0).all()


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 22, 2.0 ** 40])
def test_large_grads_after_a_small_state(size):
    n, g = 2048, gen(6)
    q = state(n, -70, -70, g)
    one_step(n, q, torch.randn(n, generator=g).abs().add(0.5) * size)
    assert all(bool(t.isfinite().all()) for t in q[1::2])


def test_small_moments_of_a_list():
    sizes, g = [300, 1, 5000], gen(7)
    q = [state(n, -80, -80, g) for n in sizes]
    p = [torch.zeros(n, device="cuda") for n in sizes]
    x = [torch.randn(n, generator=g).cuda() * 2.0 ** -78 for n in sizes]
    tl = zs.zero_tensor_list(p, q, state_bits=8)
    old = [host(s) for s in q]
    zs.zero_adamw_list(tl, zs.device_table(zs.zero_tensor_table(x)[0], 3, "cuda"), torch.float32, 1.0,
                       [(HP["lr"], HP["b1"], HP["b2"], HP["eps"], HP["wd"])], 3)
    for i, n in enumerate(sizes):
        check_step(np.zeros(n), old[i], *R.grad(f64(x[i])), p[i], None, q[i])

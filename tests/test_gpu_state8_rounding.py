"""Stochastic rounding by 16 bits on the GPU: each step's codes against the formula, and runs of thousands of steps
of the optimizers against the recurrence in 64 bits."""
import numpy as np
import pytest
import torch

import _ref8 as R
import _ref8_runs as L
import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from _helpers import norm_result_tensor, offset_view
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs
from test_gpu_state8 import DT, HP, clone, f64, gen, host, random_state8, same, shard_call

pytestmark = pytest.mark.gpu

SEED = 0x123456789ABCDEF1


def check_step16(p0, old, g, g_err, p1, new, *, t=3, stream=0, first=0, hp=HP):
    m0, r0 = R.values(old[0], old[1]), R.values(old[2], old[3])
    out = R.step(p0, m0, r0 * r0, g, g_err, t=t, root=2, div=3, **hp)
    R.check_close(f64(p1), *out["p"], "master")
    h = host(new)
    draws = L.halves(SEED, t, stream, len(p0), first)
    if hp["b1"] > 0.95:
        L.check_exp_avg16(h[0], h[1], *out["m"], L.swapped(draws))
    else:
        R.check_codes(h[0], h[1], *out["m"], k=R.draws(SEED, t, stream, len(p0), first)[0], name="exp_avg")
    L.check_root16(h[2], h[3], *out["r"], draws)


@pytest.mark.parametrize("n", [1, 255, 256, 257, 2047, 2048, 2049, 70001])
@pytest.mark.parametrize("gdt,offset,goff", [("bf16", 0, 0), ("f16", 0, 1), ("f32", 1, 0), ("f32", 0, 3)])
def test_shard_step(n, gdt, offset, goff):
    g = gen(n + offset)
    q = random_state8(n, g, offset)
    p = offset_view(n, torch.float32, offset, "cuda", torch.randn(n, generator=g))
    # grads over many octaves, so that roots reach the grid's even part below 2^-6
    x = offset_view(n, DT[gdt], goff, "cuda", (torch.randn(n, generator=g) * torch.exp2(
        torch.rand(n, generator=g) * 14 - 20)).to(DT[gdt]))
    clip = norm_result_tensor("cuda", coef=0.625)
    p0, old = f64(p), host(q)
    shard_call(p, q, x, clip=clip, seed=SEED, root_bits=16)
    gr, err = R.grad(f64(x), 1.0, None, 0.625)
    check_step16(p0, old, gr, err, p, q)


@pytest.mark.parametrize("n", [1, 257, 2047, 70001])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("b1", [0.9501, 0.99])
def test_shard_step_with_a_large_beta1(n, offset, b1):
    g, hp = gen(n + offset), {**HP, "b1": b1, "b2": 0.999}
    q = random_state8(n, g, offset)
    p = offset_view(n, torch.float32, offset, "cuda", torch.randn(n, generator=g))
    x = (torch.randn(n, generator=g) * torch.exp2(torch.rand(n, generator=g) * 14 - 20)).cuda()
    p0, old = f64(p), host(q)
    table = zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda")
    state = zs.new_adamw_device_state("cuda", 2)
    zs.zero_adamw_prepare_device(zs.device_hparams(*(hp[k] for k in ("lr", "b1", "b2", "eps", "wd")), "cuda"), None, state)
    q2, p2 = clone(q), p.clone()
    zs.zero_adamw_step8_tensors(p, q, table, 1, n, x.dtype, 0, 1.0, None, hp["lr"], b1, hp["b2"], hp["eps"], hp["wd"], 3,
                                rounding_seed=SEED)
    gr, err = R.grad(f64(x))
    check_step16(p0, old, gr, err, p, q, hp=hp)
    zs.zero_adamw_step8_tensors_device(p2, q2, table, 1, n, x.dtype, 0, 1.0, None, state, rounding_seed=SEED)
    assert same(q, q2) and torch.equal(p, p2)


def test_seven_bits_for_the_root_with_a_large_beta1():
    n, g, hp = 5000, gen(8), {**HP, "b1": 0.99, "b2": 0.999}
    q, p, x = random_state8(n, g), torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda() * 1e-2
    p0, old = f64(p), host(q)
    table = zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda")
    zs.zero_adamw_step8_tensors(p, q, table, 1, n, x.dtype, 0, 1.0, None, hp["lr"], hp["b1"], hp["b2"], hp["eps"], hp["wd"], 3,
                                rounding_seed=SEED, root_bits=7)
    out = R.step(p0, R.values(old[0], old[1]), R.values(old[2], old[3]) ** 2, *R.grad(f64(x)), t=3, root=2, div=3, **hp)
    h = host(q)
    L.check_exp_avg16(h[0], h[1], *out["m"], L.swapped(L.halves(SEED, 3, 0, n)))
    R.check_codes(h[2], h[3], *out["r"], k=R.draws(SEED, 3, 0, n)[1], floor=True, name="root")


def test_fresh_state_reaches_the_smallest_codes():
    # roots 2^-24 .. 1 of the block's largest, zeros among them
    n = 256 * 64
    x = torch.exp2(-24 * torch.rand(n, generator=gen(2)))
    x[::256], x[5::16] = 1.0, 0.0
    q, p = pkg.new_state8(n, "cuda"), torch.zeros(n, device="cuda")
    shard_call(p, q, x.cuda(), seed=SEED, step=1, root_bits=16)
    gr, err = R.grad(f64(x))
    check_step16(np.zeros(n), [np.zeros(n, np.uint8), np.zeros(n // 256), np.zeros(n, np.uint8), np.zeros(n // 256)], gr, err,
                 p, q, t=1)
    codes = q.root.view(torch.uint8).cpu()
    assert (codes[5::16] == 0).all() and (codes[x > 0] > 0).all() and set(range(1, 9)) <= set(codes.tolist())


def test_list_step_is_the_shard_step():
    sizes = [1, 300, 9999, 2048]
    g = gen(4)
    state = [random_state8(n, g) for n in sizes]
    p = [torch.randn(n, generator=g).cuda() for n in sizes]
    x = [(torch.randn(n, generator=g) * 1e-2).cuda() for n in sizes]
    new = [clone(s) for s in state]
    p2 = [t.clone() for t in p]
    tl = zs.zero_tensor_list(p2, new, state_bits=8)
    grads = zs.device_table(zs.zero_tensor_table(x)[0], len(sizes), "cuda")
    hp = (HP["lr"], HP["b1"], HP["b2"], HP["eps"], HP["wd"])
    zs.zero_adamw_list(tl, grads, torch.float32, 1.0, [hp], 3, rounding_seed=SEED, rounding_stream=40, root_bits=16)
    for i in range(len(sizes)):
        shard_call(p[i], state[i], x[i], seed=SEED, rounding_stream=40 + i, root_bits=16)
        assert same(state[i], new[i]) and torch.equal(p[i], p2[i])


@pytest.mark.parametrize("b2,bits", [(0.99, 7), (0.9901, 16), (0.999, 16)])
def test_the_bits_go_by_beta2(b2, bits):
    n, g = 5000, gen(7)
    q, p, x = random_state8(n, g), torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda() * 1e-2
    table = zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda")
    got = {}
    for root_bits in (0, 7, 16):
        a, b = clone(q), p.clone()
        zs.zero_adamw_step8_tensors(b, a, table, 1, n, x.dtype, 0, 1.0, None, 1e-2, 0.9, b2, 1e-8, 0.1, 3, rounding_seed=1,
                                    root_bits=root_bits)
        got[root_bits] = a
        a, b = clone(q), p.clone()
        tl = zs.zero_tensor_list([b], [a], state_bits=8)
        zs.zero_adamw_list(tl, table, x.dtype, 1.0, [(1e-2, 0.9, b2, 1e-8, 0.1)], 3, rounding_seed=1, root_bits=root_bits)
        assert same(a, got[root_bits])
        # with the scalars on the device
        hp = zs.device_hparams(1e-2, 0.9, b2, 1e-8, 0.1, "cuda")
        for form in ("shard", "list"):
            a, b, state = clone(q), p.clone(), zs.new_adamw_device_state("cuda", 2)
            if form == "shard":
                zs.zero_adamw_prepare_device(hp, None, state)
                zs.zero_adamw_step8_tensors_device(b, a, table, 1, n, x.dtype, 0, 1.0, None, state, rounding_seed=1,
                                                   root_bits=root_bits)
            else:
                zs.zero_adamw_prepare_list_device(hp, 1, None, state)
                zs.zero_adamw_list_device(zs.zero_tensor_list([b], [a], state_bits=8), table, x.dtype, 1.0, state,
                                          rounding_seed=1, root_bits=root_bits)
            assert same(a, got[root_bits]), (form, root_bits)
    assert same(got[0], got[bits]) and not same(got[7], got[16])


@pytest.mark.parametrize("capturable", [False, True])
def test_each_group_goes_by_its_own_beta2(capturable):
    sizes, betas = [3000, 777, 5000], [(0.9, 0.95), (0.98, 0.999), (0.8, 0.99)]
    x = [(torch.randn(n, generator=gen(n)) * 1e-2).cuda() for n in sizes]
    o = pkg.TensorListAdamW([torch.zeros(n, device="cuda") for n in sizes], lr=1e-2, state_bits=8, capturable=capturable,
                            groups=[{"betas": b} for b in betas], group_of=[0, 1, 2])
    for _ in range(2):
        o.step(x)
    for i, n in enumerate(sizes):
        one = pkg.TensorListAdamW([torch.zeros(n, device="cuda")], lr=1e-2, betas=betas[i], state_bits=8, rounding_stream=i)
        clip = norm_result_tensor("cuda", coef=1.0)
        for _ in range(2):
            one.launch_step([x[i]], norm_result=clip)
            one.finish_step(norm_result=clip)
        assert same(one.state_of(0), o.state_of(i)) and torch.equal(one.masters[0], o.masters[i]), i


def test_a_graph_follows_a_change_of_the_betas():
    n = 3000
    a, b = (pkg.FlatShardAdamW([n], lr=1e-2, betas=(0.9, 0.95), device="cuda", state_bits=8, grad_buffer=False, capturable=c)
            for c in (True, False))
    x = (torch.randn(n, generator=gen(1)) * 1e-2).cuda()
    a.register_grads([x])
    b.register_grads([x])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        a.launch_step_tensors()
    for betas in ((0.9, 0.95), (0.9, 0.999), (0.98, 0.999), (0.98, 0.95), (0.9, 0.95)):
        a.betas = b.betas = betas
        graph.replay()
        b.step_tensors()
        assert same(a.state8, b.state8) and torch.equal(a.master, b.master)


N = 4096


def run_flat(steps, b2, kind):
    opt = pkg.FlatShardAdamW([N], lr=1e-3, betas=(0.9, b2), device="cuda", state_bits=8, rounding_seed=3, grad_buffer=False,
                             lowp_dtype=None)
    x = torch.empty(N, device="cuda")
    opt.register_grads([x])
    for t in range(1, steps + 1):
        x.copy_(torch.from_numpy(L.grads(kind, t, N)))
        opt.launch_step_tensors()
        opt.finish_step()
    return host(opt.state8)


def run_list(steps, b2, kind):
    x = torch.empty(N, device="cuda")
    opt = pkg.TensorListAdamW([torch.zeros(N, device="cuda")], lr=1e-3, betas=(0.9, b2), state_bits=8, rounding_seed=3,
                              capturable=True)
    opt.register_grads([x])
    for t in range(1, steps + 1):
        x.copy_(torch.from_numpy(L.grads(kind, t, N)))
        opt.launch_step()
    return host(opt.state8)


def test_the_default_is_stochastic_with_seed_0():
    sizes = [700, 3000]
    x = [(torch.randn(n, generator=gen(n)) * 1e-2).cuda() for n in sizes]
    kw = dict(lr=1e-2, state_bits=8)
    a, b, c = (pkg.TensorListAdamW([torch.zeros(n, device="cuda") for n in sizes], **kw, **more) for more in (
        {}, dict(rounding_seed=0), dict(rounding_seed=None)))
    d, e = (pkg.FlatShardAdamW(sizes, device="cuda", **kw, **more) for more in ({}, dict(rounding_seed=0)))
    for o in (a, b, c):
        o.step(x)
    for o in (d, e):
        o.step_tensors(x)
    assert same(a.state8, b.state8) and not same(a.state8, c.state8) and same(d.state8, e.state8)


@pytest.mark.parametrize("run", [run_flat, run_list])
@pytest.mark.parametrize("kind", ["normal", "constant"])
@pytest.mark.parametrize("b2", [0.95, 0.99, 0.999, 0.9999])
def test_the_optimizers_follow_exp_avg_sq(run, b2, kind):
    steps = 3000
    h = run(steps, b2, kind)
    r = R.values(h[2], h[3])
    v = np.zeros(N)
    for t in range(1, steps + 1):
        v = b2 * v + (1 - b2) * L.grads(kind, t, N).astype(np.float64) ** 2
    lo, hi = L.run_bounds(b2)
    assert lo <= (r * r).mean() / v.mean() <= hi


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("b1", [0.9, 0.95, 0.99, 0.999])
def test_the_optimizers_follow_exp_avg(b1, capturable):
    steps = 2500
    opt = pkg.TensorListAdamW([torch.zeros(N, device="cuda")], lr=1e-3, betas=(b1, 0.999), state_bits=8, rounding_seed=3,
                              capturable=capturable)
    x = torch.empty(N, device="cuda")
    opt.register_grads([x])
    e = np.zeros(N)
    for t in range(1, steps + 1):
        g = np.float32(1.0) + L.grads("normal", t, N)
        e = b1 * e + (1 - b1) * g.astype(np.float64)
        x.copy_(torch.from_numpy(g))
        opt.launch_step()
        if not capturable:
            opt.finish_step()
    h = host(opt.state8)
    # up to 0.95 seven bits take up to u / 256 <= 1 / 2048 of an element off at each step; the elements' noise: under 1 %
    low = 1.0 / 2048 / (1 - b1) if b1 <= 0.95 else 0.0
    assert 0.99 - low <= R.values(h[0], h[1]).mean() / e.mean() <= 1.01

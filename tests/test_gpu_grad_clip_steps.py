"""Optimizer steps whose groups are clipped apart: a tensor list's AdamW that reads a result per group, and the ZeRO-2 data
plane of two processes (one GPU, gloo) with a GradClip over each rank's shard."""
import datetime
import math
import os
import socket

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from _helpers import norm_result_tensor
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

pytestmark = pytest.mark.gpu

SIZES = [300, 1, 70001, 0, 255, 4096, 9000]
OF = [0, 1, 2, 1, 0, 1, 2]
LIMITS = [0.05, math.inf, 0.2]
GROUPS = [{"weight_decay": 0.1}, {"lr": 3e-3}, {}]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def grads(step, dtype):
    return [None if i == 4 and step == 1 else (torch.randn(n, generator=gen(100 * step + i)) * 0.02).to(dtype).cuda() for i, n in enumerate(SIZES)]


def lists(bits, **kw):
    masters = [torch.randn(n, generator=gen(i)).cuda() for i, n in enumerate(SIZES)]
    lowp = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in SIZES]
    return pkg.TensorListAdamW(masters, lowp=lowp, lr=1e-2, groups=GROUPS, group_of=OF, state_bits=bits, rounding_seed=None, **kw)


def by_group(bits):
    """An optimizer for each group's tensors, whose clip is given."""
    whole = lists(bits)
    out = []
    for g in range(3):
        mine = [i for i, k in enumerate(OF) if k == g]
        out.append((mine, pkg.TensorListAdamW([whole.masters[i].clone() for i in mine], lowp=[torch.zeros_like(whole.lowp[i]) for i in mine],
                                              groups=[{"lr": 1e-2, **GROUPS[g]}], state_bits=bits, rounding_seed=None)))
    return out


def same(a, ref, bits):
    for mine, o in ref:
        for j, i in enumerate(mine):
            assert torch.equal(a.masters[i].view(torch.int32), o.masters[j].view(torch.int32)), i
            assert torch.equal(a.lowp[i], o.lowp[j]), i
            for x, y in zip(a.state_of(i), o.state_of(j)):
                assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_each_group_has_its_own_clip(bits, capturable, dtype):
    a, ref = lists(bits, max_norm=LIMITS, capturable=capturable), by_group(bits)
    for step in range(4):
        xs = grads(step, dtype)
        if step == 2:
            xs[5][17] = math.nan
        keep = [None if x is None else x.clone() for x in xs]
        r = a.step(xs, scale=0.5)
        assert all(x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(xs, keep))  # the grads stay
        assert r.finite == (step != 2) and r.clip_coef == 1.0 and a.t == (step + 1 if step < 2 else step)
        coefs = a.clip.finish().coefs
        if step != 2:
            norms = [math.sqrt(sum(float((x.double() * 0.5).square().sum()) for x, k in zip(xs, OF) if x is not None and k == g)) for g in range(3)]
            # a rounded coefficient of a norm that is right to 2.5e-10
            assert np.allclose(coefs, [min(1.0, m / (n + 1e-6)) for m, n in zip(LIMITS, norms)], rtol=2.0 ** -24 + 3e-10, atol=0)
            assert coefs[0] < 1 and coefs[1] == 1 and coefs[2] < 1
            for g, (mine, o) in enumerate(ref):
                o.launch_step([xs[i] for i in mine], scale=0.5, norm_result=(one := norm_result_tensor("cuda", coef=float(coefs[g]))))
                assert o.finish_step(norm_result=one).finite
        same(a, ref, bits)
    assert int(a.found_nonfinite) == 1


def test_limits_per_group_in_a_graph_with_a_loss_scale():
    a, b = (lists(32, max_norm=LIMITS, capturable=True) for _ in range(2))
    ls = [pkg.DeviceLossScale("cuda", init_scale=2.0 ** 8) for _ in range(2)]
    xs = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in SIZES]
    a.register_grads(xs)
    b.register_grads(xs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.launch_step(loss_scale=ls[0])
        ls[0].launch_update(a.norm_buf)
    for k in range(4):
        for i, x in enumerate(xs):
            x.copy_((torch.randn(x.numel(), generator=gen(70 * k + i)) * 2).cuda())
        if k == 1:
            xs[2][70000] = math.inf
        graph.replay()
        b.launch_step(loss_scale=ls[1])
        ls[1].launch_update(b.norm_buf)
        for x, y in zip(a.masters, b.masters):
            assert torch.equal(x, y)
        a.clip.set_max_norm([0.05 + k, 1.0, 0.2])  # the next replay follows
        b.clip.set_max_norm([0.05 + k, 1.0, 0.2])
    assert a.t == b.t == 3 and ls[0].scale == ls[1].scale == 2.0 ** 7


def test_limits_per_group_refused():
    with pytest.raises(ValueError, match="2 limits for 3 groups"):
        lists(32, max_norm=[1.0, 2.0])
    with pytest.raises(ValueError, match="max_norm"):
        lists(32, max_norm=[1.0, -1.0, 1.0])
    a = lists(32, max_norm=LIMITS)
    with pytest.raises(ValueError, match="one more"):
        zs.zero_adamw_list(a._list, a.device_table(grads(0, torch.float32))[0], torch.float32, 1.0, a._hp, 1, a.clip.results[:72], clips=True)
    with pytest.raises(ValueError, match="needs the groups' results"):
        zs.zero_adamw_list(a._list, a.device_table(grads(0, torch.float32))[0], torch.float32, 1.0, a._hp, 1, None, clips=True)
    xs = grads(0, torch.float32)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        xs[0].mul_(1.0)
        with pytest.raises(RuntimeError, match="before the capture"):
            a.launch_step(xs)
    assert a.step(xs).finite and a.t == 1


# ------------------------------------------------------------- data plane
WORLD, STEPS, BAD_STEP = 2, 3, 2


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _rank_main(rank, port, results):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=WORLD, timeout=datetime.timedelta(seconds=180))
    try:
        dev = torch.device("cuda:0")
        torch.cuda.set_device(dev)
        total = sum(SIZES)
        s, e = pkg.zero_shard_range(total, WORLD, rank)
        dp = pkg.ZeroDataPlane(SIZES, group=dist.group.WORLD, device=dev, lr=1e-2, max_norm=1e-9,
                               master=torch.randn(total, generator=gen(1))[s:e].to(dev))
        clip = dp.grad_clip(group_of=OF, max_norm=LIMITS)
        out = []
        for t in range(1, STEPS + 1):
            g = (torch.randn(total, generator=gen(10 * t + rank)) * 0.02).bfloat16()
            if t == BAD_STEP and rank == 1:
                g[3] = math.inf  # lies in rank 0's shard
            dp.flat_grad[:total] = g.to(dev)
            dp.reduce_scatter_grads()
            before = dp.opt.grad.cpu().clone()
            r = dp.step(clip=clip)
            c = clip.finish()
            out.append(dict(before=before, after=dp.opt.grad.cpu().clone(), result=(r.norm, r.clip_coef, r.finite, dp.opt.t), coefs=c.coefs,
                            group_norms=c.group_norms, tensor_norms=clip.tensor_norms.cpu().numpy()))
        results[rank] = dict(steps=out, flat_param=dp.flat_param.cpu(), master=dp.opt.master.cpu(), exp_avg=dp.opt.exp_avg.cpu())
    finally:
        dist.destroy_process_group()


def test_two_processes_clip_each_group_over_all_ranks():
    ctx = mp.get_context("spawn")
    results = ctx.Manager().dict()
    mp.start_processes(_rank_main, args=(_free_port(), results), nprocs=WORLD, start_method="spawn", join=True)
    r0, r1 = results[0], results[1]
    total = sum(SIZES)
    # one process that steps the whole FlatParameter with grads clipped as the ranks' results say
    one = pkg.FlatShardAdamW(SIZES, device="cuda", lr=1e-2, max_norm=math.inf, master=torch.randn(total, generator=gen(1)).cuda())
    applied = 0
    for t, (a, b) in enumerate(zip(r0["steps"], r1["steps"]), 1):
        for k in ("coefs", "group_norms", "tensor_norms"):
            assert np.array_equal(a[k], b[k], equal_nan=True), k
        assert repr(a["result"]) == repr(b["result"])
        fine = t != BAD_STEP
        applied += fine
        assert a["result"][1:] == (1.0, fine, applied)
        full = torch.cat([a["before"], b["before"]])
        if not fine:
            assert torch.equal(torch.cat([a["after"], b["after"]]).nan_to_num(7), full.nan_to_num(7))
            continue
        sums = [float(x.double().square().sum()) for x in full.split(SIZES)]
        norms = [math.sqrt(sum(s for s, k in zip(sums, OF) if k == g)) for g in range(3)]
        assert np.allclose(a["tensor_norms"], np.sqrt(sums), rtol=2.0 ** -24 + 3e-10, atol=0)
        assert np.allclose(a["group_norms"], norms, rtol=3e-10, atol=0)
        assert a["result"][0] == pytest.approx(math.sqrt(sum(sums)), rel=3e-10)
        assert np.allclose(a["coefs"], [min(1.0, m / (n + 1e-6)) for m, n in zip(LIMITS, norms)], rtol=2.0 ** -24 + 3e-10, atol=0)
        want = torch.cat([x * float(a["coefs"][k]) for x, k in zip(full.split(SIZES), OF)])
        assert torch.equal(torch.cat([a["after"], b["after"]]), want)
        one.grad.copy_(want)
        one.step()
    assert torch.equal(torch.cat([r0["master"], r1["master"]]), one.master.cpu())
    assert torch.equal(torch.cat([r0["exp_avg"], r1["exp_avg"]]), one.exp_avg.cpu())
    assert torch.equal(r0["flat_param"], r1["flat_param"]) and torch.equal(r0["flat_param"][:total], one.lowp.cpu())

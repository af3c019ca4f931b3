"""ZeRO-1 steps of two processes (one GPU, gloo) that are given the process group: every rank holds the whole averaged grad, so its
norms are whole already and no rank exchanges anything."""
import datetime
import math
import os
import socket

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu

SIZES = [300, 1, 70001, 0, 255, 4096, 9000]
OF = [0, 1, 2, 1, 0, 1, 2]
LIMITS = [0.05, math.inf, 0.2]
WORLD, KW = 2, dict(lr=1e-2, weight_decay=0.1, max_norm=0.5)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def grads(step):
    return (torch.randn(sum(SIZES), generator=gen(step)) * 0.02).cuda()


def master():
    return torch.randn(sum(SIZES), generator=gen(77))


def three_steps(o, group=None):
    """A step by a clip, one by the scalar limit, one straight from the tensors."""
    clip = o.grad_clip(group_of=OF, max_norm=LIMITS)
    out = []
    o.grad.copy_(grads(1))
    r = o.step(clip=clip, process_group=group)
    out += [r.norm, *clip.finish().coefs.tolist()]
    o.grad.copy_(grads(2))
    out.append(o.step(process_group=group).norm)
    out.append(o.step_tensors(list(grads(3).split(SIZES)), process_group=group).norm)
    return out


def _rank_main(rank, port, results):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=WORLD, timeout=datetime.timedelta(seconds=60))
    try:
        s, e = pkg.zero_shard_range(sum(SIZES), WORLD, rank)
        o = pkg.FlatShardAdamW(SIZES, world_size=WORLD, rank=rank, grad_range="full", device="cuda", master=master()[s:e].cuda(), **KW)
        results[rank] = (three_steps(o, dist.group.WORLD), o.t, o.master.cpu(), o.lowp.cpu())
    finally:
        dist.destroy_process_group()


def test_zero1_ranks_step_with_a_process_group():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    results = mp.get_context("spawn").Manager().dict()
    mp.start_processes(_rank_main, args=(port, results), nprocs=WORLD, start_method="spawn", join=True)
    one = pkg.FlatShardAdamW(SIZES, device="cuda", master=master().cuda(), **KW)
    want = three_steps(one)
    for r in range(WORLD):
        assert results[r][:2] == (want, 3)
    assert np.isfinite(want).all() and want[1] < 1
    assert torch.equal(torch.cat([results[r][2] for r in range(WORLD)]), one.master.cpu())
    assert torch.equal(torch.cat([results[r][3] for r in range(WORLD)]), one.lowp.cpu())

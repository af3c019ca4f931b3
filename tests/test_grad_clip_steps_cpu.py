"""The steps around a clip on the host, without a GPU: launches, streams and process groups are stand-ins that note what they get."""
import contextlib

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import optimizer as O
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs


# ------------------------------------------------- which ranks join a norm
class Group:
    """A process group of `size` ranks that counts the gathers."""

    def __init__(self, size):
        self.size, self.gathers = size, 0


@pytest.fixture
def gathers(monkeypatch):
    """Kernels do nothing; a gather of sums is counted and gives this rank's value for every rank."""
    def gather(local, group):
        group.gathers += 1
        return local.new_ones(group.size)

    monkeypatch.setattr(O, "_world", lambda group: group.size)
    monkeypatch.setattr(O, "gather_sqnorms", gather)
    monkeypatch.setattr(O, "torch_stream", lambda stream, device: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name in ("zero_grad_sqnorm", "zero_grad_sqnorm_finalize", "zero_grad_sqnorm_combine", "zero_flatten_cast", "zero_adamw_step",
                 "zero_adamw_step_tensors", "zero_reduce_chunks"):
        monkeypatch.setattr(zs, name, lambda *a, **k: None)
    monkeypatch.setattr(zs, "zero_tensor_table", lambda grads, numels=None: (None, sum(g.numel() for g in grads)))
    monkeypatch.setattr(zs, "device_table", lambda table, n, device: torch.zeros(1))
    monkeypatch.setattr(zs, "_stream", lambda s: 0)


@pytest.mark.parametrize("sizes", [[5, 3], [1], [7, 0, 1]])  # 1 element: rank 0's shard is the whole, the other ranks' are empty
@pytest.mark.parametrize("world", [1, 2, 4])
@pytest.mark.parametrize("grad_range", ["shard", "full"])
def test_every_rank_joins_the_norm_or_none_does(gathers, monkeypatch, grad_range, world, sizes):
    """A whole grad has its whole norm on every rank: a rank that gathered alone would wait for the others."""
    joined = []
    for rank in range(world):
        o = pkg.FlatShardAdamW(sizes, world_size=world, rank=rank, grad_range=grad_range, device="cpu")
        g, n = Group(world), 0
        o.step(process_group=g)
        n, g.gathers = g.gathers, 0
        o.step_tensors([torch.zeros(k) for k in sizes], process_group=g)
        direct, g.gathers = g.gathers, 0
        given = []
        c = o.grad_clip(max_norm=1.0)
        c.launch = lambda **kw: given.append(kw["process_group"])
        o.launch_clip(c, process_group=g)
        # of one rank a clip has nothing to join, with a group or without
        joined.append((n, direct, int(world > 1 and given[0] is g)))
    want = int(grad_range == "shard" and world > 1)
    assert joined == [(want,) * 3] * world


@pytest.mark.parametrize("rank", [0, 1])
def test_reduce_needs_a_shards_buffer_on_every_rank(gathers, rank):
    chunks = torch.zeros(2, 4)
    o = pkg.FlatShardAdamW([5, 3], world_size=2, rank=rank, grad_range="full", device="cpu")
    with pytest.raises(ValueError, match="shard-only"):
        o.reduce(chunks, accumulate=False, scale=0.5)
    pkg.FlatShardAdamW([5, 3], world_size=2, rank=rank, device="cpu").reduce(chunks, accumulate=False, scale=0.5)
    pkg.FlatShardAdamW([5, 3], grad_range="full", device="cpu").reduce(torch.zeros(1, 8), accumulate=False, scale=1.0)


# --------------------------------------------- the result that a step leaves
def test_a_step_with_a_clip_leaves_the_clips_result(gathers, monkeypatch):
    """norm_buf is what finish_step() and a loss scale's update read, after a step of either kind."""
    o = pkg.FlatShardAdamW([5, 3], device="cpu")
    c = o.grad_clip(group_of=[0, 1], max_norm=[1.0, 2.0])
    used = []
    monkeypatch.setattr(zs, "zero_adamw_step", lambda *a: used.append(bytes(a[11].numpy())))

    def launch(norm, finite):
        r = zs.zero_norm_result(norm * norm, norm, 1.0, finite)
        c.launch = lambda **kw: c.result.copy_(torch.frombuffer(bytearray(bytes(r)), dtype=torch.uint8))
        o.launch_clip(c)
        return bytes(r)

    want = launch(3.0, 1)
    assert used[-1] == want and bytes(o.norm_buf.numpy()) == want
    assert o.finish_step() == (9.0, 3.0, 1.0, True) and o.t == 1
    want = launch(float("inf"), 0)
    assert used[-1] == want and bytes(o.norm_buf.numpy()) == want
    assert not o.finish_step().finite and o.t == 1
    launch(2.0, 1)
    assert o.finish_step().norm == 2.0 and o.t == 2


def test_a_step_refuses_a_clip_that_other_grads_were_registered_with(gathers):
    """It would clip those and step with its own grads as they are."""
    o = pkg.FlatShardAdamW([5, 3], device="cpu")
    c = o.grad_clip(max_norm=1.0)
    with pytest.raises(ValueError):
        c.register_grads([torch.zeros(5)])
    assert c.shard is o.grad  # nothing was registered
    c.register_grads([torch.zeros(5), torch.zeros(3)])
    with pytest.raises(ValueError, match="not over this optimizer's grad buffer"):
        o.step(clip=c)

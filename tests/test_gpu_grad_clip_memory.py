"""Registered tensors whose place others take while a launch on another stream, or a captured graph, still uses their memory."""
import math

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu

N = 1 << 20
PAUSE = 100_000_000  # clock cycles


@pytest.fixture(autouse=True)
def loaded():
    """The kernels are loaded, so that no first launch outlasts the pause."""
    c = pkg.GradClip([N, 5], max_norm=1.0)
    c.launch([torch.ones(N, device="cuda"), None], out=[torch.ones(N, dtype=torch.bfloat16, device="cuda"), torch.ones(5, device="cuda")])
    c.launch([torch.ones(N, device="cuda"), None])
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()


def taken(tensors):
    """Whether new tensors of the same kinds, filled on the current stream, got the memory of any of these addresses."""
    new = [torch.full((N,), 7.0, device="cuda") for _ in range(3)] + [torch.full((N,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    return bool(tensors & {t.data_ptr() for t in new}), new


@pytest.mark.parametrize("drop", ["registration", "clip"])
def test_registered_tensors_outlast_a_launch_on_another_stream(drop):
    side = torch.cuda.Stream()
    x, y = torch.full((N,), 2.0, device="cuda"), torch.empty(N, dtype=torch.bfloat16, device="cuda")
    z = torch.full((N,), 3.0, device="cuda")
    c = pkg.GradClip([N, N], max_norm=0.5)
    c.register_grads([x, z], out=[y, z])
    at = {t.data_ptr() for t in (x, y, z)}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(PAUSE)
    c.launch(stream=side)
    del x, y, z
    if drop == "registration":
        c.register_grads([torch.zeros(N, device="cuda"), None])
    else:
        del c
    busy = not side.query()
    got, new = taken(at)
    assert busy and not got
    side.synchronize()
    assert all(bool((t == 7).all()) for t in new)
    if drop == "registration":
        assert c.finish(side).norm == math.sqrt(13.0) * 1024


def test_a_shards_grad_outlasts_a_launch_on_another_stream():
    side = torch.cuda.Stream()
    g = torch.full((N,), 2.0, device="cuda")
    at = {g.data_ptr()}
    c = pkg.GradClip.of_shard([N - 5, 5], g, 0, max_norm=0.5)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(PAUSE)
    c.launch(stream=side)
    del g, c
    busy = not side.query()
    got, new = taken(at)
    assert busy and not got
    side.synchronize()
    assert all(bool((t == 7).all()) for t in new)


def test_a_graphs_tensors_outlast_their_registration():
    x, y = torch.full((N,), 2.0, device="cuda"), torch.full((N,), 5.0, dtype=torch.bfloat16, device="cuda")
    c = pkg.GradClip([N], max_norm=512.0)
    c.register_grads([x], out=[y])
    at = {x.data_ptr(), y.data_ptr()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.launch()
    c.register_grads([torch.full((N,), 1.0, device="cuda")])
    kept = c._replayed[0].tensors
    del x, y
    got, new = taken(at)
    assert not got
    for _ in range(3):
        graph.replay()
    assert c.finish().norm == 2048.0
    assert all(bool((t == 7).all()) for t in new)
    assert bool((kept[0] == 2).all()) and bool((kept[1] == 0.5).all())
    assert c.clip_().norm == 1024.0  # and eager launches take what is registered now

"""What becomes of the tensors that a clip registered while kernels or graphs still use them, without a GPU: streams and launches
are stand-ins, and who records a tensor where is noted."""
import contextlib
import gc
import weakref

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import grad_clip as G
from fsdp_sharded_mixed_flatparameter_gb300 import optimizer as O
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

OWN, SIDE, OTHER = 11, 22, 33  # handles: the current stream's, others'


class World:
    def __init__(self):
        self.current, self.capturing, self.recorded, self.launched = [OWN], set(), [], []

    @contextlib.contextmanager
    def stream(self, s):
        self.current.append(s)
        yield
        self.current.pop()

    def on(self, t):
        """The streams that t's memory was recorded on, in order."""
        return [s for p, s in self.recorded if p == t.data_ptr()]


@pytest.fixture
def world(monkeypatch):
    w = World()
    monkeypatch.setattr(zs, "_current_handle", lambda index: w.current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", w.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.current[-1] in w.capturing)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.recorded.append((t.data_ptr(), s)), raising=False)
    for module in (G, O):
        monkeypatch.setattr(module, "torch_stream", lambda s, device: w.current[-1] if s is None else s)
    for name in ("zero_list_sums", "zero_list_norms", "zero_sums_norms", "zero_list_clip"):
        monkeypatch.setattr(zs, name, lambda *a, **k: w.launched.append(name))
    return w


def on_gpu(c):
    """The clip as if its memory were on device 0, made on the current stream."""
    c._index, c._home = 0, OWN
    return c


def clip_of(x, out=None, write=True):
    c = on_gpu(pkg.GradClip([t.numel() for t in x], device="cpu", max_norm=1.0))
    c.register_grads(x, out=out, write=write)
    return c


LAUNCHES = {"launch": lambda c, s: c.launch(stream=s), "norms": lambda c, s: c.launch_norms(stream=s), "sums": lambda c, s: c.launch_sums(stream=s),
            "joined": lambda c, s: c.launch(gathered_sums=torch.ones(2, 2, dtype=torch.float64), stream=s)}


@pytest.mark.parametrize("kind", list(LAUNCHES))
@pytest.mark.parametrize("elsewhere", [False, True])
def test_registered_tensors_are_recorded_where_they_are_used(world, kind, elsewhere):
    x, y = [torch.zeros(5), torch.zeros(3)], [torch.zeros(5), torch.zeros(3)]
    c = clip_of(x, y if elsewhere else None)
    for _ in range(3):
        LAUNCHES[kind](c, None)
        LAUNCHES[kind](c, OWN)
    assert world.recorded == [] and world.launched
    for s in (SIDE, OTHER, SIDE):
        LAUNCHES[kind](c, s)
    for t in x + (y if elsewhere else []):
        assert sorted(set(world.on(t))) == [SIDE, OTHER]  # their memory is not given out before those are done
    # others registered in their place are recorded in their turn
    z = [torch.zeros(5), None]
    c.register_grads(z)
    assert world.on(z[0]) == []
    LAUNCHES[kind](c, SIDE)
    assert set(world.on(z[0])) == {SIDE}


def test_grads_registered_on_another_stream_belong_to_it(world):
    x = [torch.zeros(5)]
    c = on_gpu(pkg.GradClip([5], device="cpu"))
    with world.stream(SIDE):
        c.register_grads(x)
    c.launch(stream=SIDE)
    assert world.on(x[0]) == [] and SIDE in world.on(c.tensor_sums)
    c.launch()
    assert world.on(x[0]) == [OWN]


def test_a_shards_grad_is_recorded_where_it_is_used(world):
    g = torch.zeros(8)
    c = on_gpu(pkg.GradClip.of_shard([5, 3], g, 0, max_norm=1.0))
    c._registered = c._registered._replace(table=c._registered.table._replace(stream=OWN))
    c.launch()
    assert world.on(g) == []
    c.launch(stream=SIDE)
    assert SIDE in world.on(g)


def gone(refs):
    gc.collect()
    return all(r() is None for r in refs)


@pytest.mark.parametrize("current", [True, False])
def test_captured_tensors_live_as_long_as_the_clip(world, current):
    """The graph may be replayed at any time."""
    x, y = [torch.zeros(5), None], [None, torch.zeros(3)]
    c = on_gpu(pkg.GradClip([5, 3], device="cpu", max_norm=1.0))
    c.register_grads(x, out=y)
    refs = [weakref.ref(x[0]), weakref.ref(y[1])]
    world.capturing.update({SIDE, OTHER})  # a capture and a stream forked from it
    with world.stream(SIDE):
        for _ in range(2):
            c.launch(stream=None if current else OTHER)
    assert len(c._replayed) == 1 and world.on(x[0]) == []
    c.register_grads([None, torch.zeros(3)])
    del x, y
    assert not gone(refs[:1]) and not gone(refs[1:])
    del c
    assert gone(refs)


def test_tensors_that_no_graph_uses_go_with_their_registration(world):
    x = [torch.zeros(5)]
    c = clip_of(x)
    c.launch()
    c.launch(stream=SIDE)
    refs = [weakref.ref(x[0])]
    del x
    assert not gone(refs)
    c.register_grads([torch.zeros(5)])
    assert gone(refs) and c._replayed == []

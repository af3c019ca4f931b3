"""Limits changed between launches, without a GPU: streams are stand-ins that note what is enqueued on them and what they wait for."""
import contextlib

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import grad_clip as G
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

OWN, SIDE = 11, 22


class World:
    def __init__(self):
        self.current, self.log, self.capturing = [OWN], [], False

    @contextlib.contextmanager
    def stream(self, s):
        self.current.append(s.handle)
        yield
        self.current.pop()


class Stream:
    def __init__(self, world, handle):
        self.world, self.handle = world, handle

    def wait_stream(self, other):
        self.world.log.append((self.handle, "waits for", other.handle))


@pytest.fixture
def world(monkeypatch):
    w = World()
    monkeypatch.setattr(zs, "_current_handle", lambda index: w.current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", w.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.capturing)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None, raising=False)
    monkeypatch.setattr(G, "torch_stream", lambda s, device: Stream(w, w.current[-1] if s is None else s))
    monkeypatch.setattr(G.GradClip, "_read_on", lambda *a: None)
    monkeypatch.setattr(zs, "zero_list_norms", lambda gl, sc, clip, b, flag, raw, **k: w.log.append((raw, "launch")))
    copy = torch.Tensor.copy_

    def noted(t, *a, **k):
        if t.dtype == torch.float64:
            w.log.append((w.current[-1], "limits"))
        return copy(t, *a, **k)

    monkeypatch.setattr(torch.Tensor, "copy_", noted)
    return w


def clip():
    c = pkg.GradClip([5, 3], device="cpu", group_of=[0, 1], max_norm=[1.0, 2.0])
    c._index, c._home = 0, OWN
    c.register_grads([torch.zeros(5), torch.zeros(3)])
    return c


def test_limits_are_written_behind_the_last_launch(world):
    c = clip()
    c.set_max_norm(3.0)  # nothing to wait for yet
    c.launch(stream=SIDE)
    c.set_max_norm([4.0, 5.0])
    c.launch(stream=SIDE)
    c.set_max_norm(6.0, stream=SIDE)
    c.launch()
    c.set_max_norm(7.0)
    c.set_max_norm(8.0, stream=SIDE)
    assert world.log == [(OWN, "limits"), (SIDE, "launch"), (OWN, "waits for", SIDE), (OWN, "limits"), (SIDE, "launch"), (SIDE, "limits"),
                         (OWN, "launch"), (OWN, "limits"), (SIDE, "waits for", OWN), (SIDE, "limits")]
    assert c.max_norms.tolist() == [8.0, 8.0]


def test_limits_are_not_changed_in_a_capture(world):
    c = clip()
    world.capturing = True
    c.launch(stream=SIDE)  # captured: nothing runs there yet
    with pytest.raises(RuntimeError, match="outside the capture"):
        c.set_max_norm(1.0)
    world.capturing = False
    with pytest.raises(ValueError, match="max_norm"):
        c.set_max_norm([1.0, -1.0])
    assert c.max_norms.tolist() == [1.0, 2.0]
    c.set_max_norm(3.0)
    assert world.log == [(SIDE, "launch"), (OWN, "limits")]


# ------------------------------------------------- limits and their groups
def test_several_limits_need_groups():
    """Without them every tensor would be clipped by the first."""
    for many in ([1.0, 0.5], (1.0, 0.5), torch.tensor([1.0, 0.5])):
        with pytest.raises(ValueError, match="2 limits: group_of"):
            pkg.GradClip([5, 3], device="cpu", max_norm=many)
        with pytest.raises(ValueError, match="2 limits: group_of"):
            pkg.GradClip.of_shard([5, 3], torch.zeros(8), 0, max_norm=many)
        with pytest.raises(ValueError, match="2 limits: group_of"):
            pkg.FlatShardAdamW([5, 3], device="cpu").grad_clip(max_norm=many)
        with pytest.raises(ValueError, match="2 limits: group_of"):
            pkg.TensorListAdamW([torch.zeros(5), torch.zeros(3)], groups=[{}, {}], max_norm=many)
    assert pkg.GradClip([5, 3], device="cpu", max_norm=[0.5]).max_norms.tolist() == [0.5]  # one for all
    assert pkg.GradClip([5, 3], device="cpu", max_norm=[1.0, 0.5], group_of=[0, 0]).n_groups == 2  # an empty group that was asked for
    assert pkg.GradClip([5, 3], device="cpu", max_norm=0.5).n_groups == 1


def test_grads_that_the_clip_refuses_are_not_registered_for_the_step_either(monkeypatch):
    """Else the step would go by the norms of the grads registered before."""
    made = []
    monkeypatch.setattr(zs, "zero_tensor_table", lambda grads, numels=None: (None, sum(g.numel() for g in grads)))
    monkeypatch.setattr(zs, "device_table", lambda table, n, device: made.append(torch.zeros(1)) or made[-1])
    monkeypatch.setattr(zs, "_stream", lambda s: OWN)
    o = pkg.TensorListAdamW.__new__(pkg.TensorListAdamW)  # host memory: without the parts that only a launch reads
    o._init_tables([5, 3], "cpu")
    o.clip = pkg.GradClip([5, 3], device="cpu", group_of=[0, 1], max_norm=[1.0, 2.0])
    with pytest.raises(ValueError, match="must be a tensor on"):  # as pinned host memory would be
        o.register_grads([torch.zeros(5, device="meta"), torch.zeros(3)])
    assert o._registered is None and o.clip._registered is None
    x = [torch.zeros(5), torch.zeros(3)]
    o.register_grads(x)
    first, norms = o._registered, o.clip._registered
    with pytest.raises(ValueError, match="must be a tensor on"):
        o.register_grads([torch.zeros(5), torch.zeros(3, device="meta")])
    assert o._registered is first and o.clip._registered is norms and norms.tensors[0] is x[0]
    o.register_grads([torch.zeros(5), torch.zeros(3)])
    assert o._registered is not first and o.clip._registered is not norms


def test_a_clips_registered_grads_have_no_flat_parameter_table(monkeypatch):
    c = pkg.GradClip([5, 3], device="cpu")
    x = [torch.zeros(5), torch.zeros(3)]
    for _ in range(2):
        with pytest.raises(ValueError, match="needs the grads"):
            c.device_table(None)
        c.register_grads(x)
    table = torch.zeros(1)
    monkeypatch.setattr(zs, "zero_tensor_table", lambda grads, numels=None: (None, sum(g.numel() for g in grads)))
    monkeypatch.setattr(zs, "device_table", lambda *a: table)
    monkeypatch.setattr(zs, "_stream", lambda s: OWN)
    assert c.device_table(x) == (table, 2, torch.float32)


# ---------------------------------------------------------- freed storages
def freed(n):
    """A tensor whose storage was given back, as sharded loops do with whole parameters between uses."""
    t = torch.zeros(n)
    t.untyped_storage().resize_(0)
    return t


def test_tensors_without_memory_are_refused():
    """Their address is NULL, which stands for a tensor without a grad."""
    plan = zs.zero_grad_plan([5, 0], None, 1, 2, "cpu")
    empty = torch.zeros(0)
    zs.grad_list(plan, [torch.zeros(5), empty])
    for kw in (dict(), dict(write=False), dict(out=[torch.zeros(5), None])):
        with pytest.raises(ValueError, match=r"grads\[0\] has no memory"):
            zs.grad_list(plan, [freed(5), empty], **kw)
    with pytest.raises(ValueError, match=r"out\[0\] has no memory"):
        zs.grad_list(plan, [torch.zeros(5), empty], [freed(5), empty])
    with pytest.raises(ValueError, match="flat grad has no memory"):
        pkg.GradClip.of_shard([5, 3], freed(8), 0)
    whole = torch.zeros(10)
    part = whole[2:]
    pkg.GradClip.of_shard([5, 3], part, 0)
    whole.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="flat grad has no memory"):
        pkg.GradClip.of_shard([5, 3], part, 0)
    pkg.GradClip.of_shard([5, 3], empty, 8)  # a rank without elements

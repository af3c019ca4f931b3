"""What becomes of a grads list's device table while kernels still read it, without a GPU: the tables, the streams and the
launches are stand-ins that note who uses what."""
import contextlib
import gc
import weakref

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import optimizer as O
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

OWN, SIDE = 11, 22  # handles: the current stream's, another's


class Table:
    def __init__(self, address):
        self.address, self.used_on = address, []

    def data_ptr(self):
        return self.address

    def record_stream(self, stream):
        self.used_on.append(stream)


class World:
    def __init__(self):
        self.tables, self.launched, self.capturing, self.current = [], [], set(), [OWN]

    def device_table(self, table, n, device):
        t = Table(4096 * (len(self.tables) + 1))
        self.tables.append(weakref.ref(t))
        return t

    @contextlib.contextmanager
    def stream(self, s):
        self.current.append(s)
        yield
        self.current.pop()


@pytest.fixture
def world(monkeypatch):
    w = World()
    monkeypatch.setattr(zs, "zero_tensor_table", lambda grads, numels=None: (None, sum(g.numel() for g in grads)))
    monkeypatch.setattr(zs, "device_table", w.device_table)
    monkeypatch.setattr(zs, "_stream", lambda s: w.current[-1] if s is None else s)
    monkeypatch.setattr(O, "torch_stream", lambda s, device: w.current[-1] if s is None else s)
    monkeypatch.setattr(torch.cuda, "stream", w.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.current[-1] in w.capturing)
    for name in ("zero_grad_sqnorm_finalize",):
        monkeypatch.setattr(zs, name, lambda *a, **k: None)
    for name in ("zero_flatten_cast", "zero_adamw_step_tensors", "zero_adamw_step8_tensors"):
        monkeypatch.setattr(zs, name, lambda *a, **k: w.launched.append([x for x in a if isinstance(x, Table)]))
    return w


def shard(bits):
    return pkg.FlatShardAdamW([5, 3], device="cpu", state_bits=bits, grad_buffer=False)


def lists(count):
    return [[torch.zeros(5), torch.zeros(3)] for _ in range(count)]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("flat", [False, True])
def test_a_table_read_on_another_stream_is_recorded_there(world, bits, flat):
    o = shard(bits)
    g = torch.zeros(8) if flat else lists(1)[0]
    step = o.launch_step_flat if flat else o.launch_step_tensors
    step(g, stream=SIDE)
    (t,) = [t() for t in world.tables]
    assert SIDE in t.used_on and all(x == [t] for x in world.launched)
    t.used_on.clear()
    step(g)  # where its memory was allocated nothing is needed
    assert t.used_on == []


def test_flatten_and_registered_grads_record_too(world):
    o = pkg.FlatShardAdamW([5, 3], device="cpu")
    a, b = lists(2)
    o.flatten(a, accumulate=False, stream=SIDE)
    o.register_grads(b)
    o.flatten(accumulate=True, stream=SIDE)
    assert [t().used_on for t in world.tables] == [[SIDE], [SIDE]]


@pytest.mark.parametrize("flat", [False, True])
def test_a_captured_table_outlives_the_cache(world, flat):
    o = shard(32)
    many = [torch.zeros(8) for _ in range(200)] if flat else lists(200)
    step = o.launch_step_flat if flat else o.launch_step_tensors
    table = o.device_flat_table if flat else o.device_table
    table(many[0])
    world.capturing.add(SIDE)
    with world.stream(SIDE):
        step(many[0])
    world.capturing.clear()
    captured = world.tables[0]
    for g in many[1:]:
        step(g)
    world.launched.clear()
    gc.collect()
    assert captured() is not None and captured().used_on == []
    alive = [t for t in world.tables if t() is not None]
    assert len(alive) <= 64 + 1  # the others leave, the oldest first
    assert world.tables[-1]() is not None and world.tables[1]() is None


def test_a_capture_on_the_tables_own_stream_keeps_it(world):
    o = shard(32)
    many = lists(100)
    o.device_table(many[0])
    world.capturing.add(OWN)
    o.launch_step_tensors(many[0])
    world.capturing.clear()
    for g in many[1:]:
        o.launch_step_tensors(g)
    world.launched.clear()
    gc.collect()
    assert world.tables[0]() is not None

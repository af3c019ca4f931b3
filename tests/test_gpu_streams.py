"""Stream arguments by handle, and what is read on streams other than their own."""
import importlib.util

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs
from fsdp_sharded_mixed_flatparameter_gb300.optimizer import torch_stream

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_handle_0_is_the_default_stream():
    dev = torch.device("cuda", torch.cuda.current_device())
    assert torch_stream(0, dev) == torch.cuda.default_stream(dev)
    s = torch.cuda.Stream()
    assert torch_stream(s.cuda_stream, dev).cuda_stream == s.cuda_stream
    with torch.cuda.stream(s):
        assert torch_stream(None, dev) == s and torch_stream(0, dev) == torch.cuda.default_stream(dev)


def test_the_current_streams_handle():
    s = torch.cuda.Stream()
    for st in (torch.cuda.default_stream(), s):
        with torch.cuda.stream(st):
            assert zs._stream(None) == st.cuda_stream == zs._stream(st) == zs._stream(st.cuda_stream)


def test_without_torchs_own_accessor(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    spec = importlib.util.find_spec(zs.__name__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert other._stream(None) == s.cuda_stream


def test_a_step_on_handle_0_waits_for_its_own_norm():
    # the norm is read on the stream that computes it, behind a pause there
    n = 3000
    opt = pkg.FlatShardAdamW([n], lr=1e-2, device="cuda")
    g = torch.randn(n, generator=gen(1)).cuda()
    want = opt.step_tensors([g]).norm
    opt.device_table([h := g * 2])
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    assert opt.step_tensors([h], stream=0).norm == 2 * want and opt.t == 2


SIZES = [3000, 1, 517]


def grads(k):
    return [(torch.randn(n, generator=gen(31 * k + i)) * 1e-2).bfloat16().cuda() for i, n in enumerate(SIZES)]


def make(kind, **kw):
    masters = [torch.randn(n, generator=gen(i)).cuda() for i, n in enumerate(SIZES)]
    if kind == "list":
        return pkg.TensorListAdamW(masters, lr=1e-2, state_bits=8, capturable=True, **kw)
    return pkg.FlatShardAdamW(SIZES, lr=1e-2, device="cuda", master=torch.cat(masters), grad_buffer=False, capturable=True, **kw)


def launch(o, *a, **kw):
    (o.launch_step if isinstance(o, pkg.TensorListAdamW) else o.launch_step_tensors)(*a, **kw)


def masters(o):
    return torch.cat([p.view(-1) for p in (o.masters if isinstance(o, pkg.TensorListAdamW) else [o.master])])


@pytest.mark.parametrize("kind", ["list", "shard"])
def test_more_lists_than_the_cache_holds_in_flight_on_another_stream(kind):
    a, b = make(kind), make(kind)
    many = [grads(k) for k in range(150)]
    s = torch.cuda.Stream()
    launch(a, many[0], stream=s)  # kernels loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    for g in many[1:]:
        launch(a, g, stream=s)
    torch.cuda.synchronize()
    for g in many:
        launch(b, g)
    torch.cuda.synchronize()
    assert a.t == b.t == 150 and torch.equal(masters(a), masters(b))


@pytest.mark.parametrize("kind", ["list", "shard"])
def test_a_graph_is_replayed_after_many_other_lists(kind):
    a, b = make(kind), make(kind)
    many = [grads(k) for k in range(100)]
    a.device_table(many[0])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        launch(a, many[0])
    for g in many[1:]:
        launch(a, g)
    graph.replay()
    for g in many[1:] + many[:1]:
        launch(b, g)
    torch.cuda.synchronize()
    assert a.t == b.t == 100 and torch.equal(masters(a), masters(b))

"""Checkpoints of optimizers over parameters that require grad, on the GPU."""
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu

SHAPES = [(40, 33), (7,), (1500,)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def parameters(dtype, seed=0):
    return [torch.nn.Parameter(torch.randn(s, generator=gen(seed + i)).to(dtype).cuda()) for i, s in enumerate(SHAPES)]


def grads(k):
    return [(torch.randn(s, generator=gen(50 * k + i)) * 1e-2).bfloat16().cuda() for i, s in enumerate(SHAPES)]


def optimizer(bits, seed=0, **kw):
    return pkg.TensorListAdamW(parameters(torch.float32, seed), lowp=parameters(torch.bfloat16, seed), lr=1e-2,
                               state_bits=bits, **kw)


def values(o):
    moments = [t.view(torch.uint8) for t in o.state8] if o.state_bits == 8 else [o.exp_avg, o.exp_avg_sq]
    return [o.t, *(t.detach().clone() for t in (*o.masters, *o.lowp, *moments))]


def equal(a, b):
    return a[0] == b[0] and all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_list_of_parameters_is_restored(bits):
    a, b = optimizer(bits), optimizer(bits, seed=9)
    a.step(grads(1))
    sd = a.state_dict()
    assert not any(t.requires_grad for t in sd["masters"])
    b.load_state_dict(sd)
    assert equal(values(a), values(b)) and all(p.requires_grad and p.is_leaf for p in b.masters + b.lowp)
    for o in (a, b):
        o.step(grads(2))
    assert equal(values(a), values(b)) and a.t == 2


@pytest.mark.parametrize("bits", [8, 32])
def test_a_list_checkpoint_that_does_not_fit_changes_nothing(bits):
    a = optimizer(bits)
    a.step(grads(1))
    sd = a.state_dict()
    name = "state8" if bits == 8 else "exp_avg"
    for bad in ({**sd, "numels": sd["numels"][:-1]}, {**sd, "masters": sd["masters"][:-1]}, {**sd, name: sd[name][:-1]},
                {k: v for k, v in sd.items() if k != name}):
        o = optimizer(bits, seed=9)
        before = values(o)
        with pytest.raises(ValueError):
            o.load_state_dict(bad)
        assert equal(before, values(o))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_load_is_ordered_on_its_stream(bits):
    # a step waits on the side stream behind a pause; the load comes after it there, another step after the load
    s = torch.cuda.Stream()
    a, b = (optimizer(bits, capturable=True) for _ in range(2))
    sd = optimizer(bits, seed=9).state_dict()
    first, second = grads(1), grads(2)
    for o in (a, b):  # kernels loaded, tables built
        o.step(first, stream=s)
        o.device_table(second)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    a.launch_step(first, stream=s)
    a.load_state_dict(sd, stream=s)
    a.launch_step(second, stream=s)
    torch.cuda.synchronize()
    b.launch_step(first)
    b.load_state_dict(sd)
    b.launch_step(second)
    torch.cuda.synchronize()
    assert a.t == b.t == 1 and equal(values(a), values(b))


@pytest.mark.parametrize("bits,capturable", [(8, False), (8, True), (32, True)])
def test_a_data_plane_load_is_ordered_on_its_stream(bits, capturable):
    # as above for a shard with its exchanges (one rank); the checkpoint's moments are fp32, which 8 bits convert
    numels = [3000, 77]
    s = torch.cuda.Stream()
    kw = dict(device="cuda", lr=1e-2, capturable=capturable)
    a, b = (pkg.ZeroDataPlane(numels, state_bits=bits, **kw) for _ in range(2))
    other = pkg.ZeroDataPlane(numels, master=torch.randn(sum(numels), generator=gen(1)).cuda(), **kw)
    other.flat_grad.copy_(torch.randn(sum(numels), generator=gen(2)))
    other.reduce_scatter_grads()
    other.step()
    sd = other.state_dict()

    def steps(dp, stream):
        dp.reduce_scatter_grads(stream=stream)
        dp.opt.launch_step(stream=stream)
        dp.load_state_dict(sd, stream=stream)
        dp.reduce_scatter_grads(stream=stream)
        dp.opt.launch_step(stream=stream)

    for dp in (a, b):
        dp.flat_grad.copy_(torch.randn(sum(numels), generator=gen(3)))
        dp.reduce_scatter_grads(stream=s)
        dp.step(stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    steps(a, s)
    torch.cuda.synchronize()
    steps(b, None)
    torch.cuda.synchronize()
    assert a.opt.t == b.opt.t
    for x, y in zip(values_of_shard(a.opt), values_of_shard(b.opt)):
        assert torch.equal(x, y)
    assert torch.equal(a.flat_param, b.flat_param)


def values_of_shard(o):
    moments = [t.view(torch.uint8) for t in o.state8] if o.state_bits == 8 else [o.exp_avg, o.exp_avg_sq]
    return [o.master, o.lowp, *moments]

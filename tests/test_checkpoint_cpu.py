"""Checkpoints of a flat shard whose master or copy is a parameter, and checkpoints that do not fit, without a GPU."""
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

N = 300


def shard(bits=32, value=1.0):
    o = pkg.FlatShardAdamW([N], device="cpu", master=torch.nn.Parameter(torch.full((N,), value)), state_bits=bits,
                           lowp_out=torch.nn.Parameter(torch.full((N,), value, dtype=torch.bfloat16)))
    assert o.master.requires_grad and o.lowp.requires_grad
    if bits == 8:
        for t in o.state8:
            t.view(torch.uint8).fill_(int(value))
    else:
        o.exp_avg.fill_(value)
        o.exp_avg_sq.fill_(2 * value)
    o.t = int(value)
    return o


def values(o):
    moments = [t.view(torch.uint8) for t in o.state8] if o.state_bits == 8 else [o.exp_avg, o.exp_avg_sq]
    return [o.t, *(t.detach().clone() for t in (o.master, o.lowp, *moments))]


def equal(a, b):
    return a[0] == b[0] and all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_shard_of_parameters_is_restored(bits):
    a, b = shard(bits, 3.0), shard(bits, 5.0)
    sd = a.state_dict()
    assert not any(t.requires_grad for t in (sd["master"], sd["lowp"]))
    b.load_state_dict(sd)
    assert equal(values(a), values(b)) and b.master.requires_grad and b.master.is_leaf


@pytest.mark.parametrize("bits", [8, 32])
def test_a_checkpoint_that_does_not_fit_changes_nothing(bits):
    sd = shard(bits, 3.0).state_dict()
    names = ("state8",) if bits == 8 else ("exp_avg", "exp_avg_sq")
    short = {nm: (sd[nm][:3] if nm == "state8" else sd[nm][:-1]) for nm in names}
    small = {"state8": tuple(t[:-1] for t in sd["state8"])} if bits == 8 else {"exp_avg_sq": sd["exp_avg_sq"][:1]}
    for bad in ({**sd, "start": 1}, {**sd, "master": sd["master"][:1]}, {**sd, "lowp": sd["lowp"][:1]}, {**sd, **short}, {**sd, **small},
                {k: v for k, v in sd.items() if k not in names}):
        o = shard(bits, 5.0)
        before = values(o)
        with pytest.raises(ValueError):
            o.load_state_dict(bad)
        assert equal(before, values(o))

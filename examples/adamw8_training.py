"""Train a small network with fp32 moments, then go on from its checkpoint in 32 and in 8 bits.

    python examples/adamw8_training.py [--steps 200]

One checkpoint, four ways to go on:

* TensorListAdamW, fp32 moments: one launch steps every tensor, matrices with weight decay, biases without;
* TensorListAdamW, 8-bit moments, rounded stochastically and, to compare, to nearest: the checkpoint's moments are
  packed on loading;
* FlatShardAdamW, 8-bit moments: the same parameters as one flat shard, the grads read where backward left them.

Prints the loss at the end and the optimizer's bytes per parameter for each.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fsdp_sharded_mixed_flatparameter_gb300 import FlatShardAdamW, TensorListAdamW  # noqa: E402

SHAPES = [(256, 1024), (1024,), (1024, 1024), (1024,), (1024, 64), (64,)]


def forward(params, x):
    """An MLP in bf16; params: the low-precision copies, with grad."""
    for i in range(0, len(params), 2):
        x = x @ params[i] + params[i + 1]
        if i + 2 < len(params):
            x = torch.nn.functional.silu(x)
    return x


class Task:
    """Regression on a fixed random network's outputs: a fresh batch for every step, the same for every run."""

    def __init__(self, device, batch=1024):
        g = torch.Generator(device=device).manual_seed(1)
        self.teacher = [torch.randn(s, device=device, generator=g) * (s[0] ** -0.5 if len(s) == 2 else 0.1) for s in SHAPES]
        self.device, self.batch = device, batch

    def loss(self, params, step):
        g = torch.Generator(device=self.device).manual_seed(1000 + step)
        x = torch.randn(self.batch, SHAPES[0][0], device=self.device, generator=g)
        with torch.no_grad():
            y = forward(self.teacher, x)
        return (forward(params, x.bfloat16()).float() - y).square().mean()


def initial(device):
    g = torch.Generator(device=device).manual_seed(2)
    return [torch.randn(s, device=device, generator=g) * (s[0] ** -0.5) if len(s) == 2 else
            torch.zeros(s, device=device) for s in SHAPES]


def tensor_list(masters, **kw):
    lowp = [p.bfloat16().requires_grad_() for p in masters]
    opt = TensorListAdamW(masters, lowp=[c.detach() for c in lowp], groups=[{"weight_decay": 0.01}, {"weight_decay": 0.0}],
                          group_of=[0 if p.dim() == 2 else 1 for p in masters], lr=1e-3, betas=(0.9, 0.95), max_norm=1.0,
                          **kw)
    return opt, lowp


def train(task, step_fn, params, first, steps):
    for k in range(first, first + steps):
        for p in params:
            p.grad = None
        task.loss(params, k).backward()
        step_fn([p.grad for p in params])
    with torch.no_grad():
        return float(sum(task.loss(params, 10 ** 6 + j) for j in range(8)) / 8)


def run(steps=200, device="cuda:0", say=print):
    """The final loss by name, and the optimizer's bytes per parameter (masters, copies, moments)."""
    task = Task(device)
    masters = initial(device)
    n = sum(p.numel() for p in masters)
    first, params = tensor_list(masters)
    start = float(task.loss(params, 10 ** 6).detach())
    reached = train(task, first.step, params, 0, steps)
    checkpoint = first.state_dict()
    say(f"loss {start:.4f} at the start, {reached:.4f} after {steps} steps with fp32 moments")

    found = {"start": start, "reached": reached}
    for name, kw in (("fp32", {}), ("8 bits, nearest", dict(state_bits=8, rounding_seed=None)),
                     ("8 bits, stochastic", dict(state_bits=8, rounding_seed=0))):
        opt, params = tensor_list([p.clone() for p in masters], **kw)
        opt.load_state_dict(checkpoint)
        found[name] = train(task, opt.step, params, steps, steps)
        say(f"{name:20s} loss {found[name]:.4f} after {opt.t} steps, {opt.resident_bytes() / n:.2f} bytes per parameter")

    # the same parameters as one flat shard
    numels = [p.numel() for p in masters]
    flat = FlatShardAdamW(numels, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.01, max_norm=1.0, device=device, state_bits=8,
                          rounding_seed=0, grad_buffer=False, master=torch.cat([p.view(-1) for p in masters]))

    def joined(storage):  # the checkpoint's moments lie at each tensor's offset of a storage
        return torch.cat([storage[a:a + k] for a, k in zip(first.offsets, numels)])

    flat.load_state_dict({"t": checkpoint["t"], "start": 0, "end": n, "master": flat.master.cpu(),
                          "exp_avg": joined(checkpoint["exp_avg"]), "exp_avg_sq": joined(checkpoint["exp_avg_sq"])})
    flat.lowp.copy_(flat.master)
    params = [v.view(s).requires_grad_() for v, s in zip(torch.split(flat.lowp, numels), SHAPES)]
    found["flat shard"] = train(task, flat.step_tensors, params, steps, steps)
    say(f"{'flat shard, 8 bits':20s} loss {found['flat shard']:.4f} after {flat.t} steps, "
        f"{flat.resident_bytes() / n:.2f} bytes per parameter")
    return found


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    run(ap.parse_args().steps)

"""The cases by which the norms of many tensors, their clipping, and both for one rank's flat shard are measured.

Three operators:

* ``norms``: the norm of each tensor of a list of mixed types, of each group of tensors and of all of them; p = 2, 1 or inf;
* ``clip``: the same norms, then every gradient scaled (unscaled, averaged) and clipped by its group's norm, in place or into
  buffers of another type;
* ``shard``: both for one rank of a sharded job: the pieces of the tensors that lie in its flat fp32 shard, their sums joined
  with the other ranks' in rank order, and the shard clipped in place.

With s the scale, x the elements of tensor i, M the limit of its group:  S_i = sum |s x|^p (the largest |s x| for inf);  the
tensor's norm is S_i^(1/p), a group's that of the sum (the largest) of its tensors' S;  c = min(1, M / (norm + 1e-6)) in fp32;
the clipped gradient is (s c) x, rounded once to its type.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
#: elements of a plain form's first sums
PIECE = 4096
#: tensors up to which a plain form scales them one by one
FEW = 400
#: the loss scale of the fp16 cases, and the mean over ranks turned into the mean over tokens (one token in five is padding)
UNSCALE, TOKENS = 2.0 ** -16, 1.25


def listed():
    """The smallest calls, ordinary ones and the largest of each operator."""
    return [
        # a small model, one fp32 tensor per layer: what a call costs
        {"name": "norms-tiny", "op": "norms", "sizes": "tiny", "grad": "f32", "p": 2, "groups": 1, "align": 128, "scale": 1.0},
        # GPT-2 small in fp32, back to back in one buffer, 1-norms
        {"name": "norms-gpt2-p1", "op": "norms", "sizes": "gpt2", "grad": "f32", "p": 1, "groups": 2, "align": 1, "scale": 1.0},
        # 20,000 ragged tensors watched one by one, small ones in fp32
        {"name": "norms-ragged", "op": "norms", "sizes": "ragged", "tensors": 20000, "elements": 1507457739, "grad": "mixed", "p": 2, "groups": 3, "align": 128, "scale": 1.0},
        # one flat fp16 gradient of a Llama-13B shard, its largest magnitude
        {"name": "norms-flat-inf", "op": "norms", "sizes": "flat", "elements": 1626983040, "grad": "f16", "p": 0, "groups": 1, "align": 1, "scale": UNSCALE},
        # the small model, clipped in place
        {"name": "clip-tiny", "op": "clip", "sizes": "tiny", "grad": "f32", "out": "same", "p": 2, "groups": 1, "align": 128, "scale": TOKENS, "limit": 0.5},
        # GPT-2 small in bf16, biases and norms in fp32, two groups
        {"name": "clip-gpt2", "op": "clip", "sizes": "gpt2", "grad": "mixed", "out": "same", "p": 2, "groups": 2, "align": 128, "scale": TOKENS, "limit": 0.5},
        # four layers of Llama-7B, the usual step late in a run: the norm is below the limit
        {"name": "clip-llama4-below", "op": "clip", "sizes": "llama", "layers": 4, "grad": "bf16", "out": "same", "p": 2, "groups": 1, "align": 1, "scale": 1.0, "limit": 50.0},
        # 4000 ragged fp16 tensors under a loss scale, each by its own norm, into fp32
        {"name": "clip-ragged-own", "op": "clip", "sizes": "ragged", "tensors": 4000, "elements": 302390543, "grad": "f16", "out": "f32", "p": 2, "groups": 0, "align": 128, "scale": UNSCALE, "limit": 0.5},
        # eight layers of Llama-7B with embedding and head, clipped in place
        {"name": "clip-llama8", "op": "clip", "sizes": "llama", "layers": 8, "grad": "bf16", "out": "same", "p": 2, "groups": 1, "align": 128, "scale": TOKENS, "limit": 0.5},
        # GPT-2 small, rank 3 of 8
        {"name": "shard-gpt2", "op": "shard", "sizes": "gpt2", "world": 8, "rank": 3, "p": 2, "groups": 2, "scale": TOKENS, "limit": 0.8},
        # 20,000 ragged tensors, rank 2 of 4, borders everywhere
        {"name": "shard-ragged", "op": "shard", "sizes": "ragged", "tensors": 20000, "elements": 1507457739, "world": 4, "rank": 2, "p": 2, "groups": 3, "scale": TOKENS, "limit": 0.8},
        # two layers of Llama-7B with embedding and head, rank 1 of 2, largest magnitudes
        {"name": "shard-llama2-inf", "op": "shard", "sizes": "llama", "layers": 2, "world": 2, "rank": 1, "p": 0, "groups": 1, "scale": TOKENS, "limit": 0.8},
    ]


def draw(rng):
    """One more case: any operator, sizes log-uniform over its listed range."""
    def spread(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    op = rng.choice(["norms", "clip", "clip", "shard"])
    tensors = spread(1, 20000)
    case = {"op": op, "sizes": "ragged", "tensors": tensors, "elements": max(spread(1000000, 1500000000), 4 * tensors), "p": rng.choice([2, 2, 2, 1, 0]),
            "groups": rng.choice([0, 1, 1, 2, 3, 17])}
    if op == "shard":
        case.update(world=rng.choice([2, 4, 8]), scale=TOKENS, limit=0.8)
        case["rank"] = rng.randrange(case["world"])
        return case
    case.update(grad=rng.choice(["f32", "bf16", "f16", "mixed"]), align=rng.choice([1, 128]))
    case["scale"] = UNSCALE if case["grad"] == "f16" else rng.choice([1.0, TOKENS])
    if case["grad"] == "f32":
        case["elements"] = max(case["elements"] // 2, 4 * tensors)
    if op == "clip":
        case["limit"] = rng.choice([0.1, 0.5, 0.9])
        case["out"] = "f32" if case["grad"] == "f16" else rng.choice(["same", "same", "bf16", "f32"]) if case["grad"] == "bf16" else "same"
        if case["out"] == "same":
            case["scale"] = TOKENS
        case["elements"] = max(case["elements"] // 2, 4 * tensors)
    return case


# ------------------------------------------------------------------ sizes
def sizes_of(case):
    """The tensors' sizes of a case, in order."""
    kind = case["sizes"]
    if kind == "tiny":
        return [262144, 262144, 262144, 475459]
    if kind == "flat":
        return [case["elements"]]
    if kind == "gpt2":
        h = 768
        block = [h, h, 3 * h * h, 3 * h, h * h, h, h, h, 4 * h * h, 4 * h, 4 * h * h, h]
        return [50257 * h, 1024 * h] + 12 * block + [h, h]
    if kind == "llama":
        h, f = 4096, 11008
        return [32000 * h] + case["layers"] * ([h * h] * 4 + [f * h] * 3 + [h, h]) + [h, 32000 * h]
    # ragged: log-uniform weights over 20 octaves, scaled to the total, at least one element each
    k, total = case["tensors"], case["elements"]
    w = np.exp(np.random.Generator(np.random.PCG64(k)).uniform(0.0, 20 * math.log(2.0), k))
    n = 1 + np.floor(w * ((total - k) / w.sum())).astype(np.int64)
    n[int(np.argmax(n))] += total - int(n.sum())
    return [int(x) for x in n]


def types_of(case, sizes):
    """The type of each tensor: mixed is bf16 for matrices and fp32 for the small ones, as norms and biases are kept."""
    if case["op"] == "shard":
        return ["f32"] * len(sizes)
    return ["f32" if n < 16384 else "bf16" for n in sizes] if case["grad"] == "mixed" else [case["grad"]] * len(sizes)


def groups_of(case, count):
    """The group of each tensor, in turn; 0 groups: each its own."""
    return list(range(count)) if case["groups"] == 0 else [i % case["groups"] for i in range(count)]


def pieces_of(case, sizes, rank):
    """How many elements of each tensor lie in a rank's shard of the flat parameter, and where the shard starts and ends."""
    ends = np.cumsum(sizes)
    chunk = -(-int(ends[-1]) // case["world"])
    start, end = min(rank * chunk, int(ends[-1])), min((rank + 1) * chunk, int(ends[-1]))
    return np.maximum(0, np.minimum(ends, end) - np.maximum(ends - sizes, start)), start, end


def mags(count):
    """The tensors' standard deviations, over six octaves as layers' gradients differ."""
    return np.exp2(np.random.Generator(np.random.PCG64(count + 1)).uniform(-12.0, -6.0, count))


def limits(case, sizes):
    """The limit of each group: a share of the norm that its tensors have by their deviations."""
    n, m = np.asarray(sizes, dtype=np.float64), mags(len(sizes))
    own_sums = {2: n * m * m, 1: n * m * math.sqrt(2 / math.pi), 0: m * np.sqrt(2 * np.log(n + 1))}[case["p"]]
    of = groups_of(case, len(sizes))
    total = np.zeros(max(of) + 1)
    {0: np.maximum}.get(case["p"], np.add).at(total, of, own_sums)
    scale = 1.0 if case["scale"] == UNSCALE else case["scale"]
    return [float(x) for x in case["limit"] * scale * (np.sqrt(total) if case["p"] == 2 else total)]


# ----------------------------------------------------------------- inputs
def noise(lengths, std, g, dtype):
    """Normal values of a deviation by stretch, one element in 50 zero."""
    total = int(sum(lengths))
    out = torch.empty(total, dtype=dtype, device="cuda")
    ends = np.cumsum(lengths)
    for a in range(0, total, 1 << 28):
        b = min(total, a + (1 << 28))
        here = np.minimum(ends, b) - np.maximum(ends - np.asarray(lengths), a)
        at = np.flatnonzero(here > 0)
        x = torch.randn(b - a, device="cuda", generator=g)
        x.masked_fill_(torch.rand(b - a, device="cuda", generator=g) < 0.02, 0)
        out[a:b] = x.mul_(torch.repeat_interleave(torch.tensor(std[at], dtype=torch.float32, device="cuda"), torch.tensor(here[at], device="cuda"), output_size=b - a))
    return out


def inputs(case, seed):
    """The tensors of each type back to back in one buffer, at multiples of `align` elements, and what the layout is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    sizes = sizes_of(case)
    types, std = types_of(case, sizes), mags(len(sizes))
    st = {"case": case, "sizes": sizes, "groups_of": groups_of(case, len(sizes)), "x": {}, "at": {}}
    if case["op"] == "shard":
        here, st["start"], end = pieces_of(case, sizes, case["rank"])
        st["x"]["f32"], st["at"]["f32"] = noise(here, std, g, torch.float32), (np.arange(len(sizes)), here, here)
        # the other ranks' sums, as their shards of the same gradient have them; this rank's row is its own to fill
        k = case["world"]
        n = np.stack([pieces_of(case, sizes, r)[0] for r in range(k)]).astype(np.float64)
        rows = {2: n * std * std, 1: n * std * math.sqrt(2 / math.pi), 0: std * np.sqrt(2 * np.log(n + 1))}[case["p"]] * case["scale"] ** max(case["p"], 1)
        st["sums"] = torch.tensor(rows, device="cuda") * (0.9 + 0.2 * torch.rand(k, len(sizes), device="cuda", generator=g))
        st["sums"][case["rank"]] = 0
        return st
    for t in sorted(set(types)):
        at = np.array([i for i, u in enumerate(types) if u == t])
        n = np.array([sizes[i] for i in at])
        padded = -(-n // case["align"]) * case["align"]
        x = noise(padded, std[at] / case["scale"] if case["scale"] == UNSCALE else std[at], g, DTYPES[t])
        if case["align"] > 1:  # the gaps hold zeros
            for a, b in zip(np.cumsum(padded) - padded + n, np.cumsum(padded)):
                if b > a:
                    x[a:b] = 0
        st["x"][t], st["at"][t] = x, (at, n, padded)
    return st


def prepare(case, seed):
    st = inputs(case, seed)
    if case["op"] != "norms":
        st["limits"] = limits(case, st["sizes"])
    st["y"] = {t: x if case.get("out", "same") == "same" else torch.empty_like(x, dtype=DTYPES[case["out"]]) for t, x in st["x"].items()}
    st["count"] = max(st["groups_of"]) + 1
    # the plain form's layout: each tensor's stretch in pieces of at most PIECE elements
    st["plan"], st["splits"] = {}, {t: padded.tolist() for t, (_, _, padded) in st["at"].items()}
    for t, (at, n, padded) in st["at"].items():
        k = -(-padded // PIECE)
        first = np.full(int(k.sum()), PIECE, dtype=np.int64)
        last = np.cumsum(k)[k > 0] - 1
        first[last] = (padded - (k - 1) * PIECE)[k > 0]
        st["plan"][t] = [torch.tensor(a, device="cuda") for a in (first, k, at, padded)]
    st["of"] = torch.tensor(st["groups_of"], device="cuda")
    if case["op"] != "norms":
        st["max"] = torch.tensor(st["limits"], dtype=torch.float64, device="cuda")
    if own:
        st["clip"] = handle(st)
    return st


def views(st, buffers):
    """The tensors of a list as views of the buffers."""
    out = [None] * len(st["sizes"])
    for t, (at, n, padded) in st["at"].items():
        for i, a, k in zip(at.tolist(), (np.cumsum(padded) - padded).tolist(), n.tolist()):
            out[i] = buffers[t][a:a + k]
    return out


# ------------------------------------------------------------- plain form
def plain_sums(st):
    """The tensors' sums of |s x|^p, or their largest |s x|, in 64 bits."""
    p, s = st["case"]["p"], st["case"]["scale"]
    sums = torch.zeros(len(st["sizes"]), dtype=torch.float64, device="cuda")
    how = "max" if p == 0 else "sum"
    for t, x in st["x"].items():
        first, k, at, _ = st["plan"][t]
        v = x.float().mul(s)
        v = v.square() if p == 2 else v.abs()
        v = v if p == 0 else v.double()
        v = torch.segment_reduce(v, how, lengths=first, unsafe=True, initial=0)
        sums[at] = torch.segment_reduce(v, how, lengths=k, unsafe=True, initial=0).double()
    return sums


def plain_norms(st, sums):
    """The norms of tensors, groups and all, in 64 bits."""
    p = st["case"]["p"]
    groups = torch.zeros(st["count"], dtype=torch.float64, device="cuda")
    groups = groups.scatter_reduce(0, st["of"], sums, "amax" if p == 0 else "sum")
    whole = sums.amax() if p == 0 else sums.sum()
    return [v.sqrt() if p == 2 else v for v in (sums, groups, whole)]


def run(st):
    if own:
        return run_own(st)
    case = st["case"]
    sums = plain_sums(st)
    if case["op"] == "shard":
        st["sums"][case["rank"]] = sums
        sums = st["sums"].amax(0) if case["p"] == 0 else st["sums"].sum(0)
    tensors, groups, whole = plain_norms(st, sums)
    out = {"tensor_norms": tensors.float(), "group_norms": groups.float(), "norm": whole.float()}
    if case["op"] == "norms":
        return out
    factor = (st["max"] / (groups + 1e-6)).clamp(max=1).float()[st["of"]] * case["scale"]
    for t, x in st["x"].items():
        _, _, at, padded = st["plan"][t]
        if len(at) <= FEW:
            for y, v, f in zip(st["y"][t].split(st["splits"][t]), x.split(st["splits"][t]), factor[at]):
                y.copy_(v.float() * f)
        else:
            st["y"][t].copy_(x.float() * torch.repeat_interleave(factor[at], padded, output_size=x.numel()))
    out["grads"] = dict(st["y"])
    return out


# ------------------------------------------------------- framework's form
def handle(st):
    """What a training loop makes once: the clip over its gradients' buffers."""
    from fsdp_sharded_mixed_flatparameter_gb300 import GradClip
    case = st["case"]
    kw = {"norm_type": case["p"] or math.inf, "group_of": st["groups_of"], "max_norm": st.get("limits", math.inf), "device": "cuda"}
    if case["op"] == "shard":
        return GradClip.of_shard(st["sizes"], st["x"]["f32"], st["start"], **kw)
    clip = GradClip(st["sizes"], **kw)
    same = case["op"] == "norms" or case["out"] == "same"
    for t, y in st["y"].items():  # the gaps between tensors are nobody's
        if not same:
            y.zero_()
    clip.register_grads(views(st, st["x"]), out=None if same else views(st, st["y"]))
    return clip


def run_own(st):
    case, clip = st["case"], st["clip"]
    if case["op"] == "norms":
        clip.launch_norms(scale=case["scale"])
    elif case["op"] == "clip":
        clip.launch(scale=case["scale"])
    else:
        clip.launch_sums(scale=case["scale"])
        st["sums"][case["rank"]].copy_(clip.tensor_sums)  # this rank's row of the all-gather
        clip.launch(scale=case["scale"], gathered_sums=st["sums"])
    out = {"tensor_norms": clip.tensor_norms, "group_norms": clip.group_norms, "norm": clip.norm}
    if case["op"] != "norms":
        out["grads"] = dict(st["y"])
    return out


def work(case):
    """Bytes: every gradient read once and, where it is clipped, written once; no write where the norm is below the limit. Operations: a square and a sum, and a product."""
    sizes = sizes_of(case)
    if case["op"] == "shard":
        here = int(pieces_of(case, sizes, case["rank"])[0].sum())
        return {"bytes": 8 * here + 8 * case["world"] * len(sizes), "flops": 3 * here}
    size = {"f32": 4, "bf16": 2, "f16": 2}
    types = types_of(case, sizes)
    read = sum(n * size[t] for n, t in zip(sizes, types))
    if case["op"] == "norms" or case["limit"] > 1:
        return {"bytes": read, "flops": 2 * sum(sizes)}
    wrote = sum(n * size[t if case["out"] == "same" else case["out"]] for n, t in zip(sizes, types))
    return {"bytes": read + wrote, "flops": 3 * sum(sizes)}


# ------------------------------------------------------ 64-bit definition
def exact(case, seed):
    """The same outputs from the formulas in binary64, tensor by tensor."""
    st = inputs(case, seed)
    p, s = case["p"], case["scale"]
    kind = {2: 2.0, 1: 1.0, 0: math.inf}[p]
    norms = [torch.zeros((), dtype=torch.float64, device="cuda")] * len(st["sizes"])
    wide = {}
    for t, (at, n, padded) in st["at"].items():
        wide[t] = st["x"][t].double().mul_(s)
        for i, a, k in zip(at.tolist(), (np.cumsum(padded) - padded).tolist(), n.tolist()):
            if k:
                norms[i] = torch.linalg.vector_norm(wide[t][a:a + k], kind)
    norms = torch.stack(norms)
    if case["op"] == "shard":
        # a tensor's norm over all ranks, from the norms of its pieces
        pieces = st["sums"] ** (0.5 if p == 2 else 1.0)
        pieces[case["rank"]] = norms
        norms = torch.linalg.vector_norm(pieces, kind, dim=0)
    of = np.asarray(st["groups_of"])
    members = [torch.tensor(a, device="cuda") for a in np.split(np.argsort(of, kind="stable"), np.cumsum(np.bincount(of))[:-1])]
    groups = torch.stack([torch.linalg.vector_norm(norms[a], kind) for a in members])
    out = {"tensor_norms": norms, "group_norms": groups, "norm": torch.linalg.vector_norm(norms, kind)}
    if case["op"] == "norms":
        return out
    coef = (torch.tensor(limits(case, st["sizes"]), dtype=torch.float64, device="cuda") / (groups + 1e-6)).clamp(max=1.0).tolist()
    for t, (at, n, padded) in st["at"].items():
        for i, a, k in zip(at.tolist(), (np.cumsum(padded) - padded).tolist(), n.tolist()):
            wide[t][a:a + k] *= coef[of[i]]
    out["grads"] = wide
    return out

"""The cases by which the many-tensor AdamW, the 8-bit optimizer states and their conversion are measured.

Four operators:

* ``list`` with ``bits`` 32: one AdamW step over many separate tensors at once (fp32 master, exp_avg, exp_avg_sq of
  their own, parameter groups, a low-precision copy);
* ``list`` with ``bits`` 8: the same with both moments held in 8 bits;
* ``shard``: the 8-bit step over one rank's flat shard, the grads read through the FlatParameter's tensor table;
* ``pack`` / ``unpack``: a flat shard's fp32 moments into 8 bits and back (checkpoints, resuming a 32-bit run).

8-bit state: exp_avg and the square root of exp_avg_sq as float8_e4m3fn values times one power of two per block of 256
elements.  The codes come back as float8 tensors beside the blocks' fp32 scales: each value is code x scale.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEP = 100
BETAS, EPS, LR = (0.9, 0.95), 1e-8, 1e-4
#: weight decay of the parameter groups, given out in turn; the second is the usual group of biases and norms
DECAYS = (0.1, 0.0, 0.01)
COEF = 0.7431640625  # the clip coefficient of a step that clips


def listed():
    """The smallest calls, ordinary ones and the largest of each operator."""
    return [
        # a small model, one fp32 tensor per layer, no low-precision copy: what a launch costs
        {"name": "list32-tiny", "op": "list", "bits": 32, "sizes": "tiny", "grad": "f32", "lowp": "none", "groups": 1, "seeded": False},
        # GPT-2 small as separate tensors with decayed and undecayed groups
        {"name": "list32-gpt2", "op": "list", "bits": 32, "sizes": "gpt2", "grad": "bf16", "lowp": "bf16", "groups": 2, "seeded": False},
        # thousands of log-uniform sizes from one element up: adapters, norms, experts
        {"name": "list32-ragged", "op": "list", "bits": 32, "sizes": "ragged", "tensors": 4000, "elements": 302390543, "grad": "bf16", "lowp": "bf16", "groups": 3, "seeded": False},
        # four layers of Llama-7B with embedding and head: the bandwidth of large tensors
        {"name": "list32-llama4", "op": "list", "bits": 32, "sizes": "llama", "layers": 4, "grad": "bf16", "lowp": "bf16", "groups": 2, "seeded": False},
        # the small model with 8-bit moments, rounded to nearest
        {"name": "list8-tiny", "op": "list", "bits": 8, "sizes": "tiny", "grad": "f32", "lowp": "none", "groups": 1, "seeded": False},
        # GPT-2 small, 8-bit moments with stochastic rounding
        {"name": "list8-gpt2", "op": "list", "bits": 8, "sizes": "gpt2", "grad": "bf16", "lowp": "bf16", "groups": 2, "seeded": True},
        # eight layers of Llama-7B on one GPU, where 8-bit moments save most
        {"name": "list8-llama8", "op": "list", "bits": 8, "sizes": "llama", "layers": 8, "grad": "bf16", "lowp": "bf16", "groups": 2, "seeded": True},
        # ZeRO-1 over GPT-2, rank 3 of 8: the last micro-batch added to the fp32 sum of the earlier ones
        {"name": "shard8-gpt2", "op": "shard", "sizes": "gpt2", "world": 8, "rank": 3, "grad": "bf16", "lowp": "bf16", "acc": True, "seeded": False},
        # 20,000 ragged tensors, rank 2 of 4: tensor borders inside most blocks
        {"name": "shard8-ragged", "op": "shard", "sizes": "ragged", "tensors": 20000, "elements": 1507457739, "world": 4, "rank": 2, "grad": "bf16", "lowp": "bf16", "acc": False, "seeded": True},
        # Llama-13B under ZeRO-3, rank 7 of 8: one flat fp16 grad of the shard
        {"name": "shard8-llama13b", "op": "shard", "sizes": "flat", "elements": 1626983040, "world": 1, "rank": 0, "grad": "f16", "lowp": "f16", "acc": False, "seeded": False},
        # a GPT-2 ZeRO-1 shard's moments packed when a 32-bit run goes on in 8 bits
        {"name": "pack-gpt2", "op": "pack", "elements": 15554976},
        # a Llama-13B shard's moments unpacked for a 32-bit checkpoint
        {"name": "unpack-llama13b", "op": "unpack", "elements": 1626983040},
    ]


def draw(rng):
    """One more case: any operator, sizes log-uniform over its listed range."""
    def spread(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    op = rng.choice(["list", "list", "shard", "pack", "unpack"])
    if op in ("pack", "unpack"):
        return {"op": op, "elements": spread(50000, 1600000000) | 1}
    grad = rng.choice(["f32", "bf16", "f16"])
    lowp = rng.choice(["none", "bf16", "f16"])
    tensors = spread(1, 4000 if op == "list" else 20000)
    if op == "list":
        bits = rng.choice([8, 32])
        elements = max(spread(1000000, 900000000 if bits == 32 else 1600000000), 4 * tensors)
        return {"op": op, "bits": bits, "sizes": "ragged", "tensors": tensors, "elements": elements, "grad": grad, "lowp": lowp,
                "groups": rng.randint(1, 3), "seeded": bits == 8 and rng.random() < 0.5}
    world = rng.choice([1, 2, 4, 8])
    elements = max(spread(4000000, 1500000000 if world > 1 else 1000000000), 4 * tensors)
    return {"op": op, "sizes": "ragged", "tensors": tensors, "elements": elements, "world": world, "rank": rng.randrange(world), "grad": grad, "lowp": lowp,
            "acc": rng.random() < 0.3, "seeded": rng.random() < 0.5}


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
    n = np.maximum(1, np.floor(w * (total / w.sum()))).astype(np.int64)
    n[int(np.argmax(n))] += total - int(n.sum())
    return [int(x) for x in n]


def shard_of(case, total):
    chunk = -(-total // case["world"])
    start = min(case["rank"] * chunk, total)
    return start, min(start + chunk, total)


def blocks(n):
    return -(-n // BLOCK)


def scalars(wd):
    """The step's scalars in binary64: lr / (1 - beta1^t), sqrt(1 - beta2^t), 1 - lr * wd."""
    return LR / (1 - BETAS[0] ** STEP), math.sqrt(1 - BETAS[1] ** STEP), 1 - LR * wd


# ----------------------------------------------------------------- inputs
def moments(n, g):
    """exp_avg and exp_avg_sq as training leaves them: magnitudes that differ by block, some elements never touched."""
    nb = blocks(n)
    mag = torch.exp2(torch.rand(nb, 1, device="cuda", generator=g) * 12 - 20)
    m = torch.randn(nb, BLOCK, device="cuda", generator=g)
    v = torch.rand(nb, BLOCK, device="cuda", generator=g)
    quiet = v < 0.01
    v.mul_(1.5).add_(0.05).mul_(mag).mul_(mag)
    m.mul_(mag).mul_(0.3)
    m.masked_fill_(quiet, 0)
    v.masked_fill_(quiet, 0)
    return m.view(-1)[:n].contiguous(), v.view(-1)[:n].contiguous()


def normal(n, g, std, dtype=torch.float32):
    out = torch.empty(n, dtype=dtype, device="cuda")
    for a in range(0, n, 1 << 28):
        b = min(n, a + (1 << 28))
        out[a:b] = torch.randn(b - a, device="cuda", generator=g).mul_(std)
    return out


def clip_result():
    """A grad norm's result as the framework's norm pass leaves it on the device: {sqnorm f64, norm f64, coef f32, finite i32}."""
    norm = 1.0 / COEF
    raw = np.array([norm * norm, norm]).tobytes() + np.float32(COEF).tobytes() + np.int32(1).tobytes()
    return torch.frombuffer(bytearray(raw), dtype=torch.uint8).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case, "op": case["op"], "rounding": (seed * 0x9E3779B97F4A7C15 + 1) % (1 << 64) if case.get("seeded") else None}
    if case["op"] in ("pack", "unpack"):
        n = case["elements"]
        m, v = moments(n, g)
        if case["op"] == "pack":
            st.update(m=m, v=v, q=empty8(n))
        else:
            st.update(m=torch.empty_like(m), v=torch.empty_like(v), q=plain_pack(m, v, empty8(n)))
        if own:
            from fsdp_sharded_mixed_flatparameter_gb300 import State8
            st["state8"] = State8(*st["q"])
        return st
    sizes = sizes_of(case)
    gdt, lowp = DTYPES[case["grad"]], DTYPES.get(case["lowp"])
    st["clip"] = clip_result()
    if case["op"] == "list":
        # each tensor starts on a block's border of one storage, as separate allocations would; the gaps hold zeros
        starts = np.concatenate([[0], np.cumsum([blocks(n) * BLOCK for n in sizes])]).tolist()
        total = starts[-1]
        m, v = moments(total, g)
        p, x = normal(total, g, 0.02), normal(total, g, 1e-3, gdt)
        ends = torch.tensor([s + n for s, n in zip(starts, sizes)], device="cuda")
        of = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor([blocks(n) for n in sizes], device="cuda"))
        gap = torch.arange(BLOCK, device="cuda")[None, :] >= (ends[of] - torch.arange(len(of), device="cuda") * BLOCK)[:, None]
        for t in (m, v, p, x):
            t.view(-1, BLOCK).masked_fill_(gap, 0)
        del gap
        st.update(p=p, x=x, lowp=torch.zeros(total, dtype=lowp, device="cuda") if lowp else None, of=of, groups_of=torch.arange(len(sizes), device="cuda") % case["groups"],
                  places=torch.arange(total // BLOCK, device="cuda") - torch.tensor(starts[:-1], device="cuda")[of] // BLOCK)
        views = lambda t: None if t is None else [t[s:s + n] for s, n in zip(starts, sizes)]  # noqa: E731
        q = None
        if case["bits"] == 8:
            q = plain_pack(m, v, empty8(total))
            del m, v
        if own:
            from fsdp_sharded_mixed_flatparameter_gb300 import TensorListAdamW
            opt = TensorListAdamW(views(p), lowp=views(st["lowp"]), group_of=[i % case["groups"] for i in range(len(sizes))], state_bits=case["bits"], rounding_seed=st["rounding"],
                                  groups=[{"lr": LR, "betas": BETAS, "eps": EPS, "weight_decay": DECAYS[k]} for k in range(case["groups"])])
            opt.t = STEP - 1
            opt.register_grads(views(x))
            if q is None:
                opt.exp_avg.copy_(m)
                opt.exp_avg_sq.copy_(v)
                m, v = opt.exp_avg, opt.exp_avg_sq
            else:
                for a, b in zip(opt.state8, q):
                    a.copy_(b)
                q = tuple(opt.state8)
            st["opt"] = opt
        st.update({"q": q} if q is not None else {"m": m, "v": v})
        return st
    # one rank's shard of the flat parameter; the grads of the tensors that it touches, each on a 128-element border
    start, end = shard_of(case, sum(sizes))
    first, pos, skipped, mine = 0, 0, 0, []
    for n in sizes:
        if pos + n > start and pos < end:
            first = first if mine else pos
            mine.append(n)
        elif not mine:
            skipped += 1
        pos += n
    n = end - start
    at = np.concatenate([[0], np.cumsum([-(-k // 128) * 128 for k in mine])]).tolist()
    x = normal(at[-1], g, 1e-3, gdt)
    grads = [x[a:a + k] for a, k in zip(at, mine)]
    m, v = moments(n, g)
    st.update(grads=grads, lo=start - first, n=n, start=start, p=normal(n, g, 0.02), lowp=torch.zeros(n, dtype=lowp, device="cuda") if lowp else None,
              acc=normal(n, g, 1e-3) if case["acc"] else None, scale=0.125 if case["acc"] else 1.0, q=plain_pack(m, v, empty8(n)))
    if own:
        from fsdp_sharded_mixed_flatparameter_gb300 import State8, device_table, zero_tensor_table
        table, total = zero_tensor_table([None] * skipped + grads + [None] * (len(sizes) - skipped - len(grads)), sizes)
        st.update(state8=State8(*st["q"]), table=device_table(table, len(sizes), "cuda"), tensors=len(sizes), total=total)
    return st


# ------------------------------------------------------------- plain form
def empty8(n):
    """(exp_avg codes, their scales, root codes, their scales) for n elements."""
    nb = blocks(n)
    return tuple(torch.zeros(k, dtype=d, device="cuda") for k, d in ((n, torch.float8_e4m3fn), (nb, torch.float32), (n, torch.float8_e4m3fn), (nb, torch.float32)))


def rows(t):
    """A flat tensor as rows of one block, the last one filled with zeros."""
    if t.numel() % BLOCK:
        z = t.new_zeros(blocks(t.numel()) * BLOCK)
        z[:t.numel()] = t
        t = z
    return t.view(-1, BLOCK)


def put(dst, src):
    dst.copy_(src.reshape(-1)[:dst.numel()])


def block_scale(x):
    """The least power of two S, at least 2^-126, with max|x| <= 448 S in each row, and 1 / S."""
    e = ((x.abs().amax(1, keepdim=True).view(torch.int32) + 0x1FFFFF) >> 23).sub_(8).clamp_(min=1)
    return (e << 23).view(torch.float32), ((254 - e) << 23).view(torch.float32)


def pcg(x):
    """The 32-bit PCG permutation (O'Neill's RXS-M-XS) of whole numbers below 2^32, in 64-bit integers."""
    x = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    x = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) & 0xFFFFFFFF
    return (x >> 22) ^ x


def pcg32(x):
    """pcg() on an int32 tensor that holds the 32 bits (its products wrap; shifts are masked to be logical)."""
    x = x * 747796405 + (2891336453 - (1 << 32))
    s = ((x >> 28) & 15) + 4
    x = (((x >> s) & (0x7FFFFFFF >> (s - 1))) ^ x) * 277803737
    return ((x >> 22) & 0x3FF) ^ x


def rounding_bits(seed, stream, row):
    """The rounding words of blocks: one 32-bit word for each pair of elements, an int32 row of 128 for each block. From the seed, the step, the stream (a list's tensor
    number; a shard's start) and the pair's index in the tensor or shard; row: the blocks' numbers there."""
    pair = row[:, None] * (BLOCK // 2)
    h = pcg(STEP ^ pcg((seed >> 32) ^ pcg(seed & 0xFFFFFFFF)))
    h = pcg((pair >> 32) ^ pcg(stream ^ h))
    low = (h ^ (pair & 0xFFFFFFFF)) & 0xFFFFFFFF
    low = torch.where(low >= 1 << 31, low - (1 << 32), low).int()
    return pcg32(low ^ torch.arange(BLOCK // 2, device="cuda", dtype=torch.int32)[None, :])


def halves(words):
    """The 7 + 7 rounding bits of each element: the low half of a pair's word is the even element's."""
    w = torch.stack((words, words >> 16), -1).reshape(words.shape[0], BLOCK)
    return w & 127, w >> 7 & 127


def code(x, bits=None):
    """x (at most 448 in size) as e4m3 values: to nearest, or by 7 random bits of each element (0..127)."""
    if bits is None:
        return x.to(torch.float8_e4m3fn)
    a = x.abs()
    unit = (((a.view(torch.int32) >> 23).clamp_(min=121)) - 3 << 23).view(torch.float32)  # the e4m3 grid's spacing at a
    down = torch.floor(a / unit * 128) + bits
    return torch.copysign(torch.floor(down / 128) * unit, x).to(torch.float8_e4m3fn)


def encode(m, r, q, words=None):
    """Moments' rows (exp_avg and the root of exp_avg_sq) into the 8-bit state; a nonzero root never becomes zero."""
    sm, im = block_scale(m)
    sr, ir = block_scale(r)
    x, y = m * im, r * ir
    y = torch.where(r > 0, y.clamp(min=2.0 ** -9), y)
    bm = br = None
    if words is not None:
        bm, br = halves(words)
    put(q[0], code(x, bm))
    put(q[1], sm)
    put(q[2], code(y, br))
    put(q[3], sr)
    return q


def decode(q):
    """exp_avg and the root of exp_avg_sq, as rows."""
    return rows(q[0]).float() * q[1][:, None], rows(q[2]).float() * q[3][:, None]


def plain_pack(m, v, q):
    return encode(rows(m), rows(v).sqrt(), q)


def plain_unpack(q, m, v):
    a, r = decode(q)
    put(m, a)
    put(v, r * r)


def f32(x):
    return float(np.float32(x))


def plain_step(p, m, v, g, decay):
    """The AdamW step on rows; p and the moments change in place. Gives back the square root of the new exp_avg_sq."""
    step, bc2, _ = scalars(0)
    p.mul_(decay)
    m.mul_(f32(BETAS[0])).add_(g, alpha=f32(1 - BETAS[0]))
    v.mul_(f32(BETAS[1])).addcmul_(g * f32(1 - BETAS[1]), g)
    root = v.sqrt()
    p.sub_(m / (root / f32(bc2) + f32(EPS)) * f32(step))
    return root


def words_of(st, a, b):
    """The rounding words of blocks a..b of the state."""
    if st["rounding"] is None:
        return None
    if st["op"] == "list":
        return rounding_bits(st["rounding"], st["of"][a:b, None], st["places"][a:b])
    return rounding_bits(st["rounding"], st["start"] & 0xFFFFFFFF, torch.arange(a, b, device="cuda"))


def run(st):
    op = st["op"]
    if own:
        return run_own(st)
    if op == "pack":
        return {"state": list(plain_pack(st["m"], st["v"], st["q"]))}
    if op == "unpack":
        plain_unpack(st["q"], st["m"], st["v"])
        return {"exp_avg": st["m"], "exp_avg_sq": st["v"]}
    coef = st["clip"][16:20].view(torch.float32)
    if op == "list":
        g = st["x"].float().view(-1, BLOCK) * coef
        decay = torch.tensor([f32(scalars(d)[2]) for d in DECAYS], device="cuda")[st["groups_of"][st["of"]]][:, None]
        p = st["p"].view(-1, BLOCK)
    else:
        x = torch.cat(st["grads"])[st["lo"]:st["lo"] + st["n"]].float() * st["scale"]
        if st["acc"] is not None:
            x = st["acc"] + x
        g, decay, p = rows(x * coef), f32(scalars(DECAYS[0])[2]), rows(st["p"])
    if "m" in st:
        plain_step(p, st["m"].view(-1, BLOCK), st["v"].view(-1, BLOCK), g, decay)
        out = {"exp_avg": st["m"], "exp_avg_sq": st["v"]}
    else:
        m, r = decode(st["q"])
        root = plain_step(p, m, r * r, g, decay)
        del r
        out = {"state": list(encode(m, root, st["q"], words_of(st, 0, p.shape[0])))}
    if p.data_ptr() != st["p"].data_ptr():
        put(st["p"], p)
    out["master"] = st["p"]
    if st["lowp"] is not None:
        out["lowp"] = st["lowp"].copy_(st["p"])
    return out


# ------------------------------------------------------- framework's form
def run_own(st):
    op = st["op"]
    import fsdp_sharded_mixed_flatparameter_gb300 as zs
    if op == "pack":
        zs.zero_state8_pack(st["m"], st["v"], st["state8"])
        return {"state": list(st["q"])}
    if op == "unpack":
        zs.zero_state8_unpack(st["state8"], st["m"], st["v"])
        return {"exp_avg": st["m"], "exp_avg_sq": st["v"]}
    if op == "list":
        st["opt"].launch_step(norm_result=st["clip"])
        out = {"exp_avg": st["m"], "exp_avg_sq": st["v"]} if "m" in st else {"state": list(st["q"])}
    else:
        zs.zero_adamw_step8_tensors(st["p"], st["state8"], st["table"], st["tensors"], st["total"], st["grads"][0].dtype, st["start"], st["scale"], st["lowp"], LR, BETAS[0], BETAS[1],
                                    EPS, DECAYS[0], STEP, st["clip"], acc=st["acc"], rounding_seed=st["rounding"])
        out = {"state": list(st["q"])}
    out["master"] = st["p"]
    if st["lowp"] is not None:
        out["lowp"] = st["lowp"]
    return out


def work(case):
    """Bytes: every input once, every output once. Operations: the update's multiplications, additions, divisions and roots."""
    if case["op"] in ("pack", "unpack"):
        n = case["elements"]
        return {"bytes": 10 * n + 8 * blocks(n), "flops": 4 * n}
    sizes = sizes_of(case)
    n = sum(sizes)
    nb = sum(blocks(k) for k in sizes)
    if case["op"] == "shard":
        a, b = shard_of(case, n)
        n, nb = b - a, blocks(b - a)
    per = (4 if case["grad"] == "f32" else 2) + 8 + (0 if case["lowp"] == "none" else 2)
    per += 16 if case.get("bits") == 32 else 4
    if case.get("acc"):
        per += 4
    return {"bytes": per * n + (0 if case.get("bits") == 32 else 16 * nb), "flops": 16 * n}


# ------------------------------------------------------ 64-bit definition
def exact(case, seed):
    """The same outputs from the formulas in binary64, a piece of blocks at a time."""
    st = prepare_inputs(case, seed)
    wide = torch.float64
    op = case["op"]
    n = st["p"].numel() if "p" in st else st["m"].numel()
    # rounding to 8 bits is part of the definition: to_grid gives the value that a code stands for
    outs = {}

    def place(key, size):
        if key not in outs:
            outs[key] = torch.empty(size, dtype=wide, device="cuda")
        return outs[key]

    group = None
    if op == "list":
        group = torch.tensor([scalars(d)[2] for d in DECAYS], dtype=wide, device="cuda")[st["groups_of"][st["of"]]]
    x_all = None
    if op == "shard":
        x_all = torch.cat(st["grads"])[st["lo"]:st["lo"] + st["n"]]
    step, bc2, decay1 = scalars(DECAYS[0])
    piece = 1 << 25
    for a in range(0, n, piece):
        b = min(n, a + piece)
        ba, bb = a // BLOCK, blocks(b)

        def block_rows(t):
            z = torch.zeros((bb - ba) * BLOCK, dtype=wide, device="cuda")
            z[:b - a] = t[a:b].to(wide)
            return z.view(-1, BLOCK)

        if "q" in st and op != "pack":
            m = block_rows(st["q"][0]) * st["q"][1][ba:bb, None].to(wide)
            root = block_rows(st["q"][2]) * st["q"][3][ba:bb, None].to(wide)
            v = root.square()
        else:
            m, v = block_rows(st["m"]), block_rows(st["v"])
        if op == "unpack":
            place("exp_avg", n)[a:b] = m.view(-1)[:b - a]
            place("exp_avg_sq", n)[a:b] = v.view(-1)[:b - a]
            continue
        if op != "pack":
            gr = block_rows(st["x"] if op == "list" else x_all)
            if op == "shard":
                gr = gr * st["scale"]
                if st["acc"] is not None:
                    gr = gr + block_rows(st["acc"])
            gr = gr * COEF
            m = BETAS[0] * m + (1 - BETAS[0]) * gr
            v = BETAS[1] * v + (1 - BETAS[1]) * gr * gr
            dec = group[ba:bb, None] if group is not None else decay1
            w = block_rows(st["p"]) * dec - step * m / (v.sqrt() / bc2 + EPS)
            place("master", n)[a:b] = w.view(-1)[:b - a]
            if st["lowp"] is not None:
                place("lowp", n)[a:b] = w.view(-1)[:b - a]
            if "q" not in st:
                place("exp_avg", n)[a:b] = m.view(-1)[:b - a]
                place("exp_avg_sq", n)[a:b] = v.view(-1)[:b - a]
                continue
        root = v.sqrt()
        rnd = (None, None) if st["rounding"] is None else halves(words_of(st, ba, bb))
        for j, (t, r) in enumerate(zip((m, root), rnd)):
            big = t.abs().amax(1, keepdim=True)
            frac, e = torch.frexp(big)
            s = torch.exp2((e.to(wide) - 9 + (frac > 0.875).to(wide)).clamp(min=-126))
            s = torch.where(big > 0, s, torch.full_like(s, 2.0 ** -126))
            c = t / s
            size = c.abs()
            if j == 1:
                size = torch.where(size > 0, size.clamp(min=2.0 ** -9), size)
            unit = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
            grid = torch.round(size / unit) if r is None else torch.floor((torch.floor(size / unit * 128) + r) / 128)
            place("code%d" % j, n)[a:b] = torch.copysign(grid * unit, c).view(-1)[:b - a]
            place("scale%d" % j, blocks(n))[ba:bb] = s[:, 0]
    if "code0" in outs:
        outs["state"] = [outs.pop(k) for k in ("code0", "scale0", "code1", "scale1")]
    return outs


def prepare_inputs(case, seed):
    """prepare()'s inputs without the framework's handles."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was

"""AdamW over many separate tensors: bit for bit the flat AdamW tensor by tensor (fp32 moments), the 64-bit formulas
(both widths), groups, alignments, absent grads, skips, graphs, checkpoints."""
import math

import numpy as np
import pytest
import torch

import _ref8 as R
import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from _helpers import norm_result_tensor, offset_view
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs
from test_gpu_state8 import DT, check_step, clone, codes_view, f64, gen, host, random_state8, same

pytestmark = pytest.mark.gpu

SIZES = [1, 0, 255, 256, 257, 2047, 2048, 2049, 3, 70001, 4096, 1, 0]
GROUPS = [dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1),
          dict(lr=3e-3, betas=(0.8, 0.99), eps=1e-6, weight_decay=0.0),
          dict(lr=1e-2, betas=(0.0, 0.9), eps=1e-8, weight_decay=0.01)]


def hp_of(g):
    return (g["lr"], *g["betas"], g["eps"], g["weight_decay"])


class Case:
    """A list of tensors with buffers at chosen offsets, and its grads."""

    def __init__(self, sizes, bits, gdt, lowp, offsets=(0, 0, 0, 0), seed=0, absent=(), n_groups=3):
        g = gen(seed + bits)
        op, os, og, ol = offsets
        self.sizes, self.bits = sizes, bits
        self.group_of = [i % n_groups for i in range(len(sizes))]
        self.n_groups = n_groups
        self.p = [offset_view(n, torch.float32, op, "cuda", torch.randn(n, generator=g)) for n in sizes]
        if bits == 8:
            self.state = [random_state8(n, g, os) if n else zs.State8(*zs.new_state8(0, "cuda")) for n in sizes]
        else:
            self.state = [(offset_view(n, torch.float32, os, "cuda", torch.randn(n, generator=g) * 1e-2),
                           offset_view(n, torch.float32, os, "cuda", torch.rand(n, generator=g) * 1e-4)) for n in sizes]
        self.x = [None if i in absent else offset_view(n, DT[gdt], og, "cuda", (torch.randn(n, generator=g) * 1e-2).to(DT[gdt]))
                  for i, n in enumerate(sizes)]
        self.lowp = None if lowp is None else [None if i % 5 == 4 else offset_view(n, DT[lowp], ol, "cuda", torch.zeros(n))
                                               for i, n in enumerate(sizes)]
        self.list = zs.zero_tensor_list(self.p, self.state, self.lowp, self.group_of, n_groups, bits)
        self.grads = zs.device_table(zs.zero_tensor_table(self.x, sizes)[0], len(sizes), "cuda")
        self.gdt = DT[gdt]

    def call(self, step=3, scale=0.5, **kw):
        zs.zero_adamw_list(self.list, self.grads, self.gdt, scale, [hp_of(GROUPS[g]) for g in range(self.n_groups)], step,
                           **kw)

    def everything(self):
        return [t for s in self.state for t in s] + self.p + [c for c in self.lowp or () if c is not None]


def bits_of(ts):
    return [t.detach().cpu().view(torch.uint8).clone() for t in ts]


@pytest.mark.parametrize("gdt,lowp", [("f32", None), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("offsets", [(0, 0, 0, 0), (0, 0, 1, 1), (1, 1, 0, 0), (3, 5, 7, 2)])
def test_32_bits_is_the_flat_adamw_bit_for_bit(gdt, lowp, offsets):
    c = Case(SIZES, 32, gdt, lowp, offsets, absent=(5, 8))
    clip = norm_result_tensor("cuda", coef=0.625)
    want = []
    for i, n in enumerate(SIZES):
        p, m, v = (t.clone() for t in (c.p[i], *c.state[i]))
        lp = None if c.lowp is None or c.lowp[i] is None else c.lowp[i].clone()
        g = torch.zeros(n, device="cuda") if c.x[i] is None else c.x[i].float() * 0.5
        if n:
            zs.zero_adamw_step(p, m, v, g, lp, *hp_of(GROUPS[c.group_of[i]]), 3, clip)
        want.append((p, m, v, lp))
    c.call(clip=clip)
    for i, (p, m, v, lp) in enumerate(want):
        for a, b in ((c.p[i], p), (c.state[i][0], m), (c.state[i][1], v)):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), i
        if lp is not None:
            assert torch.equal(c.lowp[i].view(torch.int16), lp.view(torch.int16)), i


@pytest.mark.parametrize("gdt", ["f32", "bf16", "f16"])
def test_32_bits_against_the_formulas(gdt):
    c = Case(SIZES, 32, gdt, None)
    before = [(f64(p), f64(s[0]), f64(s[1])) for p, s in zip(c.p, c.state)]
    c.call(scale=0.3)
    for i, n in enumerate(SIZES):
        h = GROUPS[c.group_of[i]]
        p, m, v = before[i]
        g, err = R.grad(f64(c.x[i]), float(np.float32(0.3)))
        out = R.step(p, m, v, g, err, lr=h["lr"], b1=h["betas"][0], b2=h["betas"][1], eps=h["eps"], wd=h["weight_decay"],
                     t=3)
        R.check_close(f64(c.p[i]), *out["p"], f"master {i}")
        R.check_close(f64(c.state[i][0]), *out["m"], f"exp_avg {i}")
        R.check_close(f64(c.state[i][1]), *out["v"], f"exp_avg_sq {i}")


@pytest.mark.parametrize("seed", [None, 0xFEDCBA9876543210])
@pytest.mark.parametrize("gdt,lowp", [("f32", None), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("offsets", [(0, 0, 0, 0), (0, 0, 1, 1), (1, 1, 0, 0), (0, 3, 7, 2)])
def test_8_bits_against_the_formulas(gdt, lowp, offsets, seed):
    c = Case(SIZES, 8, gdt, lowp, offsets, absent=(5, 8))
    before = [(f64(p), host(s)) for p, s in zip(c.p, c.state)]
    c.call(clip=norm_result_tensor("cuda", coef=0.625), rounding_seed=seed, rounding_stream=40)
    for i, n in enumerate(SIZES):
        if not n:
            continue
        h = GROUPS[c.group_of[i]]
        g, err = R.grad(np.zeros(n) if c.x[i] is None else f64(c.x[i]), 0.5, None, 0.625)
        check_step(before[i][0], before[i][1], g, err, c.p[i], c.lowp and c.lowp[i], c.state[i], seed=seed, stream=40 + i,
                   hp=dict(lr=h["lr"], b1=h["betas"][0], b2=h["betas"][1], eps=h["eps"], wd=h["weight_decay"]))


@pytest.mark.parametrize("bits", [8, 32])
def test_nothing_outside_the_tensors_is_written(bits):
    # each buffer inside a larger one with a guard on both sides
    n, pad = 2500, 64
    guard = {}

    def guarded(name, dtype, k):
        t = torch.full((k + 2 * pad,), 3, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda")
        guard[name] = (t, k)
        v = t[pad:pad + k]
        v.zero_()
        return v.view(dtype)

    p, lp = guarded("p", torch.float32, n), guarded("lowp", torch.bfloat16, n)
    if bits == 8:
        b = zs.state8_blocks(n)
        st = zs.State8(guarded("m", torch.float8_e4m3fn, n), guarded("ms", torch.float32, b),
                       guarded("r", torch.float8_e4m3fn, n), guarded("rs", torch.float32, b))
    else:
        st = (guarded("m", torch.float32, n), guarded("v", torch.float32, n))
    x = torch.randn(n, generator=gen(0)).cuda()
    grads = zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda")
    tl = zs.zero_tensor_list([p], [st], [lp], state_bits=bits)
    zs.zero_adamw_list(tl, grads, torch.float32, 1.0, [hp_of(GROUPS[0])], 1)
    for name, (t, k) in guard.items():
        assert (t[:pad] == 3).all() and (t[pad + k:] == 3).all(), name
        assert (t[pad:pad + k].float() != 0).any(), name


@pytest.mark.parametrize("bits", [8, 32])
def test_skip_and_repeat(bits):
    a, b = (Case(SIZES, bits, "bf16", "bf16") for _ in range(2))
    before = bits_of(a.everything())
    a.call(clip=norm_result_tensor("cuda", finite=False))
    assert all(torch.equal(x, y) for x, y in zip(before, bits_of(a.everything())))
    a.call()
    b.call()
    assert all(torch.equal(x, y) for x, y in zip(bits_of(a.everything()), bits_of(b.everything())))


@pytest.mark.parametrize("bits,seed", [(8, None), (8, 6), (32, None)])
def test_device_scale_and_states(bits, seed):
    a, b, c = (Case(SIZES, bits, "f16", "bf16") for _ in range(3))
    a.call(step=7, scale=0.25, rounding_seed=seed)
    b.call(step=7, scale=99.0, d_scale=torch.tensor([0.25], device="cuda"), rounding_seed=seed)
    hp = torch.cat([zs.device_hparams(*hp_of(g), "cuda") for g in GROUPS])
    states = zs.new_adamw_device_state("cuda", 6).repeat(3)
    zs.zero_adamw_prepare_list_device(hp, 3, None, states)
    zs.zero_adamw_list_device(c.list, c.grads, c.gdt, 0.25, states, rounding_seed=seed)
    want = bits_of(a.everything())
    for o in (b, c):
        assert all(torch.equal(x, y) for x, y in zip(want, bits_of(o.everything())))
    # all groups step or none: a bad group, then a non-finite norm
    for bad, clip in ((True, None), (False, norm_result_tensor("cuda", finite=False))):
        h2 = hp.clone()
        if bad:
            zs.device_hparams(-1.0, 0.9, 0.9, 1e-8, 0.0, "cuda", out=h2[zs.HPARAMS_BYTES:2 * zs.HPARAMS_BYTES])
        zs.zero_adamw_prepare_list_device(h2, 3, clip, states)
        zs.zero_adamw_list_device(c.list, c.grads, c.gdt, 0.25, states, clip)
        for i in range(3):
            st = zs.decode_adamw_device_state(states[48 * i:48 * i + 48])
            assert (st.step, st.apply) == (7, False) and st.status == (zs.ZERO_EINVAL if bad and i == 1 else zs.ZERO_OK)
        assert all(torch.equal(x, y) for x, y in zip(want, bits_of(c.everything())))


def test_other_stream_and_large_list():
    rng = np.random.default_rng(0)
    sizes = [int(x) for x in np.exp(rng.uniform(0, 9, 3000))]
    a, b = (Case(sizes, 8, "bf16", "bf16") for _ in range(2))
    a.call(rounding_seed=1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b.call(rounding_seed=1, stream=st)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(bits_of(a.everything()), bits_of(b.everything())))


def test_tens_of_thousands_of_tensors():
    # four rounds of the search; empty tensors between, at the front and at the end
    rng = np.random.default_rng(3)
    sizes = [0, 0] + [int(x) for x in rng.integers(0, 40, 36000)] + [3000, 0, 0]
    total = sum(sizes)
    g = gen(0)
    flat_x, flat_p = (torch.randn(total, generator=g).cuda() for _ in range(2))
    opt = pkg.TensorListAdamW([t.clone() for t in torch.split(flat_p, sizes)], lr=1e-2, weight_decay=0.1, max_norm=1.0)
    flat = pkg.FlatShardAdamW(sizes, lr=1e-2, weight_decay=0.1, max_norm=1.0, device="cuda", master=flat_p.clone(),
                              grad_buffer=False)
    grads = list(torch.split(flat_x, sizes))  # views at any alignment
    assert opt.step(grads) == flat.step_tensors(grads)
    assert torch.equal(torch.cat([p.view(-1) for p in opt.masters]), flat.master)
    o8 = pkg.TensorListAdamW([t.clone() for t in torch.split(flat_p, sizes)], lr=1e-2, weight_decay=0.1, max_norm=1.0,
                             state_bits=8, rounding_seed=9)
    o8.step(grads)
    # the first step's moments come from zero: the update is the fp32 one but for the hardware root and reciprocal
    off = (torch.cat([p.view(-1) for p in o8.masters]) - flat.master).abs().max()
    assert off <= 16 * R.EPS * (1e-2 + float(flat.master.abs().max()))
    for i in rng.integers(0, len(sizes), 100):
        if sizes[i]:
            h = host(o8.state_of(int(i)))
            m = 0.1 * f64(grads[int(i)]) * float(np.float32(min(1.0, 1.0 / (float(flat_x.double().norm()) + 1e-6))))
            R.check_codes(h[0], h[1], m, 8 * R.EPS * np.abs(m), k=R.draws(9, 1, int(i), sizes[i])[0], name=str(i))


@pytest.mark.parametrize("bits", [8, 32])
def test_sixty_four_groups_and_pinned_grads(bits):
    sizes = [257] * 64
    hps = [(1e-3 * (k + 1), 0.9 - 0.01 * k, 0.999 - 0.005 * k, 1e-8 * (k + 1), 0.01 * k) for k in range(64)]
    a, b = (Case(sizes, bits, "bf16", "bf16", n_groups=64) for _ in range(2))
    zs.zero_adamw_list(a.list, a.grads, a.gdt, 1.0, hps, 5)
    pinned = [x.cpu().pin_memory() for x in b.x]
    grads = zs.device_table(zs.zero_tensor_table(pinned, sizes)[0], 64, "cuda")
    zs.zero_adamw_list(b.list, grads, b.gdt, 1.0, hps, 5)
    assert all(torch.equal(x, y) for x, y in zip(bits_of(a.everything()), bits_of(b.everything())))
    c = Case(sizes, bits, "bf16", "bf16", n_groups=64)
    for i in range(64):  # one tensor at a time, as a group of its own
        one = zs.zero_tensor_list(c.p[i:i + 1], c.state[i:i + 1], None if c.lowp[i] is None else c.lowp[i:i + 1],
                                  state_bits=bits)
        t = zs.device_table(zs.zero_tensor_table(c.x[i:i + 1])[0], 1, "cuda")
        zs.zero_adamw_list(one, t, c.gdt, 1.0, [hps[i]], 5)
    assert all(torch.equal(x, y) for x, y in zip(bits_of(a.everything()), bits_of(c.everything())))


def test_one_tensor_is_the_shard_step():
    n = 9999
    a = Case([n], 8, "bf16", "bf16", n_groups=1)
    q, p, lp = clone(a.state[0]), a.p[0].clone(), a.lowp[0].clone()
    a.call(rounding_seed=3, rounding_stream=8)
    zs.zero_adamw_step8_tensors(p, q, a.grads, 1, n, torch.bfloat16, 0, 0.5, lp, *hp_of(GROUPS[0]), 3, rounding_seed=3,
                                rounding_stream=8)
    assert same(a.state[0], q) and torch.equal(a.p[0], p) and torch.equal(a.lowp[0], lp)


@pytest.mark.slow
@pytest.mark.parametrize("bits", [8, 32])
def test_indices_past_2_to_31(bits):
    n = (1 << 31) + 2500
    p = torch.zeros(n, device="cuda")
    st = zs.new_state8(n, "cuda") if bits == 8 else (torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"))
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = n - 3000
    x[at:] = (torch.randn(3000, generator=gen(1)) * 1e-2).bfloat16().cuda()
    tl = zs.zero_tensor_list([p], [st], state_bits=bits)
    zs.zero_adamw_list(tl, zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda"), torch.bfloat16, 1.0,
                       [hp_of(GROUPS[0])], 1)
    assert float(p[:at].abs().max()) == 0.0
    g = f64(x[at:])
    want = -1e-2 * g / (np.abs(g) + 1e-8)
    np.testing.assert_allclose(f64(p[at:]), want, rtol=32 * R.EPS, atol=0)


# ---------------------------------------------------------- TensorListAdamW
SHAPES = [(50, 33), (7,), (64, 128), (1,), (3, 5, 200), (2049,)]


def optimizer(bits, **kw):
    masters = [torch.randn(s, generator=gen(i)).cuda() for i, s in enumerate(SHAPES)]
    lowp = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in SHAPES]
    kw = {**dict(lowp=lowp, groups=[{}, {"weight_decay": 0.0, "lr": 3e-3}], group_of=[0, 1, 0, 1, 0, 1], lr=1e-2,
                 betas=(0.9, 0.95), weight_decay=0.1, max_norm=0.5, state_bits=bits), **kw}
    return pkg.TensorListAdamW(masters, **kw)


def grads(k, dtype=torch.bfloat16):
    return [None if i == 3 else (torch.randn(s, generator=gen(50 * k + i)) * 1e-2).to(dtype).cuda()
            for i, s in enumerate(SHAPES)]


def test_class_with_32_bits_is_the_flat_optimizer():
    o = optimizer(32, groups=None, group_of=None)
    numels = [p.numel() for p in o.masters]
    flat = pkg.FlatShardAdamW(numels, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, max_norm=0.5, device="cuda",
                              master=torch.cat([p.view(-1) for p in o.masters]))
    for k in range(3):
        r, rf = o.step(grads(k)), flat.step_tensors(grads(k))
        assert r == rf and r.clip_coef < 1.0
    assert o.t == 3
    at = 0
    for i, n in enumerate(numels):
        for a, b in ((o.masters[i], flat.master), (o.state_of(i)[0], flat.exp_avg), (o.state_of(i)[1], flat.exp_avg_sq),
                     (o.lowp[i], flat.lowp)):
            assert torch.equal(a.view(-1), b[at:at + n])
        at += n


@pytest.mark.parametrize("bits,seed", [(32, None), (8, None), (8, 12)])
def test_class_graph_matches_host_steps(bits, seed):
    host_o, dev_o = (optimizer(bits, rounding_seed=seed, capturable=c) for c in (False, True))
    stores = [None if g is None else torch.zeros_like(g) for g in grads(0, torch.float16)]
    dev_o.register_grads(stores)
    scaler = pkg.DeviceLossScale("cuda", init_scale=256.0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        dev_o.launch_step(loss_scale=scaler)
        scaler.launch_update(dev_o.norm_buf)
    scale = 256.0
    for k in range(5):
        for s, g in zip(stores, grads(k, torch.float32)):
            if s is not None:
                s.copy_(g * scale)
        if k == 1:
            stores[2].view(-1)[9] = math.nan
        if k == 3:
            for o in (host_o, dev_o):
                o.set_group(1, lr=1e-4)
        graph.replay()
        r = host_o.step(stores, scale=1.0 / scale)
        assert r.finite == (k != 1)
        scale = scaler.scale
        for a, b in zip(host_o.masters + host_o.lowp, dev_o.masters + dev_o.lowp):
            assert torch.equal(a, b)
    assert host_o.t == dev_o.t == 4


@pytest.mark.parametrize("bits", [8, 32])
def test_class_checkpoints_in_either_width(bits):
    a = optimizer(bits)
    for k in range(2):
        a.step(grads(k))
    sd = a.state_dict()
    b = optimizer(bits)
    b.load_state_dict(sd)
    for x, y in ((a, b),):
        x.step(grads(5))
        y.step(grads(5))
        assert x.t == y.t == 3 and all(torch.equal(p, q) for p, q in zip(x.masters + x.lowp, y.masters + y.lowp))
    other = optimizer(40 - bits)
    other.load_state_dict(sd)
    wide, narrow = (other, sd) if bits == 8 else (b, None)
    if narrow is not None:
        for i in range(len(SHAPES)):
            q = zs.State8(*(x.cuda() for x in sd["state8"]))
            o, n = a.offsets[i], a.numels[i]
            codes = host(q)
            np.testing.assert_array_equal(f64(wide.state_of(i)[0]), R.values(codes[0], codes[1])[o:o + n])
    other.step(grads(5))
    moved = torch.cat([(p - q.cuda()).view(-1) for p, q in zip(a.masters, sd["masters"])]).norm()
    off = torch.cat([(p - q).view(-1) for p, q in zip(a.masters, other.masters)]).norm()
    # one conversion to 8 bits is at most 1/16 off in each moment
    assert off <= 0.125 * moved
    with pytest.raises(ValueError):
        pkg.TensorListAdamW([torch.zeros(3, device="cuda")]).load_state_dict(sd)
    assert optimizer(8).resident_bytes() < optimizer(32).resident_bytes()


def test_class_shared_norm_and_refusals():
    o = optimizer(8)
    with pytest.raises(ValueError, match="registered"):
        o.launch_step()
    with pytest.raises(ValueError, match="one grad"):
        o.step(grads(0)[:-1])
    with pytest.raises(ValueError, match="elements"):
        o.step([torch.zeros(4, device="cuda")] * len(SHAPES))
    with pytest.raises(ValueError, match="dtype"):
        o.step([torch.zeros(s, dtype=torch.float32 if i else torch.float16, device="cuda") for i, s in enumerate(SHAPES)])
    with pytest.raises(ValueError, match="takes"):
        o.set_group(0, momentum=1)
    with pytest.raises(zs.ZeroError):
        bad = optimizer(8, lr=-1.0)
        bad.step(grads(0))
    with pytest.raises(ValueError, match="differ in length"):
        optimizer(8, group_of=[0])
    with pytest.raises(zs.ZeroError, match="group"):
        optimizer(8, group_of=[0, 1, 2, 0, 0, 0])
    with pytest.raises(ValueError, match="bf16 or all f16"):
        optimizer(8, lowp=[torch.zeros(s, device="cuda") for s in SHAPES])
    with pytest.raises(ValueError, match="contiguous"):
        pkg.TensorListAdamW([torch.zeros(4, 4, device="cuda").t()])
    clip = norm_result_tensor("cuda", coef=0.5)
    a, b = optimizer(8), optimizer(8, max_norm=math.inf)
    a.launch_step(grads(0), norm_result=clip)
    assert a.finish_step(norm_result=clip).finite and a.t == 1
    b.step([None if g is None else g * 0.5 for g in grads(0)])
    assert same(a.state8, b.state8) and all(torch.equal(p, q) for p, q in zip(a.masters, b.masters))

"""The 8-bit moments on the GPU: conversions and the flat-shard step against the 64-bit formulas (_ref8.py), and
FlatShardAdamW / ZeroDataPlane with state_bits=8 on every path of theirs."""
import math

import numpy as np
import pytest
import torch

import _ref8 as R
import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from _helpers import norm_result_tensor, offset_view
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HP = dict(lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
SIZES = [1, 2, 255, 256, 257, 511, 2047, 2048, 2049, 4097, 70001]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes_view(n, offset=0):
    return offset_view(n, torch.uint8, offset, "cuda").view(torch.float8_e4m3fn)


def random_state8(n, g, offset=0):
    """Any codes but NaN, scales over many octaves, one block of zeros."""
    nb = zs.state8_blocks(n)
    m = torch.randint(0, 254, (n,), generator=g)
    m = torch.where(m >= 127, m + 1, m).to(torch.uint8)
    r = torch.randint(0, 127, (n,), generator=g).to(torch.uint8)
    s = [torch.exp2(torch.randint(-30, -8, (nb,), generator=g).float()) for _ in range(2)]
    b = int(torch.randint(0, nb, (1,), generator=g))
    m[256 * b:256 * b + 256] = 0
    r[256 * b:256 * b + 256] = 0
    s[1][b] = 0.0
    out = zs.State8(codes_view(n, offset), s[0].cuda(), codes_view(n, offset), s[1].cuda())
    out.exp_avg.view(torch.uint8).copy_(m)
    out.root.view(torch.uint8).copy_(r)
    return out


def host(state):
    return [t.cpu().view(torch.uint8).numpy().copy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy().copy()
            for t in state]


def clone(state):
    return zs.State8(*(t.clone() for t in state))


def same(a, b):
    return all(np.array_equal(x.view(np.uint8), y.view(np.uint8)) for x, y in zip(host(a), host(b)))


def f64(t):
    return t.detach().double().cpu().numpy()


def check_step(p0, old, g, g_err, p1, lowp, new, *, hp=HP, t=3, seed=None, stream=0):
    """Master, copy and 8-bit state of one step against the formulas."""
    m0, r0 = R.values(old[0], old[1]), R.values(old[2], old[3])
    out = R.step(p0, m0, r0 * r0, g, g_err, t=t, root=2, div=3, **hp)
    R.check_close(f64(p1), *out["p"], "master")
    km = kr = None
    if seed is not None:
        km, kr = R.draws(seed, t, stream, len(p0))
    h = host(new)
    R.check_codes(h[0], h[1], *out["m"], k=km, name="exp_avg")
    R.check_codes(h[2], h[3], *out["r"], k=kr, floor=True, name="root")
    if lowp is not None:
        assert torch.equal(lowp, p1.to(lowp.dtype)), "the copy is the master rounded"


# ------------------------------------------------------------- conversions
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("n", SIZES)
def test_pack_and_unpack(n, offset):
    g = gen(n)
    mag = torch.exp2(torch.rand(n, generator=g) * 40 - 30)
    m = torch.randn(n, generator=g) * mag
    v = torch.rand(n, generator=g) * mag * mag
    m[::7], v[::7] = 0.0, 0.0
    dm, dv = (offset_view(n, torch.float32, offset, "cuda", x) for x in (m, v))
    q = zs.State8(codes_view(n, offset), torch.full((zs.state8_blocks(n),), -1.0, device="cuda"), codes_view(n, offset),
                  torch.full((zs.state8_blocks(n),), -1.0, device="cuda"))
    pkg.zero_state8_pack(dm, dv, q)
    h = host(q)
    R.check_codes(h[0], h[1], f64(m), np.zeros(n), name="exp_avg")
    root = np.sqrt(f64(v))
    R.check_codes(h[2], h[3], root, R.EPS * root, floor=True, name="root")
    am, av = (offset_view(n, torch.float32, offset, "cuda") for _ in range(2))
    pkg.zero_state8_unpack(q, am, av)
    np.testing.assert_array_equal(f64(am), R.values(h[0], h[1]))
    r = R.values(h[2], h[3])
    np.testing.assert_array_equal(f64(av), (r * r).astype(np.float32).astype(np.float64))
    # packing what was unpacked gives the same values
    q2 = pkg.new_state8(n, "cuda")
    pkg.zero_state8_pack(am, av, q2)
    h2 = host(q2)
    np.testing.assert_array_equal(R.values(h2[0], h2[1]), R.values(h[0], h[1]))


def test_every_value_packs_to_itself():
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    x = torch.from_numpy(R.TABLE[codes.numpy()]).float()
    m = torch.cat([x, torch.zeros(256 - len(x))])
    v = m.abs() ** 2
    q = pkg.new_state8(256, "cuda")
    pkg.zero_state8_pack(m.cuda(), v.cuda(), q)
    a, b = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    pkg.zero_state8_unpack(q, a, b)
    assert torch.equal(a.cpu(), m) and torch.equal(b.cpu(), v)
    assert float(q.exp_avg_scale) == 1.0


def test_a_block_that_is_not_finite_reads_nan_and_the_others_do_not():
    n = 6 * 256
    m, v = torch.ones(n), torch.ones(n)
    m[5], m[256], v[512 + 3], v[768], m[1024] = math.inf, math.nan, -1.0, math.inf, 2.0 ** 126
    q = pkg.new_state8(n, "cuda")
    pkg.zero_state8_pack(m.cuda(), v.cuda(), q)
    a, b = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    pkg.zero_state8_unpack(q, a, b)
    nan_m, nan_v = a.cpu().isnan().view(6, 256), b.cpu().isnan().view(6, 256)
    for blk, (bad_m, bad_v) in enumerate([(1, 0), (1, 0), (0, 1), (0, 1), (1, 0), (0, 0)]):
        assert nan_m[blk].all() if bad_m else not nan_m[blk].any()
        assert nan_v[blk].all() if bad_v else not nan_v[blk].any()
    assert (a.cpu()[2 * 256:4 * 256] == 1).all() and (b.cpu()[:512] == 1).all()


def test_a_root_never_becomes_zero():
    v = torch.full((256,), 1e-20)
    v[0], v[1] = 1.0, 0.0
    q = pkg.new_state8(256, "cuda")
    pkg.zero_state8_pack(torch.zeros(256, device="cuda"), v.cuda(), q)
    c = q.root.view(torch.uint8).cpu()
    assert c[1] == 0 and (c[2:] == 1).all() and float(q.exp_avg_scale[0]) == 2.0 ** -126


# ---------------------------------------------------------- flat-shard step
@pytest.mark.parametrize("seed", [None, 0x123456789ABCDEF1])
@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("gdt,lowp,acc,offset,goff", [
    ("bf16", "bf16", False, 0, 0), ("f16", "f16", True, 0, 1), ("f32", None, True, 0, 0), ("f32", "bf16", False, 1, 0),
    ("bf16", "f16", True, 3, 5),
])
def test_shard_step(n, gdt, lowp, acc, offset, goff, seed):
    g = gen(n + offset)
    q = random_state8(n, g, offset)
    p = offset_view(n, torch.float32, offset, "cuda", torch.randn(n, generator=g))
    x = offset_view(n, DT[gdt], goff, "cuda", (torch.randn(n, generator=g) * 1e-2).to(DT[gdt]))
    a = offset_view(n, torch.float32, offset, "cuda", torch.randn(n, generator=g) * 1e-2) if acc else None
    c = offset_view(n, DT[lowp], offset, "cuda") if lowp else None
    table, total = zs.zero_tensor_table([x])
    clip = norm_result_tensor("cuda", coef=0.625)
    p0, old = f64(p), host(q)
    pkg.zero_adamw_step8_tensors(p, q, zs.device_table(table, 1, "cuda"), 1, total, x.dtype, 0, 0.3, c, HP["lr"], HP["b1"],
                                 HP["b2"], HP["eps"], HP["wd"], 3, clip, acc=a, rounding_seed=seed)
    gr, err = R.grad(f64(x), float(np.float32(0.3)), None if a is None else f64(a), 0.625)
    check_step(p0, old, gr, err, p, c, q, seed=seed)


@pytest.mark.parametrize("seed", [None, 77])
@pytest.mark.parametrize("gdt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("align", [1, 128])
def test_shard_step_through_a_ragged_table(gdt, align, seed):
    rng = np.random.default_rng(5)
    sizes = [int(x) for x in np.exp(rng.uniform(0, 9, 120))] + [9000, 1, 0, 20000, 3]
    total = sum(sizes)
    g = gen(1)
    at = np.cumsum([0] + [-(-k // align) * align for k in sizes])
    store = (torch.randn(int(at[-1]) + 8, generator=g) * 1e-2).to(DT[gdt]).cuda()
    grads = [None if i % 11 == 4 else store[a:a + k] for i, (a, k) in enumerate(zip(at, sizes))]
    flat = np.concatenate([np.zeros(k) if x is None else f64(x) for x, k in zip(grads, sizes)])
    table = zs.device_table(zs.zero_tensor_table(grads, sizes)[0], len(sizes), "cuda")
    for lo, hi in ((0, total), (1003, total - 77), (total - 300, total), (5, 6)):
        n = hi - lo
        q, p = random_state8(n, g), torch.randn(n, generator=g).cuda()
        c = torch.empty(n, dtype=torch.bfloat16, device="cuda")
        p0, old = f64(p), host(q)
        pkg.zero_adamw_step8_tensors(p, q, table, len(sizes), total, DT[gdt], lo, 1.0, c, HP["lr"], HP["b1"], HP["b2"],
                                     HP["eps"], HP["wd"], 3, rounding_seed=seed)
        gr, err = R.grad(flat[lo:hi])
        check_step(p0, old, gr, err, p, c, q, seed=seed, stream=lo)


def test_many_tensors_table():
    sizes = [3] * 5000 + [4000]
    total, g = sum(sizes), gen(2)
    store = (torch.randn(total, generator=g)).cuda()
    at = np.cumsum([0] + sizes)
    table = zs.device_table(zs.zero_tensor_table([store[a:a + k] for a, k in zip(at, sizes)])[0], len(sizes), "cuda")
    q, p = random_state8(total, g), torch.randn(total, generator=g).cuda()
    p0, old = f64(p), host(q)
    pkg.zero_adamw_step8_tensors(p, q, table, len(sizes), total, torch.float32, 0, 1.0, None, HP["lr"], HP["b1"], HP["b2"],
                                 HP["eps"], HP["wd"], 3)
    check_step(p0, old, *R.grad(f64(store)), p, None, q)


def shard_call(p, q, x, *, clip=None, seed=None, step=3, stream=None, **kw):
    table = zs.device_table(zs.zero_tensor_table([x])[0], 1, "cuda")
    pkg.zero_adamw_step8_tensors(p, q, table, 1, x.numel(), x.dtype, 0, 1.0, kw.pop("lowp", None), HP["lr"], HP["b1"],
                                 HP["b2"], HP["eps"], HP["wd"], step, clip, stream, rounding_seed=seed, **kw)


def test_a_skipped_step_changes_nothing():
    n, g = 3000, gen(3)
    q, p = random_state8(n, g), torch.randn(n, generator=g).cuda()
    c = torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda")
    q0, p0 = clone(q), p.clone()
    shard_call(p, q, torch.full((n,), math.nan, device="cuda"), clip=norm_result_tensor("cuda", finite=False), lowp=c)
    assert same(q, q0) and torch.equal(p, p0) and (c == 7).all()


def test_non_finite_grads_without_a_norm_stay_in_their_block():
    n, g = 2000, gen(4)
    q, p, x = random_state8(n, g), torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()
    x[300], x[1999] = math.nan, math.inf
    q2, p2, y = clone(q), p.clone(), x.clone()
    y[300], y[1999] = 0.0, 0.0
    shard_call(p, q, x)
    shard_call(p2, q2, y)
    fine = torch.ones(n, dtype=torch.bool)
    for a, b in ((256, 512), (1792, 2000)):
        fine[a:b] = False
        assert math.isnan(float(q.exp_avg_scale[a // 256])) and math.isnan(float(q.root_scale[a // 256]))
    for a, b in zip(q[::2], q2[::2]):
        assert torch.equal(a.view(torch.uint8).cpu()[fine], b.view(torch.uint8).cpu()[fine])
    keep = torch.arange(n) != 300
    keep[1999] = False
    assert torch.equal(p.cpu()[keep], p2.cpu()[keep]) and p[300].isnan() and p[1999].isnan()


def test_fresh_state_first_step_is_sign_descent():
    n = 1000
    q, p = pkg.new_state8(n, "cuda"), torch.zeros(n, device="cuda")
    x = torch.linspace(-1, 1, n, device="cuda") * 1e-3
    shard_call(p, q, x, step=1)
    # p = -lr g / (|g| + eps): the moments enter before they are rounded to 8 bits; a dozen roundings, root and reciprocal
    want = -HP["lr"] * f64(x) / (np.abs(f64(x)) + HP["eps"])
    np.testing.assert_allclose(f64(p), want, rtol=32 * R.EPS)


def test_zero_grads_keep_zero_moments():
    n = 777
    q, p = pkg.new_state8(n, "cuda"), torch.ones(n, device="cuda")
    shard_call(p, q, torch.zeros(n, device="cuda"), seed=9)
    assert (q.exp_avg.view(torch.uint8) == 0).all() and (q.root.view(torch.uint8) == 0).all()
    np.testing.assert_allclose(f64(p), 1 - HP["lr"] * HP["wd"], rtol=2 * R.EPS)


def test_stochastic_rounding_keeps_the_mean_where_nearest_stalls():
    # exp_avg_sq decays by 0.95 a step towards a small constant while one element holds the block's scale:
    # each step of the root (2.5 %) is under half a spacing of most codes, so nearest stays where it is
    n, steps = 256 * 64, 40
    x = torch.full((n,), 0.03, device="cuda")
    x[::256] = 1.0
    start = torch.full((n,), 0.2 ** 2)
    start[::256] = 1.0
    want = math.sqrt(0.95 ** steps * 0.04 + (1 - 0.95 ** steps) * 0.03 ** 2)
    means = {}
    for seed in (None, 4):
        q, p = pkg.new_state8(n, "cuda"), torch.zeros(n, device="cuda")
        pkg.zero_state8_pack(torch.zeros(n, device="cuda"), start.cuda(), q)
        for t in range(1, steps + 1):
            shard_call(p, q, x, seed=seed, step=t)
        h = host(q)
        r = R.values(h[2], h[3]).reshape(-1, 256)[:, 1:]
        means[seed] = r.mean()
    assert means[None] > 1.5 * want
    # truncation to 1/128 of a spacing takes up to 2 % off the mean, the noise's square (u^2 / 6 a step) adds up to 3 %
    # to the root, its spread takes 2 % off: 15 % holds all of them
    assert abs(means[4] - want) < 0.15 * want


def test_rounding_draws_depend_on_seed_step_and_shard_only():
    n, g = 5000, gen(6)
    q, p, x = random_state8(n, g), torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda() * 1e-2
    runs = []
    for seed, step in ((1, 3), (1, 3), (2, 3), (1 << 40 | 1, 3), (1, 4)):
        a, b = clone(q), p.clone()
        shard_call(b, a, x, seed=seed, step=step)
        runs.append(a)
    assert same(runs[0], runs[1])
    for other in runs[2:]:
        assert not same(runs[0], other)


def test_other_stream():
    n, g = 1 << 20, gen(7)
    q, p, x = random_state8(n, g), torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()
    q2, p2 = clone(q), p.clone()
    shard_call(p2, q2, x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for form in (st, st.cuda_stream):
        a, b = clone(q), p.clone()
        st.wait_stream(torch.cuda.current_stream())
        shard_call(b, a, x, stream=form)
        st.synchronize()
        assert same(a, q2) and torch.equal(b, p2)


def test_binding_refusals():
    n = 300
    q, p, x = pkg.new_state8(n, "cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    with pytest.raises(ValueError, match="expected 300"):
        shard_call(p, pkg.new_state8(n + 1, "cuda"), x)
    with pytest.raises(ValueError, match="contiguous"):
        shard_call(p, q._replace(exp_avg=torch.zeros(2 * n, dtype=torch.uint8, device="cuda").view(
            torch.float8_e4m3fn)[::2]), x)
    with pytest.raises(ValueError, match="float8"):
        shard_call(p, q._replace(root=torch.zeros(n, dtype=torch.uint8, device="cuda")), x)
    with pytest.raises(ValueError, match="CUDA"):
        shard_call(p, pkg.new_state8(n, "cpu"), x)
    with pytest.raises(ValueError, match="acc"):
        shard_call(p, q, x, acc=torch.zeros(n + 1, device="cuda"))
    with pytest.raises(ValueError, match="param_lowp"):
        shard_call(p, q, x, lowp=torch.zeros(n, device="cuda"))
    with pytest.raises(zs.ZeroError):
        shard_call(p, q, x, step=0)


# ------------------------------------------------------------ FlatShardAdamW
def shard_opt(sizes, **kw):
    total = sum(sizes)
    kw = {**dict(lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, max_norm=0.5, state_bits=8), **kw}
    s, e = zs.zero_shard_range(total, kw.get("world_size", 1), kw.get("rank", 0))
    return pkg.FlatShardAdamW(sizes, device="cuda", master=torch.randn(e - s, generator=gen(8)).cuda(), **kw)


def grads_of(sizes, k, dtype=torch.bfloat16):
    return [(torch.randn(n, generator=gen(100 * k + i)) * 1e-2).to(dtype).cuda() for i, n in enumerate(sizes)]


SHAPES = [5000, 1, 2049, 700, 12345]


@pytest.mark.parametrize("seed", [None, 5])
@pytest.mark.parametrize("world,rank,full", [(1, 0, False), (3, 1, False), (3, 2, True)])
def test_every_path_of_the_flat_shard_gives_the_same_bits(world, rank, full, seed):
    kw = dict(world_size=world, rank=rank, rounding_seed=seed, grad_range="full" if full else "shard")
    a, b, c, d = (shard_opt(SHAPES, capturable=i == 2, **kw) for i in range(4))
    for k in range(3):
        micro = [grads_of(SHAPES, 10 * k + j) for j in range(2)]
        for o in (a, b, c, d):
            o.flatten(micro[0], accumulate=False, scale=0.5)
        a.flatten(micro[1], accumulate=True, scale=0.5, fuse_norm=True)
        ra = a.step()
        rb = b.step_tensors(micro[1], scale=0.5, accumulated=True)
        rc = c.step_tensors(micro[1], scale=0.5, accumulated=True)
        flat = torch.cat(micro[1])[d.glo:d.ghi].contiguous()
        rd = d.step_flat(flat, scale=0.5, accumulated=True)
        assert ra.finite and ra == rb == rc == rd
    for o in (b, c, d):
        assert o.t == a.t == 3
        assert same(a.state8, o.state8) and torch.equal(a.master, o.master) and torch.equal(a.lowp, o.lowp)


def test_flat_shard_tracks_the_32_bit_optimizer():
    a, b = shard_opt(SHAPES, rounding_seed=1, max_norm=math.inf), shard_opt(SHAPES, state_bits=32, max_norm=math.inf)
    p0 = a.master.clone()
    for k in range(10):
        for o in (a, b):
            o.step_tensors(grads_of(SHAPES, k))
    moved = (b.master - p0).norm()
    # a spacing is at most 1/8 of its moment; the noise of both moments over ten steps stays under 1/8 of the update each
    assert (a.master - b.master).norm() < 0.25 * moved


def test_skip_loss_scale_and_graph():
    sizes = SHAPES
    seed = 11
    storage = torch.zeros(sum(sizes), dtype=torch.float16, device="cuda")
    views = list(torch.split(storage, sizes))
    host_opt, dev_opt = shard_opt(sizes, rounding_seed=seed), shard_opt(sizes, rounding_seed=seed, capturable=True)
    scaler = pkg.DeviceLossScale("cuda", init_scale=1024.0, growth_interval=2)
    dev_opt.register_grads(views)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dev_opt.launch_step_tensors(loss_scale=scaler)
        scaler.launch_update(dev_opt.norm_buf)
    scale = 1024.0
    for k in range(5):
        g = torch.cat(grads_of(sizes, k, torch.float32)) * scale
        if k == 2:
            g[17] = math.inf
        storage.copy_(g.half())
        before = clone(dev_opt.state8)
        graph.replay()
        torch.cuda.synchronize()
        r = host_opt.step_tensors(views, scale=1.0 / scale)
        assert r.finite == (k != 2)
        if k == 2:
            assert same(before, dev_opt.state8)
        scale = scaler.scale
        assert same(host_opt.state8, dev_opt.state8) and torch.equal(host_opt.master, dev_opt.master)
    assert host_opt.t == dev_opt.t == 4


def test_checkpoints_in_either_width():
    sizes = SHAPES
    a = shard_opt(sizes, rounding_seed=2)
    for k in range(3):
        a.step_tensors(grads_of(sizes, k))
    sd = a.state_dict()
    b = shard_opt(sizes, rounding_seed=2)
    b.load_state_dict(sd)
    assert same(a.state8, b.state8) and b.t == 3
    wide = shard_opt(sizes, state_bits=32)
    wide.load_state_dict(sd)
    h = host(a.state8)
    np.testing.assert_array_equal(f64(wide.exp_avg), R.values(h[0], h[1]))
    back = shard_opt(sizes)
    back.load_state_dict(wide.state_dict())
    np.testing.assert_array_equal(R.values(*host(back.state8)[:2]), R.values(*h[:2]))
    assert a.resident_bytes() < wide.resident_bytes() - 5 * a.n
    with pytest.raises(ValueError):
        shard_opt([5]).load_state_dict(sd)


def test_empty_shard_and_missing_grad_buffer():
    o = shard_opt([3], world_size=8, rank=7)
    assert o.n == 0 and o.step_tensors(grads_of([3], 0)).norm == 0.0
    o = shard_opt(SHAPES, grad_buffer=False)
    o.step_tensors(grads_of(SHAPES, 0))
    with pytest.raises(ValueError, match="grad buffer"):
        o.launch_step(norm_result=o.norm_buf)


def test_data_plane_and_units_with_8_bit_states():
    sizes = SHAPES
    kw = dict(device="cuda:0", lr=1e-2, betas=(0.9, 0.95), max_norm=0.5, state_bits=8)
    dp = pkg.ZeroDataPlane(sizes, master=torch.randn(sum(sizes), generator=gen(8)).cuda(), weight_decay=0.1, **kw)
    ref = shard_opt(sizes)
    units = pkg.ZeroUnits([sizes[:2], sizes[2:]], masters=[m.clone() for m in torch.split(
        ref.master, [sum(sizes[:2]), sum(sizes[2:])])], weight_decay=0.1, **kw)
    for k in range(2):
        g = grads_of(sizes, k)
        for v, x in zip(dp.grad_views(), g):
            v.copy_(x)
        for v, x in zip([v for u in units.units for v in u.grad_views()], g):
            v.copy_(x)
        dp.reduce_scatter_grads()
        units.reduce_scatter_grads()
        r = dp.step()
        ru = units.step()
        ref.step_tensors(g)
        assert r.finite and abs(r.norm - ru.norm) <= 1e-12 * r.norm
    assert same(dp.opt.state8, ref.state8) and torch.equal(dp.opt.master, ref.master)
    assert torch.equal(dp.flat_param[:sum(sizes)], ref.lowp)
    # a unit's first block starts at its own first element: equal where both partitions' blocks agree
    assert torch.equal(units.units[0].opt.master[:4864], ref.master[:4864])


def test_units_that_share_a_seed_draw_differently():
    n = 5000
    units = pkg.ZeroUnits([[n], [n]], device="cuda:0", lr=1e-2, state_bits=8, rounding_seed=1)
    g = (torch.randn(n, generator=gen(1)) * 1e-2).bfloat16().cuda()
    for u in units.units:
        u.flat_grad.copy_(g)
    units.reduce_scatter_grads()
    units.step()
    a, b = (u.opt.state8 for u in units.units)
    assert torch.equal(a.exp_avg_scale, b.exp_avg_scale) and not same(a, b)
    one = pkg.FlatShardAdamW([n], lr=1e-2, state_bits=8, rounding_seed=1, device="cuda")
    one.step_tensors([g])
    assert same(one.state8, a)


@pytest.mark.parametrize("power", [-12, -50, -60])
def test_moments_of_any_size(power):
    # grads scaled by a power of two move moments and scales by it: the same codes, as long as nothing underflows
    n, s = 3000, 2.0 ** power
    g = gen(20)
    x = torch.randn(n, generator=g).cuda()
    runs = []
    for k in (1.0, s):
        q, p = pkg.new_state8(n, "cuda"), torch.zeros(n, device="cuda")
        for t in (1, 2):
            shard_call(p, q, x * k, seed=3, step=t)
        runs.append(q)
    a, b = runs
    if power > -54:
        assert torch.equal(a.exp_avg.view(torch.uint8), b.exp_avg.view(torch.uint8))
        assert torch.equal(a.root.view(torch.uint8), b.root.view(torch.uint8))
        assert torch.equal(a.exp_avg_scale * s, b.exp_avg_scale) and torch.equal(a.root_scale * s, b.root_scale)
    else:  # exp_avg_sq around 2^-120: still finite, still above zero wherever the grads are
        assert ((b.root.view(torch.uint8) > 0) == (a.root.view(torch.uint8) > 0)).all() and b.root_scale.isfinite().all()


@pytest.mark.slow
def test_indices_past_2_to_31():
    n = (1 << 31) + 5003
    q, p = pkg.new_state8(n, "cuda"), torch.zeros(n, device="cuda")
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = slice(n - 7000 - (n - 7000) % 256, n)
    m = tail.stop - tail.start
    g = gen(9)
    x[tail] = (torch.randn(m, generator=g) * 1e-2).bfloat16().cuda()
    p[tail] = torch.randn(m, generator=g).cuda()
    old = random_state8(m, g)
    sb = slice(tail.start // 256, None)
    for dst, src, at in zip(q, old, (tail, sb, tail, sb)):
        (dst[at].view(torch.uint8) if dst.dtype == torch.float8_e4m3fn else dst[at]).copy_(
            src.view(torch.uint8) if src.dtype == torch.float8_e4m3fn else src)
    p0, oldh = f64(p[tail]), host(old)
    shard_call(p, q, x, seed=21)
    assert float(p[:tail.start].abs().max()) == 0.0
    new = zs.State8(q.exp_avg[tail], q.exp_avg_scale[sb], q.root[tail], q.root_scale[sb])
    gr, err = R.grad(f64(x[tail]))
    out = R.step(p0, R.values(oldh[0], oldh[1]), R.values(oldh[2], oldh[3]) ** 2, gr, err, t=3, root=2, div=3, **HP)
    R.check_close(f64(p[tail]), *out["p"], "master")
    km, kr = R.draws(21, 3, 0, m, first=tail.start)
    h = host(new)
    R.check_codes(h[0], h[1], *out["m"], k=km)
    R.check_codes(h[2], h[3], *out["r"], k=kr, floor=True)

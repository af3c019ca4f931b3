"""The norms of many tensors and their clipping against the formulas in 64 bits.

Tolerances.  Sums: a thread adds at most 131072 / 128 / 2 = 512 pairs, the j-th with a tail l of at most j x 2^-24 of the
sum, whose addition is rounded by 2^-24 of it: 512^2 / 2 x 2^-48 = 4.66e-10 at worst, the rest of the tree a few 2^-48
more, and squares of tiny values up to 2^-37: SUM = 5e-10 (half of that for a root).  Binary32 outputs add 2^-24.  A clipped grad: the coefficient, scale x coefficient and the
product are each rounded to binary32, 3 x 2^-24 (and their cross terms), then eps / 2 of a 16-bit type; where the value is
subnormal there, half its type's least step."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
SUM, ULP = 5e-10, 2.0 ** -24
LEAST = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}
SIZES = [1, 0, 7, 8, 9, 255, 4095, 4096, 4097, 3, 70001, 0, 33, 65536, 8200]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def view(x, offset):
    """x on the GPU, its first element `offset` elements past a 256-byte border, guarded on both sides."""
    buf = torch.full((offset + x.numel() + 16,), 77.0, dtype=x.dtype, device="cuda")
    v = buf[offset:offset + x.numel()]
    v.copy_(x.flatten())
    return v


def tensors(dtype, offset=0, sizes=SIZES, seed=0, std=1e-2, absent=()):
    out = []
    for i, n in enumerate(sizes):
        dt = TYPES[i % 3] if dtype == "mixed" else dtype
        x = (torch.randn(n, generator=gen(seed * 1000 + i)) * std * 2.0 ** (i % 5)).to(dt)
        out.append(None if i in absent else view(x, (offset + i) % 16 if offset else 0))
    return out


def wide(t):
    return torch.zeros(0, dtype=torch.float64) if t is None else t.detach().double().cpu().flatten()


def sums_of(xs, p, scale=1.0):
    out = []
    for x in xs:
        v = (wide(x) * scale).abs()
        out.append(float(v.max() if v.numel() and p == math.inf else v.pow(p).sum() if p != math.inf else 0.0))
    return np.array(out)


def joined(sums, p):
    return float(np.max(sums, initial=0.0)) if p == math.inf else float(np.sum(sums))


def rooted(s, p):
    return np.sqrt(s) if p == 2 else s


def coefs_of(sums, of, limits, p):
    norms = [rooted(joined(sums[np.asarray(of) == g], p), p) for g in range(len(limits))]
    return norms, [min(1.0, m / (n + 1e-6)) for m, n in zip(limits, norms)]


def near(got, want, rel, least=0.0):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want)), (got, want)
    ok = np.isfinite(want)
    off = np.abs(got[ok] - want[ok]) - rel * np.abs(want[ok])
    assert off.size == 0 or off.max() <= least, off.max()


def check_clipped(y, x, factor, dtype):
    """y against factor x in 64 bits."""
    rel = 3.01 * ULP + SUM + (torch.finfo(dtype).eps / 2 if dtype != F32 else 0.0)
    near(wide(y).numpy(), wide(x).numpy() * factor, rel * 1.01, LEAST[dtype] * 1.01 + LEAST[F32] * abs(factor))


def guards_intact(v):
    base = v._base
    lo = (v.data_ptr() - base.data_ptr()) // v.element_size()
    rest = torch.cat([base[:lo], base[lo + v.numel():]])
    return bool((rest == 77.0).all())


# ------------------------------------------------------------------ norms
@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("offset", [0, 1, 5])
@pytest.mark.parametrize("dtype", [*TYPES, "mixed"])
def test_norms_of_tensors_groups_and_all(dtype, offset, p):
    xs = tensors(dtype, offset, absent=(5, 12))
    of = [i % 3 for i in range(len(xs))]
    c = pkg.GradClip(SIZES, norm_type=p, group_of=of, max_norm=[0.5, math.inf, 0.1, 7.0])  # group 3 is empty
    before = [None if x is None else x.clone() for x in xs]
    c.launch_norms(xs, scale=-0.75)
    r = c.finish()
    s = sums_of(xs, p, 0.75)
    near(c.tensor_sums.cpu(), s, SUM)
    near(c.tensor_norms.cpu(), rooted(s, p), SUM + ULP)
    norms, coefs = coefs_of(s, of, [0.5, math.inf, 0.1, 7.0], p)
    near(r.group_norms, norms, SUM)
    near(c.group_norms.cpu(), norms, SUM + ULP)
    near(r.coefs, coefs, SUM + ULP)
    assert r.norm == pytest.approx(rooted(joined(s, p), p), rel=SUM) and r.finite
    assert float(c.norm) == pytest.approx(r.norm, rel=ULP)
    assert r.whole.clip_coef == 1.0 and r.coefs[1] == 1.0 and r.group_norms[3] == 0.0 and r.coefs[3] == 1.0
    for a, b in zip(xs, before):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("total", [(1 << 23) + 77, (1 << 25) + 1, (1 << 27) + 4099, (1 << 29) + 4099])  # the larger chunk sizes
def test_norms_of_long_tensors(dtype, total):
    sizes = [total - 1003, 0, 1000, 3]
    base = torch.empty(total + 1, dtype=dtype, device="cuda")
    g = torch.Generator("cuda").manual_seed(total)
    for a in range(0, total + 1, 1 << 26):
        base[a:a + (1 << 26)].normal_(0, 0.01, generator=g)
    xs = list(base[1:].split(sizes))
    for p in (2, 1, math.inf):
        c = pkg.GradClip(sizes, norm_type=p)
        c.launch_norms(xs)
        want = []
        for x in xs:
            parts = [0.0]
            for a in range(0, x.numel(), 1 << 26):
                v = x[a:a + (1 << 26)].double().abs_()
                parts.append(float(v.max() if p == math.inf else v.pow(p).sum()))
            want.append(max(parts) if p == math.inf else math.fsum(parts))
        near(c.tensor_sums.cpu(), want, SUM)
        assert c.finish().norm == pytest.approx(rooted(joined(np.array(want), p), p), rel=SUM)


def test_norms_do_not_depend_on_the_run():
    xs = tensors("mixed", 3)
    c, d = (pkg.GradClip(SIZES, group_of=[i % 4 for i in range(len(xs))]) for _ in range(2))
    c.launch_norms(xs)
    for _ in range(3):
        d.launch_norms(xs)
        assert torch.equal(c.results, d.results) and torch.equal(c.buffers.norms, d.buffers.norms)
        assert torch.equal(c.tensor_sums, d.tensor_sums)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [2, 1, math.inf])
def test_norms_of_extreme_values(dtype, p):
    top = torch.finfo(dtype).max
    rows = {
        "top": [top] * 5000 + [0.0] * 100,
        "top and small": [top, 1e-3, -1e-3] * 40,
        "subnormal": [2.0 ** -24 if dtype == F16 else 2.0 ** -133] * 700,
        "tiny": [2.0 ** -14 if dtype == F16 else 1e-30] * 9000,
        "tiny and one": [2.0 ** -14 if dtype == F16 else 1e-30] * 9000 + [1.0],
        "at the border": [2.0 ** -24 if dtype == F16 else 2.0 ** -54] * 4000 + [2.0 ** -24 if dtype == F16 else 2.0 ** -70] * 4000,
        "below it": [2.0 ** -24 if dtype == F16 else 2.0 ** -55] * 4000,
        "zero": [0.0, -0.0] * 3000,
        "inf": [1.0] * 20 + [-math.inf] + [1.0] * 5000,
        "nan": [1.0] * 5000 + [math.nan],
        "nan and inf": [math.inf] + [1.0] * 5000 + [math.nan],
        "nan first": [math.nan, 3.0],
        "ordinary": [0.5, -0.25] * 4000,
    }
    xs = [view(torch.tensor(v, dtype=torch.float64).to(dtype), 3) for v in rows.values()]
    c = pkg.GradClip([x.numel() for x in xs], norm_type=p, group_of=range(len(xs)))
    c.launch_norms(xs)
    want = rooted(sums_of(xs, p), p)
    for i, nm in enumerate(rows):
        if "nan" in nm:
            want[i] = math.nan
    r = c.finish()
    near(r.group_norms, want, SUM)
    with np.errstate(over="ignore"):
        near(c.tensor_norms.cpu(), want.astype(np.float32), SUM + 2 * ULP, 2.0 ** -149)
    assert math.isnan(r.norm) and not r.finite and int(c.found_nonfinite) == 1


def test_scale_that_is_not_finite():
    x = [torch.ones(100, device="cuda")]
    c = pkg.GradClip([100], max_norm=1.0)
    for bad in (math.inf, math.nan):
        with pytest.raises(zs.ZeroError):
            c.launch(x, scale=bad)
        ls = pkg.DeviceLossScale("cuda")
        ls.unscale.fill_(bad)
        c.launch(x, loss_scale=ls)
        assert not c.finish().finite and int(ls.found_inf) == 1 and bool((x[0] == 1).all())
    ls = pkg.DeviceLossScale("cuda")
    ls.unscale.fill_(0.0)
    assert c.clip_(x, loss_scale=ls).norm == 0.0 and bool((x[0] == 0).all())


# --------------------------------------------------------------- clipping
@pytest.mark.parametrize("offset", [0, 1, 6])
@pytest.mark.parametrize("dtype", [*TYPES, "mixed"])
def test_clip_in_place(dtype, offset):
    xs = tensors(dtype, offset, absent=(5,))
    of = [i % 3 for i in range(len(xs))]
    limits = [0.5, math.inf, 0.0]
    c = pkg.GradClip(SIZES, group_of=of, max_norm=limits)
    before = [None if x is None else x.clone() for x in xs]
    r = c.clip_(xs, scale=1.0)
    _, coefs = coefs_of(sums_of(before, 2), of, limits, 2)
    assert r.finite and r.coefs[0] < 1 and r.coefs[2] == 0.0
    for i, (x, b) in enumerate(zip(xs, before)):
        if x is None:
            continue
        if of[i] == 1:
            assert torch.equal(x, b)
        check_clipped(x, b, coefs[of[i]], x.dtype)
        assert guards_intact(x), i


@pytest.mark.parametrize("scale", [2.0 ** -16, 3.7, -0.3])
@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("to", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_clip_into_other_buffers(dtype, to, shift, scale):
    # the grad at one place of the vector grid, its copy at the same or another
    xs = tensors(dtype, 3, absent=(4, 11), std=100.0 if scale < 0.01 and dtype != F16 else 1.0)
    ys = [None if i == 6 else view(torch.full((n,), 5.0, dtype=to), (3 + i + shift) % 16) for i, n in enumerate(SIZES)]
    keep = [None if x is None else x.clone() for x in xs]
    s = sums_of(xs, 2, scale)
    limit = 0.5 * math.sqrt(s.sum())
    c = pkg.GradClip(SIZES, max_norm=limit)
    c.register_grads(xs, out=ys)
    c.launch(scale=scale)
    coef = limit / (math.sqrt(s.sum()) + 1e-6)
    for i, (x, y) in enumerate(zip(keep, ys)):
        if y is None:
            continue
        if x is None:
            assert bool((y == 0).all())
        else:
            assert torch.equal(x, xs[i])
            check_clipped(y, x, scale * coef, to)
        assert guards_intact(y), i


def test_below_the_limit_nothing_changes_but_copies_are_made():
    xs = tensors("mixed", 2)
    before = [x.clone() for x in xs]
    c = pkg.GradClip(SIZES, max_norm=1e6)
    assert c.clip_(xs).coefs[0] == 1.0
    ys = [torch.full_like(x, 9) for x in xs]
    c.launch(xs, out=ys)
    for x, b, y in zip(xs, before, ys):
        assert torch.equal(x, b) and torch.equal(y, b)


@pytest.mark.parametrize("p", [2, 1, math.inf])
def test_each_tensor_by_its_own_norm(p):
    sizes = [int(n) for n in np.random.default_rng(4).integers(0, 400, 3001)]
    xs = [(torch.randn(n, generator=gen(n)) * 2.0 ** (i % 9)).to(TYPES[i % 3]).cuda() for i, n in enumerate(sizes)]
    before = [x.clone() for x in xs]
    c = pkg.GradClip(sizes, max_norm=3.0, norm_type=p, group_of=range(len(sizes)))
    r = c.clip_(xs)
    s = sums_of(before, p)
    norms, coefs = coefs_of(s, range(len(sizes)), [3.0] * len(sizes), p)
    near(r.group_norms, norms, SUM)
    near(r.coefs, coefs, SUM + ULP)
    near(c.tensor_norms.cpu(), norms, SUM + ULP)
    assert r.norm == pytest.approx(rooted(joined(s, p), p), rel=SUM)
    for x, b, k in zip(xs, before, coefs):
        check_clipped(x, b, k, x.dtype)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nothing_is_written_where_a_norm_is_not_finite(bad):
    xs = tensors("mixed", 1)
    xs[10].view(-1)[69000] = bad
    before = [x.clone() for x in xs]
    of = [i % 2 for i in range(len(xs))]
    c = pkg.GradClip(SIZES, max_norm=[0.1, 0.1], group_of=of)
    r = c.clip_(xs)
    assert not r.finite and (math.isnan(r.norm) if math.isnan(bad) else r.norm == math.inf)
    assert int(c.found_nonfinite) == 1
    assert not math.isfinite(r.group_norms[0]) and math.isfinite(r.group_norms[1])
    near(c.tensor_norms.cpu()[8:10], rooted(sums_of(before, 2), 2)[8:10], SUM + ULP)
    ys = [torch.full_like(x, 9) for x in xs]
    c.launch(xs, out=ys)
    for x, b, y in zip(xs, before, ys):
        assert torch.equal(x.view(torch.uint8), b.view(torch.uint8)) and bool((y == 9).all())


def test_transposed_grads_and_copies():
    x = torch.randn(96, 70, generator=gen(1)).cuda().t()
    y = torch.zeros(96, 70, dtype=BF16, device="cuda").t()
    b = x.clone()
    c = pkg.GradClip([x.numel()], max_norm=1.0)
    c.launch([x], out=[y])
    coef = 1.0 / (float(b.double().norm()) + 1e-6)
    check_clipped(y.contiguous(), b.contiguous(), coef, BF16)
    c.launch([x])
    check_clipped(x.contiguous(), b.contiguous(), coef, F32)


def test_the_function_against_torchs():
    ps = [torch.zeros(n, device="cuda", requires_grad=True) for n in (300, 1, 5000)]
    for p in ps:
        p.grad = torch.randn(p.numel(), generator=gen(p.numel())).cuda()
    mine = [p.grad.clone() for p in ps]
    for kind in (2.0, 1.0, math.inf):
        want = torch.nn.utils.clip_grad_norm_(ps, 0.5, kind)
        got = pkg.clip_grad_norm_(mine, 0.5, kind)
        assert got.dim() == 0 and got.dtype == F32
        # torch's sums are binary32 sums of up to 5000 terms in blocks
        assert float(got) == pytest.approx(float(want), rel=1e-5)
        for a, p in zip(mine, ps):
            assert torch.allclose(a, p.grad, rtol=2e-5, atol=0)


@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("dtype,to", [(F32, None), (BF16, None), (F16, F32), (BF16, BF16)])
@pytest.mark.parametrize("total", [(1 << 21) - 9, (1 << 24) - 1, (1 << 25) + 77, (1 << 27) + 4099, (1 << 29) + 4099])
def test_clip_of_long_tensors(total, dtype, to, scale):
    sizes = [total - 71003, 0, 70000, 1000, 3]
    g = torch.Generator("cuda").manual_seed(total)
    base = torch.empty(total + 9, dtype=dtype, device="cuda").normal_(0, 1, generator=g)
    flat = base[5:5 + total]
    before = flat.clone()
    out = flat if to is None else torch.full((total + 9,), 7.0, dtype=to, device="cuda")[5:5 + total]
    c = pkg.GradClip(sizes, max_norm=0.5 * scale * math.sqrt(total), group_of=[0, 0, 1, 0, 0])
    c.launch(list(flat.split(sizes)), out=None if to is None else list(out.split(sizes)), scale=scale)
    coefs = c.finish().coefs
    # group 0 has total - 70000 normal values, whose root of squares is within 1 / sqrt(2 n) < 6e-4 of sqrt(n), times 16
    assert coefs[0] == pytest.approx(0.5 * math.sqrt(total / (total - 70000)), rel=1e-2) and coefs[1] == 1.0
    f = torch.full((total,), float(np.float32(scale) * coefs[0]), device="cuda")
    f[sizes[0]:sizes[0] + 70000] = float(np.float32(scale) * coefs[1])
    assert torch.equal(out, (before.float() * f).to(out.dtype))
    if to is not None:
        assert torch.equal(flat, before) and bool((out._base[:5] == 7).all()) and bool((out._base[5 + total:] == 7).all())


def test_an_element_beyond_32_bits():
    n = (1 << 31) + 70001
    x = torch.zeros(n + 3, dtype=BF16, device="cuda")[3:]
    x[0], x[-1], x[(1 << 31) + 5] = 3.0, 4.0, 12.0
    c = pkg.GradClip([n, 2], max_norm=6.5)
    tail = torch.zeros(2, device="cuda")
    r = c.clip_([x, tail])
    assert r.norm == 13.0 and float(c.tensor_norms[0]) == 13.0
    want = torch.tensor([3.0, 4.0, 12.0]) * r.coefs[0]
    assert [float(x[0]), float(x[-1]), float(x[(1 << 31) + 5])] == want.to(BF16).float().tolist()
    assert int(torch.count_nonzero(x)) == 3


def test_more_chunks_than_a_warp_adds():
    # tensors of 4101 chunks beside small ones: their partials are added by whole blocks
    sizes = [5, 4100 * 131072 + 9, 270000, 0, 1, 4101 * 131072]
    xs = [torch.full((n,), 0.5, dtype=BF16, device="cuda") for n in sizes]
    c = pkg.GradClip(sizes, max_norm=[1.0, 2.0], group_of=[0, 1, 0, 0, 1, 0])
    assert (c.plan.head.n_wide, c.plan.head.n_narrow) == (4101 + 3 + 4101, 2)
    r = c.clip_(xs)
    assert c.tensor_sums.tolist() == [n / 4 for n in sizes]
    for x, g in zip(xs, (0, 1, 0, 0, 1, 0)):
        assert bool((x == (torch.tensor(0.5) * r.coefs[g]).to(BF16).item()).all())


@pytest.mark.parametrize("n,groups,skewed", [(1023, 256, False), (1025, 257, False), (5200, 300, False), (9000, 1, False), (9000, 2, False), (20000, 20000, False),
                                             (1000, 900, True), (1024, 40, True), (1030, 1030, True), (6000, 500, True), (9000, 300, True), (700, 1500, False)])
def test_thousands_of_tensors(n, groups, skewed):
    """The counts at which the work is split another way; two long tensors among them where the list is long."""
    rng = np.random.default_rng(n)
    sizes = [int(k) for k in rng.integers(0, 60, n)]
    if 1024 < n < 9000:
        sizes[700], sizes[33] = 600 * 32768 + 5, 1100 * 32768 + 1  # more partials than 8 lanes add, than a warp adds
    total = sum(sizes)
    flat = torch.randint(-8, 9, (total,), generator=torch.Generator("cuda").manual_seed(n), device="cuda", dtype=torch.int32).to(BF16)
    xs = list(flat.split(sizes))
    of = rng.integers(0, groups, n)
    if skewed:  # one group has most tensors
        of = np.where(rng.random(n) < 0.9, groups // 3, of)
    of[0] = groups - 1
    limits = list(rng.uniform(1.0, 100.0, groups))
    # sums of squares of small whole numbers are exact
    ends = np.cumsum(sizes)
    run = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), flat.int().square().cumsum(0)]).cpu().numpy()
    s = (run[ends] - run[ends - sizes]).astype(np.float64)
    c = pkg.GradClip(sizes, max_norm=limits, group_of=of)
    before = flat.clone()
    r = c.clip_(xs)
    sums = np.zeros(groups)
    np.add.at(sums, of, s)
    assert np.array_equal(c.tensor_sums.cpu().numpy(), s)
    near(c.tensor_norms.cpu(), np.sqrt(s), 1.01 * ULP)
    near(r.group_norms, np.sqrt(sums), 2.0 ** -52)
    assert r.norm == pytest.approx(math.sqrt(s.sum()), rel=2.0 ** -52)
    coefs = np.minimum(1.0, np.array(limits) / (np.sqrt(sums) + 1e-6))
    near(r.coefs, coefs, 1.01 * ULP)
    f = torch.repeat_interleave(torch.tensor(coefs[of].astype(np.float32)).cuda(), torch.tensor(sizes).cuda())
    assert torch.equal(flat, (before.float() * f).to(BF16))
    # and as shards, joined by threads over all SMs
    shards = [zs.zero_shard_range(total, 3, k) for k in range(3)]
    flat.copy_(before)
    clips = [pkg.GradClip.of_shard(sizes, flat[a:b], a, max_norm=limits, group_of=of) for a, b in shards]
    for k in clips:
        k.launch_sums()
    gathered = torch.stack([k.tensor_sums for k in clips])
    for k in clips:
        k.launch(gathered_sums=gathered)
        assert np.array_equal(k.joined_sums.cpu().numpy(), s)
        assert torch.equal(k.results, c.results) and torch.equal(k.buffers.norms, c.buffers.norms)
    assert torch.equal(flat, (before.float() * f).to(BF16))


# ------------------------------------------------- scales, graphs, streams
def test_loss_scale_unscales_and_skips():
    xs = [x * 2.0 ** 10 for x in tensors(F16, sizes=[300, 5000])]
    ls = pkg.DeviceLossScale("cuda", init_scale=2.0 ** 10, growth_interval=1)
    ys = [torch.zeros(x.numel(), device="cuda") for x in xs]
    c = pkg.GradClip([300, 5000], max_norm=0.25)
    c.register_grads(xs, out=ys)
    c.launch(scale=123.0, loss_scale=ls)
    s = math.sqrt(sums_of(xs, 2, 2.0 ** -10).sum())
    assert c.finish().norm == pytest.approx(s, rel=SUM)
    for x, y in zip(xs, ys):
        check_clipped(y, x, 2.0 ** -10 * min(1.0, 0.25 / (s + 1e-6)), F32)
    assert int(ls.found_inf) == 0
    xs[1][7] = math.inf
    c.launch(loss_scale=ls)
    assert int(ls.found_inf) == 1 and int(c.found_nonfinite) == 0
    ls.launch_update(c.result)
    assert ls.scale == 2.0 ** 9


def test_captured_and_replayed():
    sizes = [300, 5000, 8]
    xs = [torch.zeros(n, dtype=dt, device="cuda") for n, dt in zip(sizes, TYPES)]
    c = pkg.GradClip(sizes, max_norm=0.5)
    d = pkg.GradClip(sizes, max_norm=0.25, norm_type=math.inf)
    c.register_grads(xs)
    d.register_grads(xs)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.launch()
        d.launch_norms()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.launch(scale=2.0)
        d.launch()
        with pytest.raises(RuntimeError, match="before the capture"):
            c.launch(xs)
        with pytest.raises(RuntimeError, match="before the capture"):
            pkg.clip_grad_norm_(xs, 1.0)
    for k in range(3):
        c.set_max_norm(0.5 + k)
        for i, x in enumerate(xs):
            x.copy_(torch.randn(x.numel(), generator=gen(10 * k + i)).cuda())
        b = [x.clone() for x in xs]
        s = math.sqrt(sums_of(b, 2, 2.0).sum())
        graph.replay()
        assert c.finish().norm == pytest.approx(s, rel=SUM)
        f = 2.0 * min(1.0, (0.5 + k) / (s + 1e-6))
        first = [(v.float() * np.float32(f)).to(v.dtype) for v in b]
        assert d.finish().norm == pytest.approx(max(float(v.float().abs().max()) for v in first), rel=4 * ULP + 2.0 ** -8)
        assert max(float(x.float().abs().max()) for x in xs) <= 0.25 * (1 + 2.0 ** -8)


def test_back_to_back_launches_see_each_other():
    """Each kernel may start before the one ahead of it has ended: clips in place one after the other, with kernels of
    torch between them or not, as if each had ended first."""
    n = 1 << 22
    sizes = [n // 7] * 6 + [n - 6 * (n // 7)]
    x = torch.randn(n, generator=gen(3)).bfloat16().cuda()
    want, y = x.clone(), x.clone()
    clips = [pkg.GradClip(sizes, max_norm=2.0 ** -k * 1000.0) for k in range(6)]
    for c in clips:
        c.register_grads(list(x.split(sizes)))
    for c in clips:  # with a wait after each
        c.launch(scale=1.5)
        torch.cuda.synchronize()
    first = x.clone()
    for gap in (False, True):
        for _ in range(5):
            x.copy_(y)
            for c in clips:
                c.launch(scale=1.5)
                if gap:
                    x.mul_(1.0)
            assert torch.equal(x, first)
    assert not torch.equal(first, want)


def test_captured_behind_copies_fills_and_other_streams():
    """What a launch follows in a graph: a copy, a fill, a join of another stream, another launch."""
    sizes = [70000, 300]
    y = torch.randn(70300, generator=gen(2)).cuda()
    x, host = torch.zeros_like(y), torch.zeros(70300).pin_memory()
    c, d = pkg.GradClip(sizes, max_norm=1.0), pkg.GradClip(sizes, max_norm=0.5)
    for k in (c, d):
        k.register_grads(list(x.split(sizes)))
    norms = torch.zeros(4, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.copy_(y)
        c.launch_norms()
        norms[0].copy_(c.norm)
        x.zero_()
        d.launch_norms()
        norms[1].copy_(d.norm)
        x.copy_(host, non_blocking=True)
        c.launch()
        norms[2].copy_(c.norm)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x.mul_(3.0)
        torch.cuda.current_stream().wait_stream(side)
        d.launch()
        norms[3].copy_(d.norm)
    for k in range(3):
        host.copy_(torch.randn(70300, generator=gen(k)))
        graph.replay()
        torch.cuda.synchronize()
        got = norms.tolist()
        assert got[0] == pytest.approx(float(y.double().norm()), rel=2 * ULP) and got[1] == 0.0
        assert got[2] == pytest.approx(float(host.double().norm()), rel=2 * ULP)
        # c left a norm of 1 - 1e-6 / |host| (and the elements' roundings, 2 x 2^-24 each), tripled
        assert got[3] == pytest.approx(3.0, rel=1e-6) and float(x.double().norm()) == pytest.approx(0.5, rel=3e-6)


def test_launches_on_another_stream():
    xs = tensors("mixed", 1)
    before = [x.clone() for x in xs]
    c = pkg.GradClip(SIZES, max_norm=0.5)
    s = math.sqrt(sums_of(before, 2).sum())
    side = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)
    for x in xs:
        x.mul_(2.0)  # behind the pause; the side stream waits for it
    side.wait_stream(torch.cuda.current_stream())
    r = c.clip_(xs, stream=side)
    assert r.norm == pytest.approx(2 * s, rel=SUM)
    for x, b in zip(xs, before):
        check_clipped(x, b, 2 * 0.5 / (2 * s + 1e-6), x.dtype)
    with torch.cuda.stream(side):
        n = pkg.clip_grad_norm_(xs, 0.25)
    side.synchronize()
    assert float(n) == pytest.approx(0.5, rel=1e-3)


def test_memory_of_a_launch_on_another_stream_is_not_given_out():
    n = 1 << 20
    c = pkg.GradClip([n], max_norm=0.5)
    side = torch.cuda.Stream()
    x, y = torch.full((n,), 2.0, device="cuda"), torch.empty(n, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    c.launch([x], out=[y], stream=side)
    gathered = torch.full((2, 1), 9.0, dtype=torch.float64, device="cuda")
    at = {x.data_ptr(), y.data_ptr(), gathered.data_ptr()}
    d = pkg.GradClip([n])
    d.launch_norms([x], gathered_sums=gathered, stream=side)
    del x, y, gathered
    new = [torch.full((n,), 7.0, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros((2, 1), dtype=torch.float64, device="cuda")]
    assert not at & {t.data_ptr() for t in new}
    assert c.finish(side).norm == 2.0 * 1024 and d.finish(side).norm == math.sqrt(18.0)
    # registered ones stay
    z = torch.full((n,), 3.0, device="cuda")
    c.register_grads([z])
    del z
    torch.full((n,), 7.0, device="cuda")
    assert c.clip_().norm == 3.0 * 1024


def test_what_waits_and_what_does_not():
    xs = [x for x in tensors("mixed", 1) if x.numel()]
    sizes = [x.numel() for x in xs]
    before = [x.clone() for x in xs]
    s = math.sqrt(sums_of(before, 2).sum())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # made there, used here: its tables and zeros are in place
        torch.cuda._sleep(20_000_000)
        c = pkg.GradClip(sizes, max_norm=0.5)
        assert side.query()
    assert c.clip_(xs).norm == pytest.approx(s, rel=SUM) and int(c.found_nonfinite) == 0
    for x, b in zip(xs, before):
        x.copy_(b)
    pkg.clip_grad_norm_([x.clone() for x in xs], 0.5)  # pinned memory is there from now on
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a backward pass that still runs
    n = pkg.clip_grad_norm_(xs, 0.5)
    busy = not torch.cuda.current_stream().query()
    assert busy and float(n) == pytest.approx(s, rel=SUM + ULP)
    for x, b in zip(xs, before):
        check_clipped(x, b, 0.5 / (s + 1e-6), x.dtype)
    torch.cuda._sleep(200_000_000)
    c.launch(xs)
    assert not torch.cuda.current_stream().query()
    assert c.finish().norm == pytest.approx(0.5, rel=1e-2)


def test_refuses_at_launch():
    x = torch.zeros(9, device="cuda")
    c = pkg.GradClip([4, 5])
    with pytest.raises(ValueError, match="overlaps"):
        c.launch([x[:4], x[3:8]])
    c.launch_norms([x[:4], x[3:8]])
    for bad in ([torch.zeros(4), x[:5]], [torch.zeros(4).pin_memory(), x[:5]]):
        with pytest.raises(ValueError, match="must be a tensor on"):
            c.launch(bad)
    with pytest.raises(ValueError, match="gathered_sums"):
        c.launch([x[:4], x[4:]], gathered_sums=torch.zeros(3, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="gathered_sums"):  # [tensors, ranks]
        c.launch_norms([x[:4], x[4:]], gathered_sums=torch.zeros(2, 3, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="float64"):
        c.launch([x[:4], x[4:]], gathered_sums=torch.zeros(2, device="cuda"))
    other = pkg.GradClip([9])
    for call in (lambda: zs.zero_list_norms(zs.grad_list(c.plan, [x[:4], x[4:]]), 1.0, False, other.buffers),
                 lambda: zs.zero_list_clip(other._entries([x], None, True)[0], 1.0, c.buffers)):
        with pytest.raises(ValueError, match="another plan"):
            call()


# ---------------------------------------------------------------- shards
@pytest.mark.parametrize("world", [2, 3, 8])
@pytest.mark.parametrize("p", [2, 1, math.inf])
def test_shards_join_to_the_whole(p, world):
    total = sum(SIZES)
    flat = torch.randn(total, generator=gen(9)) * 0.01
    xs = list(flat.split(SIZES))
    of = [i % 3 for i in range(len(SIZES))]
    limits = [0.5, 1e9, 0.01]
    s = sums_of(xs, p, 0.5)
    norms, coefs = coefs_of(s, of, limits, p)
    clips, shards = [], []
    for r in range(world):
        a, e = zs.zero_shard_range(total, world, r)
        shards.append(view(flat[a:e], 1 + r % 3))
        clips.append(pkg.GradClip.of_shard(SIZES, shards[-1], a, max_norm=limits, norm_type=p, group_of=of))
        clips[-1].launch_sums(scale=0.5)
    gathered = torch.stack([c.tensor_sums for c in clips])
    for c in clips:
        c.launch(scale=0.5, gathered_sums=gathered)
        res = c.finish()
        near(res.group_norms, norms, SUM)
        near(c.tensor_norms.cpu(), rooted(s, p), SUM + ULP)
        assert res.norm == pytest.approx(rooted(joined(s, p), p), rel=SUM)
        assert torch.equal(c.results, clips[0].results) and torch.equal(c.buffers.norms, clips[0].buffers.norms)
    got = torch.cat(shards).cpu().split(SIZES)
    for i, (y, x) in enumerate(zip(got, xs)):
        check_clipped(y, x, 0.5 * coefs[of[i]], F32)
    assert all(guards_intact(v) for v in shards)


def test_ranks_without_elements():
    x = torch.full((3,), 2.0, device="cuda")
    parts = [zs.zero_shard_range(3, 8, r) for r in range(8)]
    shards = [x[a:b].clone() for a, b in parts]
    clips = [pkg.GradClip.of_shard([2, 1], s, a, max_norm=np.float32(1.0)) for s, (a, _) in zip(shards, parts)]
    for c in clips:
        c.launch_sums()
    sums = torch.stack([c.tensor_sums for c in clips])
    assert sums.sum(0).tolist() == [8.0, 4.0] and sums[3:].abs().sum() == 0
    for c in clips:
        c.launch(gathered_sums=sums)
        assert c.finish().norm == math.sqrt(12.0)
    want = torch.full((3,), 2.0) * clips[0].finish().coefs[0]
    assert torch.equal(torch.cat(shards).cpu(), want)
    o = pkg.FlatShardAdamW([2, 1], world_size=8, rank=7, device="cuda")
    assert o.step(clip=o.grad_clip(max_norm=1.0)).finite and o.t == 1
    e = pkg.GradClip([0, 0], max_norm=1.0)
    assert e.clip_([None, torch.zeros(0, device="cuda")]).norm == 0.0


def test_one_ranks_overflow_stops_every_rank():
    flat = torch.ones(64, device="cuda")
    flat[40] = math.nan
    shards = [flat[:32].clone(), flat[32:].clone()]
    clips = [pkg.GradClip.of_shard([20, 44], x, 32 * r, max_norm=0.1) for r, x in enumerate(shards)]
    for c in clips:
        c.launch_sums()
    for c in clips:
        c.launch(gathered_sums=torch.stack([c.tensor_sums for c in clips]))
        assert not c.finish().finite
    assert bool((shards[0] == 1).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_a_shards_step_with_a_clip_per_group(bits, capturable):
    kw = dict(lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, device="cuda", state_bits=bits, capturable=capturable)
    total = sum(SIZES)
    master = torch.randn(total, generator=gen(5)).cuda()
    a = pkg.FlatShardAdamW(SIZES, master=master.clone(), max_norm=1e-9, **kw)  # its own limit is not used
    b = pkg.FlatShardAdamW(SIZES, master=master.clone(), max_norm=math.inf, **kw)
    of = [i % 3 for i in range(len(SIZES))]
    clip = a.grad_clip(group_of=of, max_norm=[0.1, 10.0, 0.01])
    for step in range(3):
        xs = tensors(BF16, 0, seed=step)
        a.flatten(xs, accumulate=False, scale=0.5, fuse_norm=step == 1)
        r = a.step(clip=clip)
        assert r.finite and r.clip_coef == 1.0 and a.t == step + 1
        b.flatten(xs, accumulate=False, scale=0.5)
        c = clip.finish().coefs
        at = 0
        for i, n in enumerate(SIZES):
            b.grad[at:at + n].mul_(float(c[of[i]]))  # fl(c x), as the clip rounds it
            at += n
        assert torch.equal(a.grad, b.grad)
        b.step()
        assert torch.equal(a.master.view(torch.int32), b.master.view(torch.int32)) and torch.equal(a.lowp, b.lowp)
    a.grad[3] = math.inf
    before = a.master.clone()
    assert not a.step(clip=clip).finite and a.t == 3 and torch.equal(a.master, before)


@pytest.mark.parametrize("grad_range", ["shard", "full"])
def test_a_captured_shard_step_with_a_clip(grad_range):
    """Flatten, clip by groups and AdamW of a rank's shard (ZeRO-2 and ZeRO-1), captured and replayed against eager steps."""
    total = sum(SIZES)
    s, e = zs.zero_shard_range(total, 2, 1)
    master = torch.randn(total, generator=gen(8))[s:e].cuda()
    kw = dict(world_size=2, rank=1, lr=1e-2, device="cuda", grad_range=grad_range, capturable=True)
    a, b = (pkg.FlatShardAdamW(SIZES, master=master.clone(), **kw) for _ in range(2))
    of = [i % 2 for i in range(len(SIZES))]
    ca, cb = (o.grad_clip(group_of=of, max_norm=[0.05, 0.5]) for o in (a, b))
    xs = tensors(BF16)
    a.register_grads(xs)
    b.register_grads(xs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.flatten(accumulate=False, scale=0.5, fuse_norm=True)
        a.launch_clip(ca)
    for k in range(3):
        for i, x in enumerate(xs):
            x.copy_((torch.randn(x.numel(), generator=gen(90 * k + i)) * 0.02).cuda())
        if k == 1:
            a.grad.fill_(math.nan)  # flatten writes it anew
            xs[13][5] = math.inf
        graph.replay()
        b.flatten(accumulate=False, scale=0.5)
        r = b.step(clip=cb)
        assert torch.equal(ca.results.view(torch.int32), cb.results.view(torch.int32)) and r.finite == (k != 1)
        assert torch.equal(a.master, b.master) and torch.equal(a.exp_avg, b.exp_avg) and torch.equal(a.lowp, b.lowp)
    assert a.t == b.t == 2


def test_two_clips_at_once():
    sizes = [1 << 20, 5, 300000, 16384]
    data = [[torch.randn(n, generator=gen(n + k)).to(TYPES[k]).cuda() for n in sizes] for k in range(3)]
    want = []
    for xs in data:
        one = [x.clone() for x in xs]
        c = pkg.GradClip(sizes, max_norm=[3.0, 1.0], group_of=[0, 1, 1, 0])
        for _ in range(6):
            c.launch(one, scale=1.5)
        want.append((one, c.results.clone()))
    torch.cuda.synchronize()
    clips, streams = [pkg.GradClip(sizes, max_norm=[3.0, 1.0], group_of=[0, 1, 1, 0]) for _ in data], [torch.cuda.Stream() for _ in data]
    for c, xs in zip(clips, data):
        c.register_grads(xs)
    for _ in range(6):
        for c, st in zip(clips, streams):
            c.launch(scale=1.5, stream=st)
    torch.cuda.synchronize()
    for c, xs, (one, results) in zip(clips, data, want):
        assert torch.equal(c.results, results) and all(torch.equal(x, y) for x, y in zip(xs, one))


def test_a_list_step_after_a_clip_in_one_graph():
    """Unscale and clip fp16 grads into fp32 by groups, then AdamW over the list, captured once."""
    sizes = [300, 7, 4100]
    of = [0, 1, 0]
    xs = [torch.zeros(n, dtype=F16, device="cuda") for n in sizes]
    ys = [torch.zeros(n, device="cuda") for n in sizes]
    ls = pkg.DeviceLossScale("cuda", init_scale=2.0 ** 8)
    masters = [torch.randn(n, generator=gen(n)).cuda() for n in sizes]
    opt = pkg.TensorListAdamW([m.clone() for m in masters], lr=1e-2, capturable=True)
    ref = pkg.TensorListAdamW([m.clone() for m in masters], lr=1e-2)
    opt.register_grads(ys)
    clip = pkg.GradClip(sizes, max_norm=[0.1, 0.01], group_of=of)
    clip.register_grads(xs, out=ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip.launch(loss_scale=ls)
        opt.launch_step(norm_result=clip.result)
        ls.launch_update(clip.result)
    for k in range(4):
        for i, x in enumerate(xs):
            x.copy_((torch.randn(x.numel(), generator=gen(50 * k + i)) * 20).cuda())
        if k == 2:
            xs[1][3] = math.inf
        graph.replay()
        r = clip.finish()
        assert r.finite == (k != 2)
        if k != 2:
            scale = np.float32(2.0 ** -8 if k < 2 else 2.0 ** -7)
            ref.launch_step([x.float() * float(scale * r.coefs[g]) for x, g in zip(xs, of)], norm_result=clip.result)
            ref.finish_step(norm_result=clip.result)
        for a, b in zip(opt.masters, ref.masters):
            assert torch.equal(a, b), k
    assert opt.t == ref.t == 3 and ls.scale == 2.0 ** 7

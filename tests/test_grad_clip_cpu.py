"""Host side of the norms and clipping of a list, without a GPU: the plan, the checks of a list's tensors, what is refused."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs


def parts(plan):
    n, g = len(plan.numels), plan.n_groups
    a = plan.ints.numpy()
    assert len(a) == 4 * n + g + 2
    return a[:n + 1], a[n + 1:n + g + 2], a[n + g + 2:2 * n + g + 2], a[2 * n + g + 2:3 * n + g + 2], a[3 * n + g + 2:]


@pytest.mark.parametrize("sizes,chunk", [([1], 4096), ([0], 4096), ([4096, 4097, 0, 4095, 0, 0, 1], 4096), ([1 << 21], 4096),
                                         ([(1 << 21) + 1], 8192), ([1 << 24], 8192), ([1, 1 << 24, 5], 16384),
                                         ([1 << 26], 16384), ([16384, 1 << 27, 16385], 32768), ([(1 << 29) + 1], 131072),
                                         ([4095, 1 << 40, 16384, 16385, 3], 131072)])
def test_plan_cuts_long_tensors_into_chunks(sizes, chunk):
    p = zs.zero_grad_plan(sizes, None, 1, 2, "cpu")
    first, group_first, members, narrow_of, narrow = parts(p)
    assert p.head.chunk == chunk
    assert first.tolist() == np.concatenate([[0], np.cumsum([-(-n // chunk) if n > min(chunk, 16384) else 0 for n in sizes])]).tolist()
    small = [i for i, n in enumerate(sizes) if 0 < n <= min(chunk, 16384)]
    assert narrow[:len(small)].tolist() == small and p.head.n_narrow == len(small) and p.head.n_wide == first[-1]
    assert narrow_of.tolist() == [small.index(i) if i in small else -1 for i in range(len(sizes))]
    assert members.tolist() == list(range(len(sizes))) and group_first.tolist() == [0, len(sizes)]
    assert zs.zero_list_norms_workspace_bytes(p) == 8 * (p.head.n_wide + len(small))
    assert (p.head.n_tensors, p.head.n_groups, p.head.in_place, p.head.d_entries) == (len(sizes), 1, 0, None)


def test_plan_sorts_groups_and_keeps_list_order():
    of = [2, 0, 2, 4, 0, 0, 2]
    _, group_first, members, _, _ = parts(zs.zero_grad_plan([3] * 7, of, 6, math.inf, "cpu"))
    got = [members[group_first[g]:group_first[g + 1]].tolist() for g in range(6)]
    assert got == [[i for i, k in enumerate(of) if k == g] for g in range(6)]


@pytest.mark.parametrize("args", [([], None, 1), ([1], None, 0), ([-1], None, 1), ([1, 1], [0, 2], 2), ([1, 1], [0, -1], 2),
                                  ([1 << 62, 1 << 62], None, 1), ([1 << 50], None, 1)])
def test_plan_refuses(args):
    with pytest.raises(zs.ZeroError):
        zs.zero_grad_plan(*args, 2, "cpu")


def test_plan_refuses_counts_and_nothing():
    a, h = np.zeros(16, np.int64), zs.zero_grad_list()
    call = zs.lib().zero_grad_plan
    ok = (a.ctypes.data, None, 1, 1, a.ctypes.data, ctypes.byref(h))
    for i, bad in ((0, None), (2, (1 << 28) + 1), (3, (1 << 28) + 1), (4, None), (5, None)):
        assert call(*ok[:i], bad, *ok[i + 1:]) == zs.ZERO_EINVAL
    assert zs.lib().zero_list_norms_workspace_bytes(None) == 0


def test_plan_refuses_by_name():
    with pytest.raises(ValueError, match="norm_type"):
        zs.zero_grad_plan([1], None, 1, 3, "cpu")
    with pytest.raises(ValueError, match="one group per tensor"):
        zs.zero_grad_plan([1, 2], [0], 1, 2, "cpu")


def a_plan(sizes):
    return zs.zero_grad_plan(sizes, None, 1, 2, "cpu")


def test_list_takes_dense_tensors_in_any_order_of_dimensions():
    t = torch.zeros(4, 6)
    plan = a_plan([24, 24, 0, 24])
    u = torch.zeros(2, 3, 4).permute(2, 0, 1)
    gl = zs.grad_list(plan, [t.t(), u, torch.zeros(0, 5), None])
    e = gl.entries.numpy().view(zs._GRAD_ENTRY)
    assert e["src"].tolist()[:2] == [t.data_ptr(), u.data_ptr()] and e["src"][3] == 0 and (e["dst"] == e["src"]).all()
    assert zs._dense(torch.zeros(1, 4)[:, :].expand(1, 4)) and zs._dense(torch.zeros(3, 1, 2).transpose(0, 1))


@pytest.mark.parametrize("bad,match", [
    (lambda: [torch.zeros(4, 6)[:, :5], None], "one run of memory"),
    (lambda: [torch.zeros(1, 4).expand(5, 4), None], "one run of memory"),
    (lambda: [torch.zeros(20, dtype=torch.float64), None], "not f32"),
    (lambda: [torch.zeros(20, dtype=torch.int32), None], "not f32"),
    (lambda: [torch.zeros(19), None], "19 elements"),
    (lambda: [torch.zeros(20)], "per tensor"),
    (lambda: [np.zeros(20, np.float32), None], "must be a tensor"),
    (lambda: [torch.zeros(20, device="meta"), None], "must be a tensor on"),
])
def test_list_refuses(bad, match):
    with pytest.raises(ValueError, match=match):
        zs.grad_list(a_plan([20, 7]), bad())


def test_list_refuses_what_overlaps_a_written_one():
    x = torch.zeros(64)
    plan = a_plan([20, 20])
    ok = [x[:20], x[20:40]]
    zs.grad_list(plan, ok)
    for bad in ([x[:20], x[:20]], [x[:20], x[19:39]], [x[10:30], x[:20]]):
        with pytest.raises(ValueError, match="overlaps"):
            zs.grad_list(plan, bad)
        zs.grad_list(plan, bad, write=False)  # norms may count a tensor twice
        zs.grad_list(plan, bad, [torch.zeros(20), torch.zeros(20)])  # and read one twice
    y = torch.zeros(64)
    with pytest.raises(ValueError, match="overlaps"):  # one destination over the other
        zs.grad_list(plan, ok, [y[:20], y[1:21]])
    with pytest.raises(ValueError, match="overlaps"):  # a destination over another tensor's grad
        zs.grad_list(plan, ok, [x[20:40], None])
    with pytest.raises(ValueError, match="overlaps"):  # or partly over its own
        zs.grad_list(plan, [x[:20], None], [x[1:21], None])
    with pytest.raises(ValueError, match="overlaps"):  # a 16-bit copy written over its own grad's memory
        zs.grad_list(plan, [x[:20], None], [x[10:20].view(torch.bfloat16), None])
    zs.grad_list(plan, ok, [x[:20], y[:20]])  # in place and elsewhere in one list
    # a long one over two short ones
    with pytest.raises(ValueError, match="overlaps"):
        zs.grad_list(a_plan([60, 2, 2]), [x[:60], torch.zeros(2), x[50:52]])


def test_list_refuses_other_layouts_of_out():
    plan = a_plan([24])
    with pytest.raises(ValueError, match="laid out"):
        zs.grad_list(plan, [torch.zeros(4, 6).t()], [torch.zeros(6, 4)])
    zs.grad_list(plan, [torch.zeros(4, 6).t()], [torch.zeros(4, 6, dtype=torch.bfloat16).t()])
    with pytest.raises(ValueError, match="has 23 elements"):
        zs.grad_list(plan, [torch.zeros(24)], [torch.zeros(23)])


def entry(**kw):
    e = np.zeros(1, dtype=zs._GRAD_ENTRY)
    x = np.zeros(16, np.float32)
    e["src"], e["numel"] = x.ctypes.data, 4
    for k, v in kw.items():
        e[k] = v
    return e, x


@pytest.mark.parametrize("kw", [dict(numel=5), dict(numel=-1), dict(group=1), dict(group=-1), dict(reserved=1), dict(src_dtype=3),
                                dict(dst_dtype=-1), dict(src=2 ** 20 + 2), dict(dst=2 ** 20 + 1, dst_dtype=1),
                                dict(src=2 ** 20, dst=2 ** 20, dst_dtype=1)])
def test_entries_check_refuses(kw):
    e, _x = entry(**kw)
    n = np.array([4], np.int64)
    assert zs.lib().zero_grad_entries_check(e.ctypes.data, n.ctypes.data, 1, 1) == zs.ZERO_EINVAL
    good, _y = entry()
    assert zs.lib().zero_grad_entries_check(good.ctypes.data, n.ctypes.data, 1, 1) == zs.ZERO_OK


def test_c_entries_refuse_before_any_launch():
    L = zs.lib()
    P = ctypes.c_void_p
    buf = ctypes.cast(ctypes.create_string_buffer(4096 + 64), P).value
    a = (buf + 63) & ~63

    def head(**kw):
        f = dict(d_entries=a, d_plan=a, n_tensors=2, n_groups=1, n_wide=1, n_narrow=2, chunk=4096, norm_type=2, in_place=0)
        f.update(kw)
        return ctypes.byref(zs.zero_grad_list(**f))

    heads = [dict(d_plan=None), dict(d_plan=a + 2), dict(n_tensors=0), dict(n_groups=0), dict(n_wide=-1), dict(n_narrow=-1), dict(n_narrow=3),
             dict(n_wide=1 << 28), dict(chunk=0), dict(chunk=5000),
             dict(chunk=262144), dict(norm_type=3), dict(norm_type=-1), dict(in_place=2)]
    for kw in heads + [dict(d_entries=None), dict(d_entries=a + 4)]:
        assert L.zero_list_sums(head(**kw), 1.0, None, a, 24, a, None) == zs.ZERO_EINVAL, kw
        assert L.zero_list_clip(head(**kw), 1.0, None, a, None) == zs.ZERO_EINVAL, kw
        assert L.zero_list_norms(head(**kw), 1.0, None, 1, a, 24, a, a, a, a, a, None) == zs.ZERO_EINVAL, kw
    for kw in heads:
        assert L.zero_sums_norms(head(**kw), a, 1, a, a, a, a, None, None) == zs.ZERO_EINVAL, kw
    h = head()
    assert L.zero_list_sums(None, 1.0, None, a, 24, a, None) == zs.ZERO_EINVAL
    for bad in ((math.nan, None, a, 24, a), (math.inf, None, a, 24, a), (1.0, a + 1, a, 24, a), (1.0, None, None, 24, a), (1.0, None, a, 23, a),
                (1.0, None, a + 4, 24, a), (1.0, None, a, 24, None), (1.0, None, a, 24, a + 4)):
        assert L.zero_list_sums(h, *bad, None) == zs.ZERO_EINVAL, bad
        sc, ds, ws, nb, sums = bad
        assert L.zero_list_norms(h, sc, ds, 0, ws, nb, sums, a, a, a, None, None) == zs.ZERO_EINVAL, bad
    ok = (a, 1, a, a, a, a, None)
    for i, v in ((0, None), (0, a + 4), (1, 0), (2, None), (2, a + 4), (3, None), (3, a + 4), (4, None), (4, a + 2), (5, None), (5, a + 4), (6, a + 2)):
        bad = ok[:i] + (v,) + ok[i + 1:]
        assert L.zero_sums_norms(h, *bad, None) == zs.ZERO_EINVAL, bad
    assert L.zero_list_clip(h, 1.0, None, None, None) == zs.ZERO_EINVAL
    assert L.zero_list_clip(h, math.nan, None, a, None) == zs.ZERO_EINVAL


def test_clip_refuses_on_the_host():
    make = lambda **kw: pkg.GradClip([4, 5], device="cpu", **kw)  # noqa: E731
    for kw, match in ((dict(max_norm=-1.0), "max_norm"), (dict(max_norm=math.nan), "max_norm"), (dict(max_norm=[1.0, 2.0, -3.0]), "max_norm"),
                      (dict(norm_type=0), "norm_type"), (dict(group_of=[0]), "one group per tensor")):
        with pytest.raises(ValueError, match=match):
            make(**kw)
    with pytest.raises(zs.ZeroError):  # a group beyond the limits
        make(group_of=[0, 2], max_norm=[1.0, 1.0])
    with pytest.raises(ValueError, match="empty"):
        pkg.GradClip([], device="cpu")
    c = make(group_of=[0, 1])
    assert c.n_groups == 2 and c.max_norms.tolist() == [math.inf] * 2
    c.set_max_norm([1.0, 0.0])
    with pytest.raises(ValueError, match="limits for 2 groups"):
        c.set_max_norm([1.0])
    with pytest.raises(ValueError, match="none registered"):
        c.launch()
    with pytest.raises(ValueError, match="out needs grads"):
        c.launch(out=[None, None])
    x = torch.zeros(9)
    c.register_grads([x[:4], x[:5]], write=False)
    with pytest.raises(ValueError, match="norms only"):
        c.launch()
    with pytest.raises(ValueError, match="max_norms"):
        zs.norm_buffers(c.plan, torch.zeros(3, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):  # host memory never reaches a kernel
        c.launch_norms()
    with pytest.raises(ValueError, match="gathered_sums"):
        c.launch_norms(gathered_sums=torch.zeros(3, dtype=torch.float64))
    with pytest.raises(ValueError, match="no grads"):
        pkg.clip_grad_norm_([None], 1.0)


@pytest.mark.parametrize("world", [1, 2, 3, 8])
def test_shard_pieces_cover_every_tensor_once(world):
    sizes = [5, 0, 1, 17, 3, 0, 40, 2]
    total = sum(sizes)
    got = np.zeros(len(sizes), np.int64)
    flat = torch.arange(total, dtype=torch.float32)
    for r in range(world):
        s, e = zs.zero_shard_range(total, world, r)
        c = pkg.GradClip.of_shard(sizes, flat[s:e], s)
        got += c.plan.numels
        ent = c._registered[0].entries.numpy().view(zs._GRAD_ENTRY)
        at = 0
        for i, n in enumerate(sizes):
            lo, hi = max(at, s), min(at + n, e)
            assert c.numels[i] == max(0, hi - lo)
            if hi > lo:
                assert ent["src"][i] == ent["dst"][i] == flat.data_ptr() + 4 * lo
            at += n
    assert got.tolist() == sizes
    with pytest.raises(ValueError, match="not a shard"):
        pkg.GradClip.of_shard(sizes, flat, 1)
    with pytest.raises(ValueError, match="1-D"):
        pkg.GradClip.of_shard([4], torch.zeros(2, 2), 0)
    with pytest.raises(ValueError, match="1-D"):
        pkg.GradClip.of_shard([4], torch.zeros(4, dtype=torch.float64), 0)
    with pytest.raises(ValueError, match="outside"):
        zs.flat_grad_list(a_plan([4, 3]), torch.zeros(7), np.array([0, 5]))


def test_optimizer_refuses_a_clip_over_another_buffer():
    o = pkg.FlatShardAdamW([8], device="cpu")
    c = pkg.GradClip.of_shard([8], torch.zeros(8), 0)
    with pytest.raises(ValueError, match="not over this optimizer"):
        o.step(clip=c)
    with pytest.raises(ValueError, match="extra_sqnorm"):
        o.step(1.0, clip=o.grad_clip())
    with pytest.raises(ValueError, match="grad buffer"):
        pkg.FlatShardAdamW([8], device="cpu", grad_buffer=False).grad_clip()


def test_one_limit_or_one_for_each_group():
    for one in (1, 1.0, np.float32(1), np.array(1.0), torch.tensor(1.0), math.inf):
        assert pkg.GradClip([4, 5], device="cpu", group_of=[0, 1], max_norm=one).max_norms.tolist() == [float(one)] * 2
    for each in ([1, 2.0], (1.0, 2.0), np.array([1.0, 2.0]), torch.tensor([1.0, 2.0])):
        assert pkg.GradClip([4, 5], device="cpu", group_of=[0, 1], max_norm=each).max_norms.tolist() == [1.0, 2.0]


def test_list_steps_with_clips_refuse():
    L = zs.lib()
    buf = ctypes.cast(ctypes.create_string_buffer(4096 + 64), ctypes.c_void_p).value
    a = (buf + 63) & ~63
    hp = zs.list_groups([(1e-3, 0.9, 0.99, 1e-8, 0.0)])
    for bad in (None, a + 4):
        assert L.zero_adamw_list_clips(a, 1, a, 1, 32, a, 0, 1.0, None, 1, hp, 1, 1, None, bad, None) == zs.ZERO_EINVAL
        assert L.zero_adamw_list_clips_device(a, 1, a, 1, 32, a, 0, 1.0, None, 1, a, 1, None, bad, None) == zs.ZERO_EINVAL
    assert L.zero_adamw_list_clips(a, 1, a, 1, 16, a, 0, 1.0, None, 1, hp, 1, 1, None, a, None) == zs.ZERO_EINVAL
    assert L.zero_adamw_list_clips(a, 1, a, 0, 32, a, 0, 1.0, None, 1, hp, 1, 1, None, a, None) == zs.ZERO_OK

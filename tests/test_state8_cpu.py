"""8-bit moments and tensor lists without a GPU: the list's chunks, the refusals of the C entries and of the binding, and the 64-bit reference's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs
import _ref8 as R

FAKE = 0x10000  # an address that no call may touch: every call below is refused before a launch
HP = zs.zero_adamw_hparams(1e-3, 0.9, 0.99, 1e-8, 0.1)


def entry(numel, bits=32, **kw):
    e = dict(master=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, numel=numel)
    if bits == 8:
        e.update(exp_avg_scale=FAKE, root_scale=FAKE)
    e.update(kw)
    return zs.zero_list_tensor(**e)


def chunks_of(entries, n_groups=1, bits=32, fill=True):
    """(status, first_chunk) of a list."""
    arr = (zs.zero_list_tensor * max(len(entries), 1))(*entries)
    count = ctypes.c_int32(-1)
    out = np.full(len(entries) + 2, -7, dtype=np.int32)
    st = zs.lib().zero_list_chunks(arr, len(entries), n_groups, bits, ctypes.c_void_p(out.ctypes.data) if fill else None,
                                   ctypes.byref(count))
    assert out[-1] == -7
    if st == zs.ZERO_OK and fill:
        assert count.value == out[-2]
    return st, out[:-1]


# --------------------------------------------------------------- reference
def test_reference_grid_is_torch_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.TABLE, t)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(200000, generator=g) * torch.exp2(torch.rand(200000, generator=g) * 24 - 14)
    x = x.clamp(-448, 448)
    np.testing.assert_array_equal(R.grid(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_reference_stochastic_rounding_has_the_right_mean():
    # over the 128 values of k the mean is floor(128 x / u) u / 128: within u / 128 below x
    x = np.random.default_rng(0).uniform(-448, 448, 500)
    x[:100] *= 2.0 ** -14
    mean = np.mean([R.grid(x, k) for k in range(128)], axis=0)
    u = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    assert (np.abs(mean) <= np.abs(x)).all() and (np.abs(x) - np.abs(mean) < u / 128).all()


def test_reference_scale():
    a = np.array([0.0, 448.0, np.nextafter(448.0, 500), 224.0, 2.0 ** -130, 1e-30, 2.0 ** 126, np.inf, np.nan])
    s = R.scale_of(a)
    np.testing.assert_array_equal(s[:5], [2.0 ** -126, 1.0, 2.0, 0.5, 2.0 ** -126])
    assert 224 * s[5] < 1e-30 <= 448 * s[5] and np.isnan(s[6:]).all()


def test_reference_step_is_torch_adamw():
    rng = np.random.default_rng(1)
    p0, g = rng.normal(size=50), rng.normal(size=(3, 50))
    t = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for i in range(3):
        t.grad = torch.from_numpy(g[i].copy())
        opt.step()
        out = R.step(p, m, v, g[i], 0 * g[i], lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, wd=0.1, t=i + 1)
        p, m, v = out["p"][0], out["m"][0], out["r"][0] ** 2
    np.testing.assert_allclose(p, t.detach().numpy(), rtol=1e-12)


# ------------------------------------------------------------------ chunks
def test_chunks_follow_the_tensors():
    sizes = [0, 1, zs.LIST_CHUNK - 1, zs.LIST_CHUNK, zs.LIST_CHUNK + 1, 0, 10000]
    st, c = chunks_of([entry(n) for n in sizes])
    assert st == zs.ZERO_OK and c.tolist() == np.cumsum([0] + [-(-n // zs.LIST_CHUNK) for n in sizes]).tolist()
    st, c = chunks_of([])
    assert st == zs.ZERO_OK and c.tolist() == [0]
    st, c = chunks_of([zs.zero_list_tensor(numel=0)], bits=8)  # nothing to point at
    assert st == zs.ZERO_OK and c.tolist() == [0, 0]


@pytest.mark.parametrize("bad", [
    [entry(-1)], [entry(5, group=1)], [entry(5, group=-1)], [entry(5, reserved=1)], [entry(5, master=None)],
    [entry(5, exp_avg=None)], [entry(5, exp_avg_sq=None)], [entry(5, exp_avg_scale=FAKE)], [entry(5, root_scale=FAKE)],
    [entry(5, master=FAKE + 2)], [entry(5, exp_avg=FAKE + 1)], [entry(5, lowp=FAKE + 1)], [entry(1 << 43)],
    [entry(1 << 41), entry(1 << 41)],
])
def test_bad_lists_are_refused(bad):
    assert chunks_of(bad, fill=False)[0] == zs.ZERO_EINVAL


def test_bad_8bit_lists_and_arguments_are_refused():
    ok = [entry(5, 8)]
    assert chunks_of(ok, bits=8)[0] == zs.ZERO_OK
    assert chunks_of([entry(5, 8, exp_avg=FAKE + 3)], bits=8)[0] == zs.ZERO_OK  # codes may start anywhere
    assert chunks_of([entry(5)], bits=8)[0] == zs.ZERO_EINVAL
    assert chunks_of([entry(5, 8, root_scale=None)], bits=8)[0] == zs.ZERO_EINVAL
    assert chunks_of([entry(5, 8, root_scale=FAKE + 2)], bits=8)[0] == zs.ZERO_EINVAL
    assert chunks_of(ok, bits=16)[0] == zs.ZERO_EINVAL
    for groups in (0, 65):
        assert chunks_of(ok, n_groups=groups, bits=8)[0] == zs.ZERO_EINVAL
    assert zs.lib().zero_list_chunks(None, 1, 1, 32, None, None) == zs.ZERO_EINVAL
    assert zs.lib().zero_list_chunks(None, -1, 1, 32, None, None) == zs.ZERO_EINVAL
    assert zs.lib().zero_list_chunks(None, 0, 1, 32, None, None) == zs.ZERO_OK


# ---------------------------------------------------------------- refusals
def call_list(**kw):
    hp = kw.pop("hp", HP)
    a = dict(list=FAKE, n_tensors=1, first=FAKE, n_chunks=1, bits=8, grads=FAKE, dt=0, scale=1.0, dscale=None, lowp=1,
             groups=ctypes.byref(hp) if hp is not None else None, n_groups=1, step=1, seed=None, clip=None, stream=None)
    a.update(kw)
    return zs.lib().zero_adamw_list(*a.values())


@pytest.mark.parametrize("bad", [
    dict(list=None), dict(first=None), dict(grads=None), dict(n_tensors=0), dict(n_tensors=-1), dict(n_chunks=-1),
    dict(bits=4), dict(dt=3), dict(scale=float("nan")), dict(lowp=0), dict(hp=None), dict(n_groups=0),
    dict(n_groups=65), dict(step=0), dict(list=FAKE + 4), dict(first=FAKE + 2), dict(grads=FAKE + 4),
    dict(bits=32, seed=ctypes.byref(zs.zero_rounding(1, 0))), dict(hp=zs.zero_adamw_hparams(-1, 0.9, 0.9, 1e-8, 0)),
    dict(hp=zs.zero_adamw_hparams(1e-3, 1.0, 0.9, 1e-8, 0)), dict(hp=zs.zero_adamw_hparams(1e-3, 0.9, 0.9, 0, 0)),
])
def test_list_step_refuses(bad):
    assert call_list(**bad) == zs.ZERO_EINVAL


def test_list_step_of_nothing_is_a_no_op():
    assert call_list(n_chunks=0, list=None, first=None, grads=None, n_tensors=0) == zs.ZERO_OK


def test_list_device_forms_refuse():
    L = zs.lib()

    def dev(states=FAKE, n_groups=1, **kw):
        a = dict(list=FAKE, n_tensors=1, first=FAKE, n_chunks=1, bits=8, grads=FAKE, dt=0, scale=1.0, dscale=None,
                 lowp=1, states=states, n_groups=n_groups, seed=None, clip=None, stream=None)
        a.update(kw)
        return L.zero_adamw_list_device(*a.values())

    for bad in (dict(states=None), dict(states=FAKE + 4), dict(n_groups=0), dict(n_groups=65), dict(bits=7),
                dict(scale=float("inf"))):
        assert dev(**bad) == zs.ZERO_EINVAL
    for args in ((None, 1, None, FAKE), (FAKE + 4, 1, None, FAKE), (FAKE, 0, None, FAKE), (FAKE, 65, None, FAKE),
                 (FAKE, 1, None, None), (FAKE, 1, None, FAKE + 4)):
        assert L.zero_adamw_prepare_list_device(*args, None) == zs.ZERO_EINVAL


def state8(**kw):
    return zs.zero_state8(**{**dict(exp_avg=FAKE, exp_avg_scale=FAKE, root=FAKE, root_scale=FAKE), **kw})


def call_step8(**kw):
    q, hp = kw.pop("q", state8()), kw.pop("hp", HP)
    a = dict(master=FAKE, q=None if q is None else ctypes.byref(q), table=FAKE, n_tensors=1, total=100, dt=1, start=0,
             scale=1.0, dscale=None, acc=None, lowp=None, lowp_dt=1, n=100, hp=None if hp is None else ctypes.byref(hp),
             step=1, seed=None, clip=None, stream=None)
    a.update(kw)
    return zs.lib().zero_adamw_step8_tensors(*a.values())


@pytest.mark.parametrize("bad", [
    dict(master=None), dict(q=None), dict(q=state8(exp_avg=None)), dict(q=state8(exp_avg_scale=None)),
    dict(q=state8(root=None)), dict(q=state8(root_scale=None)), dict(q=state8(root_scale=FAKE + 1)), dict(table=None),
    dict(n_tensors=-1), dict(n_tensors=0), dict(total=-1), dict(dt=5), dict(start=1), dict(start=-1), dict(n=101),
    dict(n=-1), dict(scale=float("inf")), dict(lowp=FAKE, lowp_dt=0), dict(hp=None), dict(step=0),
])
def test_step8_refuses(bad):
    assert call_step8(**bad) == zs.ZERO_EINVAL


def test_step8_and_conversions_of_nothing():
    empty = zs.zero_state8()
    assert call_step8(q=empty, n=0, total=0, master=None) == zs.ZERO_OK
    L, q = zs.lib(), state8()
    assert L.zero_state8_pack(None, None, 0, ctypes.byref(empty), None) == zs.ZERO_OK
    assert L.zero_state8_unpack(ctypes.byref(empty), 0, None, None, None) == zs.ZERO_OK
    for n, a, b, s in ((-1, FAKE, FAKE, q), (4, None, FAKE, q), (4, FAKE, None, q), (4, FAKE, FAKE, empty)):
        assert L.zero_state8_pack(a, b, n, ctypes.byref(s), None) == zs.ZERO_EINVAL
        assert L.zero_state8_unpack(ctypes.byref(s), n, a, b, None) == zs.ZERO_EINVAL
    assert L.zero_state8_pack(FAKE, FAKE, 4, None, None) == zs.ZERO_EINVAL
    assert L.zero_adamw_step8_tensors_device(FAKE, ctypes.byref(q), FAKE, 1, 4, 0, 0, 1.0, None, None, None, 1, 4, None,
                                             None, None, None) == zs.ZERO_EINVAL


def test_binding_refuses_host_tensors_and_bad_states():
    n = 300
    s = zs.new_state8(n, "cpu")
    assert s.exp_avg.dtype == torch.float8_e4m3fn and s.exp_avg_scale.numel() == 2
    with pytest.raises(ValueError, match="CUDA"):
        pkg.zero_state8_pack(torch.zeros(n), torch.zeros(n), s)
    with pytest.raises(ValueError, match="differs in size"):
        pkg.zero_state8_unpack(s, torch.zeros(n), torch.zeros(n + 1))
    with pytest.raises(ValueError, match="State8"):
        pkg.zero_state8_pack(torch.zeros(n), torch.zeros(n), [1, 2])
    with pytest.raises(ValueError, match="CUDA"):
        pkg.TensorListAdamW([torch.zeros(n)])
    with pytest.raises(ValueError, match="state_bits"):
        pkg.TensorListAdamW([torch.zeros(n)], state_bits=16)
    with pytest.raises(ValueError, match="rounding_seed"):
        pkg.TensorListAdamW([torch.zeros(n)], rounding_seed=1)
    with pytest.raises(ValueError, match="group"):
        pkg.TensorListAdamW([torch.zeros(n)], groups=[{"momentum": 1}])
    with pytest.raises(ValueError, match="empty"):
        pkg.TensorListAdamW([])
    with pytest.raises(ValueError, match="state_bits"):
        pkg.FlatShardAdamW([n], device="cpu", state_bits=4)
    with pytest.raises(ValueError, match="rounding_seed"):
        pkg.FlatShardAdamW([n], device="cpu", rounding_seed=4)

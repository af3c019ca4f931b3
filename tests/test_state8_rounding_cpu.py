"""Stochastic rounding of 8-bit moments without a GPU: what its two forms do to a recurrence, and the refusals of a bad one."""
import ctypes
import inspect

import numpy as np
import pytest

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs
import _ref8 as R
import _ref8_runs as L
from test_state8_cpu import call_list, call_step8


def test_halves_hold_the_seven_bit_draws():
    h = L.halves(0x123456789ABCDEF1, 7, 5, 1001, first=3).astype(np.uint64)
    km, kr = R.draws(0x123456789ABCDEF1, 7, 5, 1001, first=3)
    np.testing.assert_array_equal(h & np.uint64(127), km)
    np.testing.assert_array_equal((h >> np.uint64(7)) & np.uint64(127), kr)


def test_sixteen_bit_rounding_has_the_right_mean():
    # over the 65536 values of h the mean is x to 2^-17 of the spacing; the smallest code is not undercut
    h = np.arange(65536.0)
    for x in np.concatenate([np.random.default_rng(0).uniform(0, 448, 60), np.geomspace(2.0 ** -9, 2.0 ** -5, 30), [448.0]]):
        u = 2.0 ** (np.floor(np.log2(max(x, 2.0 ** -6))) - 3)
        assert abs(L.grid16(np.full(65536, x), h).mean() - x) <= u * 2.0 ** -17 * 1.001
    assert L.grid16(np.array([0.0, 1e-6]), np.array([65535.0, 0.0])).tolist() == [0.0, 2.0 ** -9]


def test_sixteen_bits_keep_a_signed_mean():
    h = np.arange(65536.0)
    assert sorted(L.swapped(h)) == h.tolist()
    for x in np.concatenate([np.random.default_rng(1).uniform(-448, 448, 60), -np.geomspace(2.0 ** -12, 2.0 ** -5, 30), [-448.0]]):
        u = 2.0 ** (np.floor(np.log2(max(abs(x), 2.0 ** -6))) - 3)
        assert abs(L.signed16(np.full(65536, x), L.swapped(h)).mean() - x) <= u * 2.0 ** -17 * 1.001


@pytest.mark.parametrize("b1", [0.95, 0.99, 0.999])
def test_sixteen_bits_follow_exp_avg(b1):
    # the mean is kept at each step; 2048 elements' own noise, a spacing each at most, is under 1 % of their mean
    e, m = L.follow_exp_avg(2500, b1, 2048, seed=3)
    assert abs(m.mean() / e.mean() - 1) <= 0.01


@pytest.mark.parametrize("kind", ["normal", "constant"])
@pytest.mark.parametrize("b2", [0.9, 0.95, 0.99, 0.999, 0.9999])
def test_sixteen_bits_follow_exp_avg_sq(b2, kind):
    v, w = L.follow(1500, b2, kind, 2048, seed=3)
    assert 0.98 <= w.mean() / v.mean() <= 1.02 + 1 / 16  # (L.run_bounds)


def test_the_optimizers_round_stochastically_unless_told_otherwise():
    for kw, want in (({}, 0), (dict(rounding_seed=7), 7), (dict(rounding_seed=None), None)):
        assert pkg.FlatShardAdamW([300], device="cpu", state_bits=8, **kw).rounding_seed == want
        assert pkg.ZeroDataPlane([300], device="cpu", state_bits=8, **kw).opt.rounding_seed == want
        units = pkg.ZeroUnits([[300], [5]], device="cpu", state_bits=8, **kw)
        assert [u.opt.rounding_seed for u in units.units] == [want, want]
    assert pkg.FlatShardAdamW([300], device="cpu").rounding_seed is None
    assert zs.rounding_choice(8, zs.DEFAULT_SEED) == 0 and zs.rounding_choice(32, None) is None
    for bits, seed in ((32, 1), (16, None), (8, "nearest")):
        with pytest.raises(ValueError):
            zs.rounding_choice(bits, seed)
    default = inspect.signature(pkg.TensorListAdamW).parameters["rounding_seed"].default
    assert default == zs.DEFAULT_SEED


@pytest.mark.parametrize("bits", [1, 8, 17, -1])
def test_bad_root_bits_are_refused(bits):
    bad = zs.zero_rounding(1, 0, bits, 0)
    assert call_step8(seed=ctypes.byref(bad)) == zs.ZERO_EINVAL
    assert call_list(seed=ctypes.byref(bad)) == zs.ZERO_EINVAL


def test_reserved_fields_are_refused():
    bad = zs.zero_rounding(1, 0, 16, 1)
    assert call_step8(seed=ctypes.byref(bad)) == zs.ZERO_EINVAL
    assert call_list(seed=ctypes.byref(bad)) == zs.ZERO_EINVAL

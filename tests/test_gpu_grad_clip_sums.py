"""Norms from other ranks' sums alone: zero_sums_norms of a list that has no entries."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg
from fsdp_sharded_mixed_flatparameter_gb300 import zero_shard as zs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("n,groups,ranks", [(1, 1, 1), (7, 3, 2), (1500, 1, 8), (1500, 1100, 3)])
def test_norms_of_sums_without_entries(n, groups, ranks, p):
    rng = np.random.default_rng(n + ranks)
    of = rng.integers(0, groups, n)
    of[0] = groups - 1
    rows = rng.integers(0, 1 << 20, (ranks, n)).astype(np.float64)  # sums of whole numbers are exact
    limits = rng.uniform(1.0, 5000.0, groups)
    plan = zs.zero_grad_plan([1] * n, of, groups, p, "cuda")
    b = pkg.norm_buffers(plan, torch.tensor(limits, device="cuda"))
    bare = pkg.norms_only_list(plan)
    pkg.zero_sums_norms(bare, torch.tensor(rows, device="cuda"), ranks, b)
    joined = rows.max(0) if p == math.inf else rows.sum(0)
    sums = np.zeros(groups)
    (np.maximum if p == math.inf else np.add).at(sums, of, joined)
    whole = joined.max() if p == math.inf else joined.sum()
    norms = [np.sqrt(v) if p == 2 else v for v in (joined, sums, np.array([whole]))]
    assert np.array_equal(b.joined.cpu().numpy(), joined)
    # binary32 norms: 2^-24, and 2^-21 of that for a root
    assert np.allclose(b.norms.cpu().numpy(), np.concatenate(norms), rtol=2.0 ** -24 * (1 + 2.0 ** -21), atol=0)
    r = np.frombuffer(b.results.cpu().numpy().tobytes(), dtype=[("sqnorm", "f8"), ("norm", "f8"), ("coef", "f4"), ("finite", "i4")])
    assert np.array_equal(r["sqnorm"], np.append(sums, whole)) and (r["finite"] == 1).all() and int(b.found) == 0
    assert np.allclose(r["norm"], np.concatenate(norms[1:]), rtol=2.0 ** -52, atol=0)
    coefs = np.minimum(1.0, limits / (norms[1] + 1e-6))
    assert np.allclose(r["coef"], np.append(coefs, 1.0), rtol=2.0 ** -24 * (1 + 2.0 ** -19), atol=0)
    # the other calls need entries
    for call in (lambda: pkg.zero_list_sums(bare, 1.0, b), lambda: pkg.zero_list_norms(bare, 1.0, False, b),
                 lambda: pkg.zero_list_clip(bare, 1.0, b)):
        with pytest.raises(zs.ZeroError, match="d_entries"):
            call()

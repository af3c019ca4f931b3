"""Long chunks whose sums leave the binary32 range, against the formulas in 64 bits.

A list above 2^29 elements has chunks of 131072, of which a lane of a thread adds 512 elements (or a few fewer): a sum is
within 512^2 / 2 x 2^-48 = 4.66e-10, a few 2^-48 of the tree and 2^-37 of squares that lose bits: SUM = 5e-10."""
import math

import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SUM = 5e-10
CHUNK = 131072


@pytest.fixture(scope="module")
def pad():
    """Zeros that make a list long."""
    return torch.zeros(1 << 29, dtype=BF16, device="cuda")


def sums(xs, pad, p):
    c = pkg.GradClip([x.numel() for x in xs] + [pad.numel()], norm_type=p)
    assert c.plan.head.chunk == CHUNK
    c.launch_norms([*xs, pad])
    return c.tensor_sums.tolist()[:-1], c.finish()


def test_a_lanes_worst_magnitudes(pad):
    """Magnitudes whose sum overflows, and whose residuals round the same way at every addition: one of 2^122 for each thread
    and 1023 of 16725503 x 2^74, just below half a unit of its last place.  In a lane of 1024 additions the error is 9.3e-10."""
    x = torch.full((1024, 128), 16725503.0 * 2.0 ** 74)
    x[0] = 2.0 ** 122
    (got,), r = sums([x.flatten().cuda()], pad, 1)
    want = float(128 * (2 ** 122 + 1023 * 16725503 * 2 ** 74))
    assert abs(got - want) <= SUM * want and r.norm == got


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_long_chunks_of_extreme_values(pad, dtype, p):
    g = torch.Generator().manual_seed(5)
    top = torch.finfo(dtype).max
    xs, odd = [], 0
    for scale in (2.0 ** -24 if dtype == F16 else 1e-30, 2.0 ** -14 if dtype == F16 else 2.0 ** -56, top / 8):
        for n in (3 * CHUNK + 77, CHUNK, CHUNK + 20000, 16385):
            v = (torch.randn(n, generator=g, dtype=torch.float64).clamp(-8, 8) * scale).clamp(-top, top).to(dtype)
            odd += 1
            b = torch.zeros(n + 16, dtype=dtype, device="cuda")[odd % 8:]
            b[:n] = v.cuda()
            xs.append(b[:n])
    # one element apart from all others: the sum is its, or nearly
    for alone in (top, 2.0 ** -24 if dtype == F16 else 2.0 ** -133):
        v = torch.full((CHUNK,), 2.0 ** -24 if dtype == F16 else 2.0 ** -133, dtype=dtype, device="cuda")
        v[70001] = alone
        xs.append(v)
    got, r = sums(xs, pad, p)
    want = [float(x.double().abs().max() if p == math.inf else x.double().abs().pow(p).sum()) for x in xs]
    for a, b in zip(got, want):
        assert b > 0 and abs(a - b) <= (SUM + 1e-13) * b  # 1e-13: torch's own sums of up to 393,293 terms, pairwise
    whole = max(want) if p == math.inf else math.fsum(want) ** (1 / p)
    assert abs(r.norm - whole) <= (SUM + 1e-13) * whole and r.finite

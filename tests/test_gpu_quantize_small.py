"""vt_quantize_rows on rows whose scale is among the smallest normal numbers: its
last place is the smallest subnormal then, and half of it is no fp32 number."""
import numpy as np
import pytest
import torch

import frequency_ranked_drafter_gb300 as vt
import serving_ref as ref
from gpu_util import need_cuda

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -149  # the smallest subnormal


def near_halves(rows, d, lo, hi, seed):
    """fp32 rows with scales in [2^lo, 2^hi) and values at the multiples of the
    smallest subnormal next to every half of the scale."""
    rng = np.random.default_rng(seed)
    X = np.zeros((rows, d), dtype=np.float32)
    for r in range(rows):
        top = np.float32(127.0 * 2.0 ** rng.uniform(lo, hi))
        s = np.float64(max(np.float32(top * np.float32(1 / 127)), np.float32(2.0 ** -126)))
        k = rng.integers(-126, 126, d)
        v = np.floor((k + 0.5) * s / UNIT) + rng.integers(-1, 3, d)
        X[r] = (v * UNIT).astype(np.float32)
        X[r, rng.integers(d)] = top
    return X


@pytest.mark.parametrize("lo,hi", [(-128, -126), (-126, -125), (-125.5, -124.5), (-124, -120)])
@pytest.mark.parametrize("d", [64, 2064, 9904])
def test_smallest_scales(lo, hi, d):
    dev = need_cuda()
    X = near_halves(60, d, lo, hi, d)
    q, s = vt.quantize_rows(torch.from_numpy(X).to(dev))
    rq, rs = ref.quantize(X)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_random_patterns_of_small_rows(dtype):
    dev = need_cuda()
    g = torch.Generator().manual_seed(3)
    X = torch.randn(300, 4096, generator=g) * 10.0 ** (-38 + 3 * torch.rand(300, 1, generator=g))
    X = X.to(dtype)
    q, s = vt.quantize_rows(X.to(dev))
    rq, rs = ref.quantize(X.double().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)

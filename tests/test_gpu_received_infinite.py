"""Accumulated weights of queries whose log-sum-exp is infinite or very large: the same in both forms (few
and many rows), and as the formula says."""
import math

import pytest
import torch

import diffusion_decoding_gb300 as dd
from test_gpu_received import check, run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 100])
@pytest.mark.parametrize("scale", [0.125, -0.125, 0.3])
def test_infinite_lse(D, n, scale):
    """exp(x - inf) is 0; a query of -inf saw nothing.  The neighbours count as ever."""
    cache, q, _ = setup(1, 4, 2, 32, D, n, 3, 10)
    lse = run(cache, q, None, 128, scale=scale)[1]
    lse[0, 2, 0] = math.inf
    lse[0, 4, n // 2] = math.inf
    lse[0, 5, n - 1] = -math.inf
    got = check(cache, q, None, 128, lse=lse, scale=scale)
    assert bool(got.isfinite().all())
    lse[:] = math.inf
    got, _ = run(cache, q, None, 128, lse=lse, scale=scale)
    assert bool((got == 0.0).all())


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("scale", [0.125, -0.125])
def test_large_lse(n, scale):
    """Finite, but beyond the largest float once divided by the scale: 0, or infinite where it is negative."""
    cache, q, _ = setup(1, 4, 2, 32, 128, n, 3, 11)
    lse = run(cache, q, None, 128, scale=scale)[1]
    nothing = lse.clone()
    nothing[0, 2, 0] = nothing[0, 3, n // 2] = math.inf
    want = check(cache, q, None, 128, lse=nothing, scale=scale)
    lse[0, 2, 0] = 2e38
    lse[0, 3, n // 2] = 1e30
    got, _ = run(cache, q, None, 128, lse=lse, scale=scale)
    assert torch.equal(got, want)
    lse[0, 1, 0] = -2e38
    got, _ = run(cache, q, None, 128, lse=lse, scale=scale)
    assert bool((got == math.inf).all())

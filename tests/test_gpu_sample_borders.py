"""dllm_sample of numbers beside the borders between tokens: the sums are exact to 2^-36."""
import math

import numpy as np
import pytest
import torch

import diffusion_decoding_gb300 as dd

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, dd.DLLM_BF16), "f32": (torch.float32, dd.DLLM_F32)}


def draw(z, dtype, u, **how):
    """z [R, V] of that dtype, on the GPU."""
    R, V = z.shape
    stats = dd.StatsBuffers(R)
    dd.dllm_sample(z, dd.make_shape(1 if R <= 1024 else R // 64, R if R <= 1024 else 64, V, DT[dtype][1]), None,
                   torch.as_tensor(u, dtype=torch.float32, device="cuda"), stats, **how)
    return stats


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,R", [(3, 100), (3, 1024), (16, 1024), (900, 200), (900, 1024), (40003, 60), (40003, 140),
                                 (40003, 1024)])
@pytest.mark.parametrize("temperature", [0.7, 1.0])
def test_beside_borders(V, R, dtype, temperature):
    """A few heavy tokens a row, and u beside a border between two of them.  A weight is off by 2^-36 of
    itself and half a unit of 2^-42 (equal logits all the same way, so that V of them are off by V 2^-43);
    the sum up to a border and u times the total by as much each, which makes 2^-35 total + V 2^-42, and the
    64-bit sums here add V 2^-52 total.  Numbers closer than that are put two floats further off."""
    rng = np.random.default_rng(1000 * V + R)
    z = np.full((R, V), -math.inf)
    for r in range(R):
        if V > 16:
            z[r] = -[6.0, 12.0, 20.0, 40.0][r % 4] + rng.random(V)  # a bulk of some weight, little or none
        k = min(V, int(rng.integers(2, 17)))
        z[r, rng.choice(V, k, replace=False)] = 1.2 * rng.standard_normal(k)
    z = torch.from_numpy(z).to(DT[dtype][0]).cuda()
    seen, t = z.double().cpu().numpy(), float(np.float32(temperature))
    w = np.exp((seen - seen.max(1, keepdims=True)) / t)
    upto = np.cumsum(w, 1)
    border = upto / upto[:, -1:]
    tol = 2.0 ** -35 + V * 2.0 ** -52 + V * 2.0 ** -42 / upto[:, -1]
    u = np.empty(R, np.float32)
    for r in range(R):
        heavy = np.flatnonzero(w[r] > 2.0 ** -7)
        at = border[r][heavy[rng.integers(len(heavy))]]
        u[r] = at
        for _ in range(int(rng.integers(0, 3))):
            u[r] = np.nextafter(u[r], np.float32(rng.integers(0, 2)))
        while np.abs(border[r] - float(u[r])).min() < tol[r] and 0.0 < u[r] < 1.0:
            u[r] = np.nextafter(np.nextafter(u[r], np.float32(0.0)), np.float32(0.0))
    u = np.minimum(u, np.float32(1.0 - 2.0 ** -24))
    far = np.array([np.abs(border[r] - float(u[r])).min() >= tol[r] for r in range(R)])
    assert far.mean() > 0.9
    want = np.array([np.searchsorted(upto[r], float(u[r]) * upto[r, -1], side="right") for r in range(R)])
    got = draw(z, dtype, u, temperature=temperature).argmax.cpu().numpy()
    wrong = np.flatnonzero(far & (got != want))
    assert wrong.size == 0, [(int(r), int(got[r]), int(want[r]), float(u[r])) for r in wrong[:5]]
    # the same rows split otherwise
    few = z[:7].contiguous()
    assert torch.equal(draw(few, dtype, u[:7], temperature=temperature).argmax.cpu(), torch.from_numpy(got[:7]))

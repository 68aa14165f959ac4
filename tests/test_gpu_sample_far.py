"""dllm_sample of logits far from 1: whatever is finite, tokens and statistics as of any other row."""
import math

import numpy as np
import pytest
import torch

import diffusion_decoding_gb300 as dd
from bounded_ref import sample_row

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, dd.DLLM_BF16), "f32": (torch.float32, dd.DLLM_F32)}


def draw(z, dtype, u, **how):
    """z [R, V] of that dtype, on the GPU."""
    R, V = z.shape
    stats = dd.StatsBuffers(R)
    dd.dllm_sample(z, dd.make_shape(1 if R <= 1024 else R // 64, R if R <= 1024 else 64, V, DT[dtype][1]), None,
                   torch.as_tensor(u, dtype=torch.float32, device="cuda"), stats, **how)
    return stats


def check_statistics(stats, z):
    """row_max exact; conf and lse - row_max, of which nothing is lost however large the logits are."""
    z = z.double().cpu().numpy()
    token, conf, lse, top = (x.cpu().numpy() for x in (stats.argmax, stats.conf, stats.lse, stats.row_max))
    for r in range(z.shape[0]):
        m = z[r].max()
        total = np.exp(z[r] - m).sum()
        below = m - z[r][token[r]]
        assert top[r] == m
        # sums of up to 2^10 additions a lane and the terms' own errors; the exponent z - m by a rounded log2(e)
        p = math.exp(-below) / total
        assert abs(conf[r] - p) <= p * (2.0 ** -12 + below * 2.0 ** -22) + 1e-37, (r, conf[r], p)
        assert abs(lse[r] - (m + math.log(total))) <= 2.0 ** -13 + abs(m) * 2.0 ** -23, (r, lse[r])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e5, 1e7, 1e9, 5e9, 1e10, 1e12, 1e15, 1e20, 1e25, 1e30])
def test_logits_far_from_one(dtype, scale):
    """Any finite logit: rows around +scale, around -scale and of that spread, some maxima tied."""
    g = torch.Generator(device="cuda").manual_seed(int(math.log2(scale)))
    V = 3001
    z = scale * (1.0 + 0.25 * torch.rand(6, V, device="cuda", generator=g))
    z[2:4] *= -1.0
    z[4:] = scale * torch.randn(2, V, device="cuda", generator=g)
    z = z.to(DT[dtype][0])
    for r in (1, 3, 5):
        z[r, 5:2500:499] = z[r].max()
    u = torch.rand(6, device="cuda", generator=g)
    for how in (dict(temperature=1.0), dict(temperature=1.0, top_p=0.5), dict(temperature=2.0 ** -10, top_p=0.5),
                dict(temperature=2.0 ** -10), dict(temperature=1024.0, top_p=0.9), dict(temperature=0.5, top_k=3),
                dict(temperature=0.0)):
        stats = draw(z, dtype, u, **how)
        seen = z.double().cpu().numpy()
        want = [sample_row(seen[r], u[r].item(), **how) for r in range(6)]
        assert stats.argmax.tolist() == want, how
        check_statistics(stats, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cold_and_large(dtype):
    """Temperature 2^-10 and logits of a few million, where their product is far beyond 2^31: ties of the
    maximum and values one step below."""
    V, R = 5000, 8
    z = torch.full((R, V), 1e6, device="cuda")
    for r in range(R):
        z[r, r::997 - r] = 3.0e6
        z[r, 400:4000:701] = 2.96e6 if dtype == "bf16" else 3.0e6 - 0.25
    z = z.to(DT[dtype][0])
    u = (torch.arange(R, device="cuda") + 0.5) / R
    seen = z.double().cpu().numpy()
    for how in (dict(), dict(top_p=0.5), dict(top_p=0.9), dict(min_p=0.5), dict(top_k=2, top_p=0.5)):
        stats = draw(z, dtype, u, temperature=2.0 ** -10, **how)
        want = [sample_row(seen[r], u[r].item(), temperature=2.0 ** -10, **how) for r in range(R)]
        assert stats.argmax.tolist() == want, how
        check_statistics(stats, z)

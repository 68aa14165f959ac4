"""dllm_sample of as many equal maxima as its list of candidates holds, one fewer and one more."""
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2047, 2048, 2049])
@pytest.mark.parametrize("R", [5, 700])
def test_equal_maxima_around_a_full_list(n, dtype, R):
    V = 9001
    g = torch.Generator(device="cuda").manual_seed(n)
    z = torch.randn(R, V, device="cuda", generator=g) - 14.0
    z.scatter_(1, torch.rand(R, V, device="cuda", generator=g).argsort(1)[:, :n], 1.5)
    z = z.to(DT[dtype][0])
    u = torch.rand(R, device="cuda", generator=g)
    for how in (dict(top_p=0.9), dict(top_p=0.25), dict(top_k=n, top_p=0.75), dict(min_p=1.0), dict()):
        stats = draw(z, dtype, u, temperature=1.0, **how)
        for r in range(min(R, 20)):
            assert stats.argmax[r] == sample_row(z[r].double().cpu().numpy(), u[r].item(), temperature=1.0, **how)

"""The 4-bit cache of fp32 rows, code by code: bf16 rows have to be exact (test_gpu_refresh_ops.py); of
fp32 rows a quotient of 24 bits next to a tie may round either way, and nothing else may differ."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
import refresh_ref as ref
from test_gpu_refresh_ops import DEV, entries, gen, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,n,H,D,ps", [(1, 1, 1, 32, 16), (2, 300, 3, 96, 48), (4, 700, 8, 128, 64),
                                        (1, 200, 2, 512, 16)])
@pytest.mark.parametrize("spread", [0.0, 1.0, 20.0])
def test_fp32_rows(B, n, H, D, ps, spread):
    g = gen(n + D)
    c = make_cache(g, B, n, H, D, ps)
    size = torch.exp2(spread * randn(g, B, n, H, D // 32, 1))
    k, v = ((randn(g, B, n, H, D // 32, 32) * size).flatten(-2) for _ in range(2))
    v = v.abs()  # no zero point
    pos = torch.arange(n, dtype=torch.int32, device=DEV).repeat(B, 1)
    dd.dllm_kv4_write(c, k, v, pos)
    for x, codes, params in ((k, c.k_codes, c.k_params), (v, c.v_codes, c.v_params)):
        s, z = (t.repeat_interleave(32, -1) for t in ref.steps(x))
        steps = (entries(c, codes, params, n) - ref.quantised(x)) / s
        # 2^-20: the quotient (at most 15 and half an ulp, 2^-21) and the sum with 1/2
        r = x.double() / s
        tie = ((r.abs() - r.abs().floor()) - 0.5).abs() < 2.0 ** -20
        assert (steps == 0)[~tie].all()
        assert (steps.abs() <= 1)[tie].all()
        assert tie.float().mean() < 1e-4

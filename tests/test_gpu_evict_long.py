"""dllm_kv4_evict of sequences that a cluster's registers do not hold, and of one after the other."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
from test_gpu_evict import ARRAYS, check, make_cache, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_len", [65536, 65537, 70001, 140003])
@pytest.mark.parametrize("values", [0, 7, 5000])
def test_beyond_registers(max_len, values):
    """Weights all different, or of so few values that the border lies among thousands of equals."""
    per = -(-max_len // 64)
    cache = make_cache(2, per, 1, 64, 32, 3)
    w = rand(2, max_len, max_len)
    if values:
        w = torch.round(w * values) / values
    lens = torch.tensor([max_len, max_len - 40], dtype=torch.int32, device="cuda")
    check(cache, w, lens, max_len, max_len // 3, 5, 100, in_place=values == 7, pad=3)


def test_one_after_the_other():
    """Evictions through one workspace with nothing between them, as against each waited for."""
    B, n, rounds = 24, 1024, 12
    a, b = (make_cache(B, n // 64, 2, 64, 64, 5) for _ in range(2))
    w = [rand(B, n, k) for k in range(rounds)]
    budgets = [n - 1 - 60 * k for k in range(rounds)]
    found = []
    for cache, wait in ((a, True), (b, False)):
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        ws = dd.workspace(dd.dllm_kv4_evict_workspace_bytes(cache, B, n))
        slots = torch.empty(rounds, B, n, dtype=torch.int32, device="cuda")
        out = torch.empty(rounds, B, n, device="cuda")
        torch.cuda.synchronize()
        for k in range(rounds):
            dd.dllm_kv4_evict(cache, w[k], lens, n, budgets[k], slots[k], lens, ws, first=3, last=k, weights_out=out[k])
            if wait:
                torch.cuda.synchronize()
        found.append((slots, out, lens))
    for x, y in zip(*found):
        assert torch.equal(x, y)
    for x in ARRAYS:
        assert torch.equal(getattr(a, x), getattr(b, x))

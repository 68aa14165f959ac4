"""Calls of the refresh operators in forms that the other tests do not use: each has to give what the plain
form of the same call gives, bit for bit."""
import pytest
import torch

from test_gpu_refresh_ops import DEV, fill, gen, make_cache, randn, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 40])
def test_attention_masks_without_strides_of_their_own(n):
    g = gen(n)
    B, H, T = 3, 2, 100
    c = make_cache(g, B, T, H, 64, 16)
    fill(g, c, T)
    q = randn(g, B, n, 2 * H, 64).to(torch.bfloat16)
    one = (torch.rand(1, T, generator=g, device=DEV) < 0.7)
    # one mask for all sequences
    for a, b in zip(run(c, q, None, T, mask=one.expand(B, T)), run(c, q, None, T, mask=one.repeat(B, 1))):
        assert torch.equal(a, b)
    # of one sequence, and of one entry, whose strides say nothing
    c1 = make_cache(g, 1, T, H, 64, 16)
    fill(g, c1, T)
    row = torch.empty(T, 1, dtype=torch.bool, device=DEV).copy_(one.t()).t()
    assert row.shape == (1, T) and row.stride(0) < T
    for m in (row, one[0].expand(1, T)):
        for a, b in zip(run(c1, q[:1], None, T, mask=m), run(c1, q[:1], None, T, mask=one)):
            assert torch.equal(a, b)
    wide = torch.zeros(B, 8, dtype=torch.uint8, device=DEV)
    wide[1, 0] = 1
    column = wide[:, ::8]
    assert column.shape == (B, 1) and column.stride(1) == 8
    for a, b in zip(run(c, q, None, 1, mask=column), run(c, q, None, 1, mask=column.contiguous())):
        assert torch.equal(a, b)

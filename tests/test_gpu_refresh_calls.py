"""Calls of the refresh operators in forms that the other tests do not use: each has to give what the plain
form of the same call gives, bit for bit."""
import pytest
import torch

from test_gpu_refresh_ops import DEV, fill, gen, make_cache, randn, run, strided

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


@pytest.mark.parametrize("n,H,G,D,T,layout", [
    (1, 2, 4, 128, 300, "plain"), (1, 2, 4, 128, 5000, "packed"), (4, 3, 4, 64, 900, "plain"),
    (40, 2, 2, 128, 200, "plain"), (64, 2, 4, 128, 5000, "packed"), (100, 1, 3, 256, 1500, "heads_first"),
    (300, 2, 1, 64, 700, "odd")])
def test_attention_in_place(n, H, G, D, T, layout):
    # out may be q: a query's row is read by those CTAs alone that work out its output
    g = gen(n + T)
    B = 2
    c = make_cache(g, B, T, H, D, 32)
    fill(g, c, T)
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    for causal in (False, True):
        want, lse = run(c, q, [T, T - 3], T, causal=causal)
        x = strided(q, layout)
        _, l = run(c, x, [T, T - 3], T, causal=causal, out=x)
        assert torch.equal(x, want) and torch.equal(l, lse)

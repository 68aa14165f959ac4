"""Attention over the 4-bit cache for heads of 256 channels and many rows, and for some rows of many
heads: sizes around the row and entry tiles, against the 64-bit statement (tolerances as for the
other sizes: weights and the result rounded to bf16)."""
import pytest
import torch

import refresh_ref as ref
from test_gpu_refresh_ops import DEV, check_attention, entries, fill, gen, make_cache, randn, run, seen_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,n,H,G,ps,T,lens", [
    (1, 33, 1, 1, 16, 1, None), (2, 64, 1, 2, 64, 64, [64, 63]), (1, 43, 2, 3, 48, 65, None),
    (3, 17, 1, 8, 16, 300, [300, 0, 129]), (2, 128, 2, 1, 256, 1000, [1000, 700]),
    (1, 200, 1, 3, 32, 777, None), (2, 40, 5, 4, 64, 2500, [2500, 100]), (40, 36, 4, 1, 16, 40, None)])
def test_attention_of_wide_heads(B, n, H, G, ps, T, lens, causal, masked):
    D = 256
    g = gen(n + T)
    c = make_cache(g, B, T, H, D, ps)
    k, v = fill(g, c, T)
    q = randn(g, B, n, H * G, D).to(torch.bfloat16)
    mask = None
    if masked:
        mask = (torch.rand(B, T, generator=g, device=DEV) < 0.7).to(torch.uint8)
        mask[0, :min(T, 40)] = 0
    out, lse = run(c, q, lens, T, causal=causal, mask=mask)
    check_attention(out, lse, q, k, v, seen_of(B, n, T, lens or [T] * B, mask, causal, c),
                    D ** -0.5)


@pytest.mark.parametrize("B,n,H,G,D,ps,T,lens", [
    (16, 5, 4, 4, 128, 16, 200, None), (9, 9, 8, 1, 256, 48, 70, None), (33, 8, 2, 3, 128, 64, 65, None),
    (2, 8, 3, 4, 128, 64, 30000, [30000, 17]), (1, 3, 2, 7, 256, 256, 80000, None),
    (1, 3, 2, 7, 256, 16, 500, None), (3, 11, 4, 2, 128, 32, 900, [900, 0, 31])])
def test_attention_of_some_rows(B, n, H, G, D, ps, T, lens):
    """9 to 32 rows: either kernel, by how much there is to do."""
    g = gen(n + T)
    c = make_cache(g, B, T, H, D, ps)
    k, v = fill(g, c, T)
    q = randn(g, B, n, H * G, D).to(torch.bfloat16)
    for causal in (False, True):
        out, lse = run(c, q, lens, T, causal=causal)
        check_attention(out, lse, q, k, v, seen_of(B, n, T, lens or [T] * B, None, causal, c),
                        D ** -0.5)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,n,H,G,ps,T,lens", [
    (1, 33, 1, 1, 16, 1, None), (2, 64, 1, 2, 64, 64, [64, 63]), (1, 43, 2, 3, 48, 65, None),
    (3, 17, 1, 8, 16, 300, [300, 0, 129]), (2, 128, 2, 1, 256, 1000, [1000, 700]),
    (1, 200, 1, 3, 32, 777, None), (20, 5, 5, 4, 64, 500, None)])
def test_attention_of_six_groups(B, n, H, G, ps, T, lens, causal, masked):
    """192 channels: six groups of an entry, three slabs of a tile."""
    D = 192
    g = gen(n + T)
    c = make_cache(g, B, T, H, D, ps)
    k, v = fill(g, c, T)
    q = randn(g, B, n, H * G, D).to(torch.bfloat16)
    mask = None
    if masked:
        mask = (torch.rand(B, T, generator=g, device=DEV) < 0.7).to(torch.uint8)
        mask[0, :min(T, 40)] = 0
    out, lse = run(c, q, lens, T, causal=causal, mask=mask)
    check_attention(out, lse, q, k, v, seen_of(B, n, T, lens or [T] * B, mask, causal, c), D ** -0.5)

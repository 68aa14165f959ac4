"""dllm_attention_kv4_weights against a 64-bit statement of it, entry by entry."""
import math

import pytest
import torch

import diffusion_decoding_gb300 as dd
from bounded_ref import received

pytestmark = pytest.mark.gpu


def setup(B, per, heads, ps, D, n, G, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    cache = dd.Kv4Cache(B * per + 1, heads, ps, D, B, per)
    cache.table.copy_(torch.randperm(B * per + 1, device="cuda", generator=g)[:B * per].view(B, per))
    T = per * ps
    dd.dllm_kv4_write(cache, rand(B, T, heads, D), rand(B, T, heads, D),
                      torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1))
    return cache, (1.3 * rand(B, n, heads * G, D)).to(torch.bfloat16), g


def visible(B, n, T, lens, key_mask, causal):
    j = torch.arange(T, device="cuda")
    last = lens.long()[:, None].expand(B, n)
    if causal:
        last = last - n + 1 + torch.arange(n, device="cuda")
    seen = j < last[..., None]
    return seen if key_mask is None else seen & (key_mask[:, :T] != 0)[:, None]


def run(cache, q, lens, T, key_mask=None, causal=False, prior=None, keep=1.0, lse=None, scale=None, weights=None):
    B, n, H, D = q.shape
    if lse is None:
        out, lse = torch.empty_like(q), torch.empty(B, H, n, device="cuda")
        ws = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(cache, B, n, H, T))
        dd.dllm_attention_kv4(q, cache, lens, T, out, ws, lse=lse, key_mask=key_mask, causal=causal, scale=scale)
    if weights is None:
        weights = torch.full((B, T), 7.0, device="cuda")
    ws = dd.workspace(dd.dllm_attention_kv4_weights_workspace_bytes(cache, B, n, H, T))
    dd.dllm_attention_kv4_weights(q, cache, lens, T, lse, weights, ws, prior=prior, keep=keep, key_mask=key_mask,
                                  causal=causal, scale=scale)
    assert dd.dllm_get_status(ws) == dd.DLLM_OK
    return weights, lse


def check(cache, q, lens, T, key_mask=None, causal=False, prior=None, keep=1.0, scale=None, lse=None):
    B, n, H, D = q.shape
    held = None if prior is None else prior.clone()
    got, lse = run(cache, q, lens, T, key_mask, causal, prior, keep, lse=lse, scale=scale)
    full = torch.full((B,), T, device="cuda") if lens is None else lens.clamp(0, T)
    scale = D ** -0.5 if scale is None else scale
    want, size = received(q, cache, full, lse, visible(B, n, T, full, key_mask, causal), scale, keep, held)
    there = torch.arange(T, device="cuda") < full[:, None]
    assert bool((got[~there] == 7.0).all())
    # a term's exponent: the products' sum (2^-20 of their magnitudes' sum), the rounding of lse and of
    # the exponent itself; then one addition a term and one of the prior
    top = float(lse[lse.isfinite()].abs().max()) if bool(lse.isfinite().any()) else 0.0
    # The terms' errors are relative to their sum, which is want - keep * prior and not want: with a negative
    # keep the two may cancel.  keep * prior + sum is one fused operation, off by half an ulp of itself.
    gain = want if prior is None else want - float(torch.tensor(keep)) * held[:, :T].double()
    tol = gain.abs() * (2.0 ** -20 * size + 2.0 ** -22 * (top + size) + 2.0 ** -21 + n * H * 2.0 ** -24) \
        + want.abs() * 2.0 ** -24 + 1e-37
    bad = there & ~((got.double() - want).abs() <= tol) & ~(got.isnan() & want.isnan())
    assert not bool(bad.any()), (got[bad][:5], want[bad][:5])
    return got


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("n,G,heads", [(1, 1, 1), (1, 7, 2), (3, 2, 3), (40, 4, 2), (130, 3, 1), (70, 8, 1)])
def test_shapes(D, n, G, heads):
    cache, q, _ = setup(2, 9, heads, 32, D, n, G, D + n)
    lens = torch.tensor([9 * 32 - 5, 150], dtype=torch.int32, device="cuda")
    check(cache, q, lens, 9 * 32 - 2)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("n", [1, 33, 200])
def test_lengths(T, n):
    cache, q, _ = setup(1, -(-T // 48), 2, 48, 64, n, 2, T)
    check(cache, q, None, T)


@pytest.mark.parametrize("D,n,G", [(64, 20, 2), (128, 64, 4), (128, 5, 3), (256, 90, 2), (192, 50, 3)])
def test_causal_and_masked(D, n, G):
    cache, q, g = setup(4, 12, 2, 16, D, n, G, n)
    T = 190
    lens = torch.tensor([190, n, max(1, n // 2), 0], dtype=torch.int32, device="cuda")
    key_mask = (torch.rand(4, T, device="cuda", generator=g) < 0.6).to(torch.uint8)
    key_mask[0, 16:64] = 0
    check(cache, q, lens, T, causal=True)
    check(cache, q, lens, T, key_mask=key_mask)
    check(cache, q, lens, T, key_mask=key_mask, causal=True)
    key_mask[1] = 0  # a sequence that sees nothing
    check(cache, q, lens, T, key_mask=key_mask, causal=True)
    one = key_mask[:1].expand(4, T)
    check(cache, q, lens, T, key_mask=one)


@pytest.mark.parametrize("n", [1, 60])
def test_prior(n):
    cache, q, g = setup(2, 6, 2, 32, 128, n, 4, 5)
    lens = torch.tensor([180, 77], dtype=torch.int32, device="cuda")
    prior = torch.rand(2, 200, device="cuda", generator=g)[:, :192]
    for keep in (1.0, 0.9, 0.0, -0.5):
        check(cache, q, lens, 190, prior=prior, keep=keep)
    # in place: the same numbers, and nothing behind the sequence
    want, lse = run(cache, q, lens, 190, prior=prior, keep=0.75)
    both = prior.clone()
    run(cache, q, lens, 190, prior=both, keep=0.75, lse=lse, weights=both)
    there = torch.arange(190, device="cuda") < lens[:, None]
    assert torch.equal(both[:, :190][there], want[there])
    assert torch.equal(both[:, :190][~there], prior[:, :190][~there])


def test_sum_of_weights():
    """Every query that sees something gives 1 in all."""
    cache, q, _ = setup(2, 10, 3, 64, 128, 70, 2, 6)
    lens = torch.tensor([640, 333], dtype=torch.int32, device="cuda")
    got = run(cache, q, lens, 640)[0]
    there = torch.arange(640, device="cuda") < lens[:, None]
    total = torch.where(there, got, torch.zeros_like(got)).double().sum(1)
    # lse is 2^-20 of its scale off, about 10 here, and the sums of terms 2^-16
    assert float((total / (70 * 6) - 1).abs().max()) < 2e-4


@pytest.mark.parametrize("n", [1, 80])
def test_strides(n):
    cache, q, g = setup(3, 6, 2, 32, 64, n, 2, 7)
    wide = torch.zeros(3, n, 9, 67, device="cuda", dtype=torch.bfloat16)
    wide[:, :, 2:6, 1:65] = q
    lens = torch.tensor([192, 60, 100], dtype=torch.int32, device="cuda")
    a = check(cache, wide[:, :, 2:6, 1:65], lens, 192)
    b = check(cache, q, lens, 192)
    turned = q.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    c = check(cache, turned, lens, 192)
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("n", [1, 100])
def test_nan(n):
    """A NaN among the keys reaches its own entry, one in lse what its query sees; hidden ones nothing."""
    cache, q, _ = setup(2, 4, 2, 32, 128, n, 2, 8)
    T = 128
    lens = torch.tensor([128, 60], dtype=torch.int32, device="cuda")
    key_mask = torch.ones(2, T, dtype=torch.uint8, device="cuda")
    key_mask[0, 40] = 0
    clean, lse = run(cache, q, lens, T, key_mask)
    page, params = cache.table.long(), cache.k_params
    params[page[0, 40 // 32], 1, 40 % 32, 2] = 0x7FE0       # hidden by the mask
    params[page[1, 70 // 32], 0, 70 % 32, 0] = 0x7FE0       # behind the sequence
    params[page[0, 9 // 32], 0, 9 % 32, 1] = 0x7FE0         # seen
    got, _ = run(cache, q, lens, T, key_mask, lse=lse)
    where = torch.zeros(2, T, dtype=torch.bool, device="cuda")
    where[0, 9] = True
    assert torch.equal(got.isnan(), where)
    assert torch.equal(got[~where], clean[~where])
    lse[1, 2, n - 1] = math.nan
    got, _ = run(cache, q, lens, T, key_mask, lse=lse)
    assert bool(got[1, :60].isnan().all()) and not bool(got[1, 60:].isnan().any())


@pytest.mark.parametrize("n", [1, 90])
def test_absent_pages(n):
    cache, q, _ = setup(2, 6, 2, 32, 128, n, 2, 9)
    cache.table[0, 2] = -1
    cache.table[1, 0] = cache.pages
    cache.table[1, 5] = 1 << 30
    check(cache, q, None, 190)


@pytest.mark.parametrize("n", [1, 100])
def test_lse_of_nothing(n):
    """A query whose lse is -inf adds nothing, though its neighbours do."""
    cache, q, _ = setup(1, 4, 2, 32, 64, n, 3, 10)
    lse = run(cache, q, None, 128)[1]
    lse[0, 1, 0] = -math.inf
    lse[0, 5, n // 2] = -math.inf
    check(cache, q, None, 128, lse=lse)


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.02])
def test_scales(scale):
    cache, q, _ = setup(1, 4, 2, 32, 64, 70, 2, 11)
    check(cache, q, None, 100, scale=scale)


@pytest.mark.parametrize("n,B", [(1, 40), (2, 3), (64, 20), (300, 2)])
def test_larger_and_repeated(n, B):
    """Several waves of work; the same call again agrees bit for bit, captured or on another stream."""
    cache, q, g = setup(B, 20, 2, 64, 128, n, 4, 12)
    lens = torch.randint(1, 1281, (B,), device="cuda", generator=g).to(torch.int32)
    first = check(cache, q, lens, 1280, causal=n == 300)
    H = q.shape[2]
    again, lse = run(cache, q, lens, 1280, causal=n == 300)
    assert torch.equal(first, again)
    ws = dd.workspace(dd.dllm_attention_kv4_weights_workspace_bytes(cache, B, n, H, 1280))
    out = torch.full((B, 1280), 7.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dd.dllm_attention_kv4_weights(q, cache, lens, 1280, lse, out, ws, causal=n == 300)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("n", [8, 9, 16, 17, 32, 33])
def test_few_and_many_rows(D, n):
    """Rows around the numbers at which one kernel takes over from the other."""
    cache, q, _ = setup(2, 6, 2, 48, D, n, 1, n)
    lens = torch.tensor([257, 255], dtype=torch.int32, device="cuda")
    check(cache, q, lens, 280, causal=n % 2 == 0)


@pytest.mark.parametrize("scale", [1e-7, -1e-7])
def test_scales_beyond_the_many_rows_form(scale):
    cache, q, _ = setup(1, 8, 2, 64, 128, 50, 2, 13)
    check(cache, q, None, 500, scale=scale, causal=True)

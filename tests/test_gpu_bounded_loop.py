"""Sampling, accumulated weights and eviction as a decode loop runs them together
(diffusion_decoding_gb300/refresh.py)."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
import refresh_ref as ref
from bounded_ref import evict

pytestmark = pytest.mark.gpu

B, P, L, KV, D = 2, 96, 32, 2, 64


def values(layer, T=P + L):
    k, v = (torch.empty(B, T, KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dd.dllm_kv4_read(layer.cache, k, v)
    return k, v


def test_greedy_sampling_is_the_argmax_loop():
    """A temperature so low that only the most probable token is left draws what the loop without one takes,
    unless logits tie."""
    from diffusion_decoding_gb300.refresh import decode_block
    a = decode_block(iterations=3)
    b = decode_block(iterations=3, temperature=2.0 ** -10)
    assert torch.equal(a[2], b[2]) and torch.equal(a[0].masked, b[0].masked)


def test_bounded_loop_keeps_its_entries_current():
    """Every position that still has an entry finds there what it finds in a loop without a budget whose
    tokens are the same; at most `budget` entries are left, the block's among them."""
    from diffusion_decoding_gb300.refresh import decode_block
    how = dict(temperature=0.8, top_k=50, top_p=0.95)
    # before the first iteration is over the budget has not touched the logits: the same draws
    _, whole, tokens, _ = decode_block(iterations=1, **how)
    _, cut, tokens_cut, _ = decode_block(iterations=1, budget=80, **how)
    assert torch.equal(tokens, tokens_cut)
    assert cut.lens.tolist() == [80, 80]
    k0, v0 = values(whole)
    k1, v1 = values(cut)
    for b in range(B):
        at = cut.entry[b]
        left = (at >= 0).nonzero().flatten()
        assert left.numel() == 80 and sorted(at[left].tolist()) == list(range(80))
        assert at[P:].tolist() == list(range(L))  # the block's entries stay in front
        assert torch.equal(k1[b, at[left].long()], k0[b, left])
        assert torch.equal(v1[b, at[left].long()], v0[b, left])


def test_bounded_loop_repeats():
    from diffusion_decoding_gb300.refresh import decode_block
    how = dict(iterations=5, temperature=1.0, top_p=0.9, budget=64)
    _, a, ta, _ = decode_block(**how)
    _, b, tb, _ = decode_block(**how)
    assert torch.equal(ta, tb) and torch.equal(a.entry, b.entry) and torch.equal(a.weights, b.weights)
    assert a.lens.tolist() == [64, 64]
    assert bool((a.weights[:, 64:] == 0).all()) and bool((a.weights[:, :64] > 0).any(1).all())


@pytest.mark.parametrize("n,causal", [(1, False), (40, False), (40, True)])
def test_layer_weighs_and_evicts(n, causal):
    """attend -> weigh -> evict -> attend: the entries left are those of largest weight, and attention over
    them is attention over the entries that were kept."""
    from diffusion_decoding_gb300.refresh import CachedAttention
    dev, T, Hq = torch.device("cuda"), 150, 8
    g = torch.Generator(device=dev).manual_seed(n)
    layer = CachedAttention(B, Hq, KV, D, T, max(n, T), page_size=16)
    rows = torch.randn(B, T, Hq + 2 * KV, D, device=dev, generator=g).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)
    layer.write(rows, pos)
    asked = torch.randn(B, n, Hq + 2 * KV, D, device=dev, generator=g).to(torch.bfloat16)
    lens = torch.tensor([T, T - 60], dtype=torch.int32, device=dev)
    out, lse = torch.empty(B, n, Hq, D, dtype=torch.bfloat16, device=dev), torch.empty(B, Hq, n, device=dev)
    layer.attend(asked, lens, out, causal=causal, lse=lse)
    weights = torch.zeros(B, T, device=dev)
    layer.weigh(asked, lens, lse, weights, causal=causal)
    held, before = weights.clone(), lens.tolist()
    k0, v0 = values(layer, T)
    slots = torch.empty(B, T, dtype=torch.int32, device=dev)
    layer.evict(weights, lens, 70, slots, first=3, last=5)
    assert lens.tolist() == [70, 70]
    k1, v1 = values(layer, T)
    for b in range(B):
        want, _ = evict(held[b].double().tolist(), before[b], 70, 3, 5)
        assert slots[b].tolist() == want + [-1] * (T - before[b])
        left = (slots[b] >= 0).nonzero().flatten()
        at = slots[b, left].long()
        assert torch.equal(k1[b, at], k0[b, left]) and torch.equal(v1[b, at], v0[b, left])
        assert torch.equal(weights[b, at], held[b, left]) and bool((weights[b, 70:] == 0).all())
    layer.attend(asked, lens, out)
    seen = torch.ones(B, n, 70, dtype=torch.bool, device=dev)
    o, _, mag, _ = ref.attention(layer.split(asked)[0], k1[:, :70], v1[:, :70], seen, D ** -0.5)
    # weights rounded to bf16 and the output too, and as much again for the scores and the sums
    assert ((out.double() - o).abs() <= 2.0 ** -8 * 1.03 * (mag + o.abs()) + 1e-30).all()
    assert dd.dllm_get_status(layer.weigh_ws) == dd.DLLM_OK

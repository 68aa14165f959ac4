"""The refresh operators put together (diffusion_decoding_gb300/refresh.py): a layer's calls against
the 64-bit statements, and the decode loop's cache against its tokens."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
import refresh_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,Hq,Hk,D", [(1, 4, 2, 128), (9, 3, 1, 64), (40, 8, 2, 128)])
def test_layer_write_and_attend(n, Hq, Hk, D):
    from diffusion_decoding_gb300.refresh import CachedAttention
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(n)
    B, T = 2, 150
    wq, wk = (torch.rand(D, device=dev, generator=g).to(torch.bfloat16) + 0.5 for _ in range(2))
    layer = CachedAttention(B, Hq, Hk, D, T, max(n, T), page_size=16, q_weight=wq, k_weight=wk)
    first = torch.randn(B, T, Hq + 2 * Hk, D, device=dev, generator=g).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)
    before = first.clone()
    layer.write(first, pos)
    # queries and keys: 4e-6 of the pair for the fp32 arithmetic and half an ulp of bf16
    for part, w in ((0, wq), (1, wk)):
        x, y = layer.split(before)[part], layer.split(first)[part]
        o, size = ref.norm_rope(x, pos, ref.frequencies(D, 10000.0), w, 1e-6, False)
        assert ((y.double() - o).abs() <= 4e-6 * size + 2.0 ** -8 * o.abs() + 1e-30).all()
    # n entries anew, with one row skipped, then the queries of those rows over the whole cache
    again = torch.randn(B, n, Hq + 2 * Hk, D, device=dev, generator=g).to(torch.bfloat16)
    at = torch.stack([torch.randperm(T, device=dev, generator=g)[:n] for _ in range(B)])
    at = at.to(torch.int32)
    at[1, 0] = -1
    layer.write(again, at)
    want = {}
    for part in (1, 2):
        x = layer.split(first)[part].clone()
        for b in range(B):
            ok = at[b] >= 0
            x[b, at[b, ok].long()] = layer.split(again)[part][b, ok]
        want[part] = ref.quantised(x)
    k, v = (torch.empty(B, T, Hk, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    dd.dllm_kv4_read(layer.cache, k, v)
    assert torch.equal(k.double(), want[1]) and torch.equal(v.double(), want[2])
    out = torch.empty(B, n, Hq, D, dtype=torch.bfloat16, device=dev)
    lens = torch.tensor([T, T - 60], dtype=torch.int32, device=dev)
    layer.attend(again, lens, out)
    seen = (torch.arange(T, device=dev)[None, :] < lens[:, None])[:, None].expand(B, n, T)
    o, _, mag, _ = ref.attention(layer.split(again)[0], k, v, seen, D ** -0.5)
    # weights rounded to bf16 and the output too: 2^-9 of each term's size and of the result, and
    # as much again for the scores' rounding and the sums
    assert ((out.double() - o).abs() <= 2.0 ** -8 * 1.03 * (mag + o.abs()) + 1e-30).all()
    assert dd.dllm_get_status(layer.ws) == dd.DLLM_OK


def test_decode_loop_keeps_the_cache_current():
    """Entries follow their tokens: those of committed positions are written anew, others stay."""
    from diffusion_decoding_gb300.refresh import decode_block
    state, layer, tokens, count = decode_block(iterations=3)
    assert int(state.masked.sum()) < state.masked.numel()
    k0, v0 = (torch.empty(2, 128, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dd.dllm_kv4_read(layer.cache, k0, v0)
    # a second run agrees bit for bit
    state1, layer1, tokens1, _ = decode_block(iterations=3)
    k1, v1 = torch.empty_like(k0), torch.empty_like(v0)
    dd.dllm_kv4_read(layer1.cache, k1, v1)
    assert torch.equal(tokens, tokens1) and torch.equal(k0, k1) and torch.equal(v0, v1)
    # a layer's entry is a function of its token and position alone: it changes where the token did
    state2, layer2, tokens2, _ = decode_block(iterations=0)
    k2, v2 = torch.empty_like(k0), torch.empty_like(v0)
    dd.dllm_kv4_read(layer2.cache, k2, v2)
    changed = (v0 != v2).flatten(2).any(-1)
    assert torch.equal(changed, tokens != tokens2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,Hq,Hk,D", [(1, 1, 1, 1, 64), (2, 7, 1, 1, 128), (3, 5, 2, 1, 64),
                                         (1, 13, 1, 1, 32), (2, 9, 3, 2, 32), (1, 6, 1, 1, 256)])
def test_few_heads_share_a_warp(dtype, B, n, Hq, Hk, D):
    """Tokens share a warp where heads are few: skipped tokens, and ends that do not fill one."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(n + D)
    q, k, v = (torch.randn(B, n, h, D, device=dev, generator=g).to(dtype) for h in (Hq, Hk, Hk))
    pos = torch.stack([torch.randperm(60, device=dev, generator=g)[:n] for _ in range(B)])
    pos = pos.to(torch.int32)
    pos[0, n // 2] = -1
    live = pos >= 0
    phases = torch.empty(D // 2, dtype=torch.int64, device=dev)
    dd.dllm_rope_phases(D, phases)
    qo, ko = (torch.full_like(x, 3.0) for x in (q, k))
    dd.dllm_qk_norm_rope(q, k, qo, ko, pos, phases)
    for x, y in ((q, qo), (k, ko)):
        o, size = ref.norm_rope(x, pos, ref.frequencies(D, 10000.0), None, 1e-6, False)
        tol = 4e-6 * size + (2.0 ** -8 * o.abs() if dtype == torch.bfloat16 else 0) + 1e-30
        assert ((y.double() - o).abs() <= tol)[live].all()
        assert (y[~live] == 3.0).all()
    cache = dd.Kv4Cache(4 * B, Hk, 16, D, B, 4)
    cache.table.copy_(torch.arange(4 * B, dtype=torch.int32, device=dev).view(B, 4))
    for t in (cache.k_codes, cache.v_codes, cache.k_params, cache.v_params):
        t.zero_()
    dd.dllm_kv4_write(cache, k, v, pos)
    kr, vr = (torch.full_like(k, 5.0) for _ in range(2))
    dd.dllm_kv4_read(cache, kr, vr, pos)
    for x, y in ((k, kr), (v, vr)):
        if dtype == torch.bfloat16:
            assert torch.equal(y[live].double(), ref.quantised(x)[live])
        else:  # a quotient next to a tie may round either way: within half a step, a step in all
            s, _ = ref.steps(x)
            half = s.repeat_interleave(32, -1).view_as(x)
            assert ((y.double() - x.double()).abs() <= 0.5001 * half + 1e-30)[live].all()
        assert (y[~live] == 0).all()
    everything = torch.empty(B, 64, Hk, D, dtype=dtype, device=dev)
    dd.dllm_kv4_read(cache, everything, torch.empty_like(everything))
    untouched = torch.ones(B, 64, dtype=torch.bool, device=dev)
    for b in range(B):
        untouched[b, pos[b, live[b]].long()] = False
    assert (everything[untouched] == 0).all()

"""The operators behind the KV refresh put together: one attention layer whose keys and values lie in
a 4-bit cache, and a small decode loop that runs it (dInfer explainer, KV-cache manager).

    python -m diffusion_decoding_gb300.refresh [iterations [temperature [budget]]]

decodes one block per sequence with a toy decoder of a single attention layer and random weights
(nothing is trained: it shows the calls and their order).  The prompt's keys and values are
written once; then each iteration
  1. projects the block's rows, attends over the cached prompt and block, and takes the logits,
  2. commits positions (dllm_commit_threshold),
  3. lists the entries around them (dllm_kv_refresh_mask) and recomputes only those.
With a temperature the tokens are sampled (dllm_sample) instead of the most probable ones; with a budget
the attention that every entry receives is added up (dllm_attention_kv4_weights) and each sequence's
cache is cut to its `budget` entries of largest weight (dllm_kv4_evict).
"""
import sys

import torch

import diffusion_decoding_gb300 as dd


class CachedAttention:
    """One attention layer: norm of each head, rotation, the 4-bit cache and attention over it.

    Rows come as one projection [B, n, q_heads + 2 * kv_heads, head_dim] bf16 (queries, keys,
    values); the calls take its slices where they lie.  Pages are given to the sequences in
    order here; a server would write its own page ids into `cache.table`."""

    def __init__(self, B: int, q_heads: int, kv_heads: int, head_dim: int, max_len: int,
                 max_rows: int, page_size: int = 64, rope_base: float = 10000.0,
                 q_weight=None, k_weight=None, eps: float = 1e-6, device=None):
        dev = device or torch.device("cuda")
        self.q_heads, self.kv_heads, self.max_len = q_heads, kv_heads, max_len
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        per = -(-max_len // page_size)
        self.cache = dd.Kv4Cache(B * per, kv_heads, page_size, head_dim, B, per, dev)
        self.cache.table.copy_(torch.arange(B * per, dtype=torch.int32, device=dev).view(B, per))
        self.phases = torch.empty(head_dim // 2, dtype=torch.int64, device=dev)
        dd.dllm_rope_phases(head_dim, self.phases, base=rope_base)
        self.ws = dd.workspace(max(dd.dllm_attention_kv4_workspace_bytes(
            self.cache, B, n, q_heads, max_len) for n in (1, max_rows)), dev)
        self.weigh_ws = self.evict_ws = None  # made when first used
        self.max_rows = max_rows

    def split(self, qkv):
        """The queries, keys and values of a projection (views)."""
        a, b = self.q_heads, self.q_heads + self.kv_heads
        return qkv[:, :, :a], qkv[:, :, a:b], qkv[:, :, b:]

    def write(self, qkv, pos, stream=None, entries=None) -> None:
        """Store the rows' keys and values as the entries pos ([B, >= n] int32, < 0: skipped; as
        dllm_kv_refresh_mask lists them), or as `entries` where these are not the positions.  Queries and
        keys are turned in place on the way."""
        q, k, v = self.split(qkv)
        dd.dllm_qk_norm_rope(q, k, q, k, pos, self.phases, self.q_weight, self.k_weight, self.eps,
                             stream=stream)
        dd.dllm_kv4_write(self.cache, k, v, pos if entries is None else entries, stream=stream)

    def attend(self, qkv, lens, out, causal: bool = False, lse=None, stream=None) -> None:
        """out [B, n, q_heads, head_dim]: attention of turned queries over the first lens[b] entries
        (None: max_len)."""
        dd.dllm_attention_kv4(self.split(qkv)[0], self.cache, lens, self.max_len, out, self.ws,
                              lse=lse, causal=causal, stream=stream)

    def weigh(self, qkv, lens, lse, weights, keep: float = 1.0, causal: bool = False, stream=None) -> None:
        """weights ([B, max_len] fp32) = keep * weights + the attention that each entry received in the
        `attend` call that wrote lse."""
        q = self.split(qkv)[0]
        if self.weigh_ws is None:
            self.weigh_ws = dd.workspace(max(dd.dllm_attention_kv4_weights_workspace_bytes(
                self.cache, q.shape[0], n, self.q_heads, self.max_len) for n in (1, self.max_rows)), q.device)
        dd.dllm_attention_kv4_weights(q, self.cache, lens, self.max_len, lse, weights, self.weigh_ws,
                                      prior=weights, keep=keep, causal=causal, stream=stream)

    def evict(self, weights, lens, budget: int, slots, first: int = 0, last: int = 0, stream=None) -> None:
        """Cut every sequence to `budget` entries; lens and weights are updated, slots ([B, max_len]
        int32) tells where each entry went."""
        if self.evict_ws is None:
            self.evict_ws = dd.workspace(dd.dllm_kv4_evict_workspace_bytes(
                self.cache, self.cache.B, self.max_len), weights.device)
        dd.dllm_kv4_evict(self.cache, weights, lens, self.max_len, budget, slots, lens, self.evict_ws,
                          first=first, last=last, weights_out=weights, stream=stream)

    def turn_queries(self, qkv, pos, stream=None) -> None:
        """Norm and rotation of the queries alone, in place (their keys are cached already)."""
        q = self.split(qkv)[0]
        dd.dllm_qk_norm_rope(q, None, q, None, pos, self.phases, self.q_weight, None, self.eps,
                             stream=stream)


def decode_block(iterations: int = 4, B: int = 2, P: int = 96, L: int = 32, V: int = 4096,
                 q_heads: int = 8, kv_heads: int = 2, head_dim: int = 64, window: int = 2,
                 tau: float = 0.02, seed: int = 1, temperature: float = 0.0, top_k: int = 0,
                 top_p: float = 1.0, min_p: float = 0.0, budget: int = 0, keep: float = 0.9):
    """The toy decode loop; returns the block state, the layer, the tokens and the last iteration's counts
    of refreshed entries ([B]).  temperature > 0: sampled tokens (with the filters); budget > 0: at most
    that many cache entries per sequence (the block's own L among them), the others' weights fading by
    `keep` an iteration.  The layer's `lens` are the entries left, its `entry` where each position's is."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    bf16 = torch.bfloat16
    d, T, heads = q_heads * head_dim, P + L, q_heads + 2 * kv_heads
    embed = torch.randn(V + 1, d, device=dev, generator=g).to(bf16)  # row V: the mask token
    to_qkv = (torch.randn(d, heads * head_dim, device=dev, generator=g) * d ** -0.5).to(bf16)
    tokens = torch.randint(0, V, (B, T), device=dev, generator=g)
    tokens[:, P:] = V
    layer = CachedAttention(B, q_heads, kv_heads, head_dim, T, max(P, L))
    everywhere = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)
    block = everywhere[:, P:]
    lens = torch.full((B,), T, dtype=torch.int32, device=dev)

    def project(rows):
        return (embed[rows] @ to_qkv).view(*rows.shape, heads, head_dim)

    shape = dd.make_shape(B, L, V, dd.DLLM_BF16)
    state, stats = dd.BlockState(B, L), dd.StatsBuffers(B * L)
    ws = dd.workspace(dd.dllm_workspace_bytes(shape))
    refresh = torch.empty(B * T, dtype=torch.uint8, device=dev)
    idx = torch.empty(B, T, dtype=torch.int32, device=dev)
    count = torch.empty(B, dtype=torch.int32, device=dev)
    out = torch.empty(B, L, q_heads, head_dim, dtype=bf16, device=dev)
    # The entry of each position, -1 once it is dropped.  With a budget the block's entries come first:
    # entries from the new length on move into the places of dropped ones, the first `first` never do.
    entry, lse, weights, slots = None, None, None, None
    if budget > 0:
        entry = torch.cat((everywhere[:, :P] + L, everywhere[:, P:] - P), 1).contiguous()
        lse = torch.empty(B, q_heads, L, device=dev)
        weights = torch.zeros(B, T, device=dev)
        slots = torch.empty(B, T, dtype=torch.int32, device=dev)
    layer.lens = lens

    layer.write(project(tokens), everywhere, entries=entry)  # the prompt and the block of mask tokens
    for _ in range(iterations):
        qkv = project(tokens[:, P:])
        layer.turn_queries(qkv, block)
        layer.attend(qkv, lens, out, lse=lse)
        if budget > 0:
            layer.weigh(qkv, lens, lse, weights, keep)
            layer.evict(weights, lens, budget, slots, first=min(L, budget))
            entry = torch.where(entry >= 0, slots.gather(1, entry.clamp(min=0).long()), entry)
        hidden = embed[tokens[:, P:]] + out.view(B, L, d)
        logits = (hidden.float() * d ** -0.5 @ embed[:V].float().t()).to(bf16).contiguous()
        if temperature > 0.0:
            uniform = torch.rand(B * L, device=dev, generator=g)
            dd.dllm_sample(logits, shape, state.masked, uniform, stats, temperature, top_k, top_p, min_p)
            dd.dllm_commit_threshold(None, shape, stats, state, tau, -1, ws)
        else:
            dd.dllm_commit_threshold(logits, shape, stats, state, tau, -1, ws)
        found = state.tokens.view(B, L).long()
        tokens[:, P:] = torch.where(found >= 0, found, torch.full_like(found, V))
        dd.dllm_kv_refresh_mask(state, P, window, refresh, idx, count)
        # the listed entries (padded with -1, which the calls skip)
        listed = idx.clamp(min=0).long()
        layer.write(project(tokens.gather(1, listed)), idx,
                    entries=None if entry is None else torch.where(idx >= 0, entry.gather(1, listed), idx))
    layer.entry, layer.weights = entry, weights
    for w in (layer.ws, layer.weigh_ws):
        if w is not None and dd.dllm_get_status(w) != dd.DLLM_OK:
            raise RuntimeError("attention reported a fault")
    return state, layer, tokens, count


def main(argv) -> None:
    state, layer, tokens, count = decode_block(
        int(argv[0]) if argv else 4, temperature=float(argv[1]) if len(argv) > 1 else 0.0,
        budget=int(argv[2]) if len(argv) > 2 else 0)
    left = int(state.masked.sum())
    print(f"{state.masked.numel() - left} of {state.masked.numel()} positions committed; entries "
          f"refreshed last, by sequence: {count.tolist()}; entries cached: {layer.lens.tolist()}")


if __name__ == "__main__":
    main(sys.argv[1:])

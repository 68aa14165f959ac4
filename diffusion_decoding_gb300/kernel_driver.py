"""Run one kernel family of the decode step a fixed number of times, for external profilers.

    python -m diffusion_decoding_gb300.kernel_driver {stats|probs|gemm|step|fused} [n [B L]]
    python -m diffusion_decoding_gb300.kernel_driver {rope|cache|token|block|piece} [n]
    python -m diffusion_decoding_gb300.kernel_driver {whole|nucleus|top_k} [n [B L]]
    python -m diffusion_decoding_gb300.kernel_driver {token_weights|block_weights|piece_weights|evict} [n]

The inputs have the smoothing-step sizes (B=16, L=64, V=126464 bf16 logits, d=2048 embedding
table; about 0.8 GB on the device), so every launch reads more than the L2 holds; `stats`
takes another block shape as B and L (every position masked, as in a loop's first
iteration).  Nothing is timed here: a profiler (ncu) attaches to the launches.  `stats` runs
the fused statistics + threshold commit; `probs` the probability rows; `gemm` the smoothing
GEMM (after one probability pass); `step` the whole step (commit, probabilities, GEMM, KV
refresh) through the separate calls; `fused` the whole step through the single-read call.

The second line runs the operators of the KV refresh (below 0.5 GB on the device): `rope` norm and
rotation of 16384 tokens, `cache` write and read of 32768 entries, `token` attention of single tokens
over 32 sequences of 8192 entries, `block` of 64-token blocks over 16 of 4160, `piece` of 1024 tokens of
a prompt over 2 of 16384.

The third line draws tokens of a block: `whole` from the distribution at temperature 0.7, `nucleus` with
top_p 0.9 too, `top_k` with top_k 50 at temperature 1.  The fourth runs the accumulated weights of the
second line's three calls of attention, and `evict` cuts 32 sequences of 8192 entries to 4096.
"""
import sys

import torch

import diffusion_decoding_gb300 as dd

B_, L_, V, D = 16, 64, 126464, 2048
PREFIX, WINDOW, TAU = 1024, 4, 0.9


def refresh_operator(what: str, n: int) -> None:
    dev, bf16 = torch.device("cuda"), torch.bfloat16
    D, page = 128, 64
    if what == "rope":
        qkv = torch.randn(4, 4096, 40, D, device=dev).to(bf16)
        q, k = qkv[:, :, :32], qkv[:, :, 32:]
        qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), \
            torch.empty_like(k, memory_format=torch.contiguous_format)
        pos = torch.arange(4096, dtype=torch.int32, device=dev).repeat(4, 1)
        phases = torch.empty(D // 2, dtype=torch.int64, device=dev)
        dd.dllm_rope_phases(D, phases)
        for _ in range(n):
            dd.dllm_qk_norm_rope(q, k, qo, ko, pos, phases)
        torch.cuda.synchronize()
        return
    B, m, heads, group, T, causal = {"cache": (8, 4096, 8, 1, 4096, False),
                                     "token": (32, 1, 8, 4, 8192, False),
                                     "block": (16, 64, 2, 8, 4160, False),
                                     "evict": (32, 1, 8, 4, 8192, False),
                                     "piece": (2, 1024, 8, 4, 16384, True)}[what.removesuffix("_weights")]
    cache = dd.Kv4Cache(B * (T // page), heads, page, D, B, T // page, dev)
    cache.table.copy_(torch.randperm(B * (T // page), device=dev).view(B, -1).to(torch.int32))
    for b in range(0, T, 1024):  # fill it, a stretch of entries at a time
        k = torch.randn(B, min(1024, T - b), heads, D, device=dev).to(bf16)
        pos = torch.arange(b, b + k.shape[1], dtype=torch.int32, device=dev).repeat(B, 1)
        dd.dllm_kv4_write(cache, k, k, pos)
    if what == "cache":
        k, v = (torch.randn(B, m, heads, D, device=dev).to(bf16) for _ in range(2))
        pos = torch.arange(m, dtype=torch.int32, device=dev).repeat(B, 1)
        for _ in range(n):
            dd.dllm_kv4_write(cache, k, v, pos)
            dd.dllm_kv4_read(cache, k, v, pos)
        torch.cuda.synchronize()
        return
    weights = torch.rand(B, T, device=dev)
    if what == "evict":
        lens = torch.empty(B, dtype=torch.int32, device=dev)
        slots = torch.empty(B, T, dtype=torch.int32, device=dev)
        ws = dd.workspace(dd.dllm_kv4_evict_workspace_bytes(cache, B, T), dev)
        for _ in range(n):
            dd.dllm_kv4_evict(cache, weights, None, T, T // 2, slots, lens, ws)
        torch.cuda.synchronize()
        return
    q = torch.randn(B, m, heads * group, D, device=dev).to(bf16)
    out = torch.empty_like(q)
    if what.endswith("_weights"):
        lse = torch.full((B, heads * group, m), 9.0, device=dev)  # about what such queries have
        ws = dd.workspace(dd.dllm_attention_kv4_weights_workspace_bytes(cache, B, m, heads * group, T), dev)
        for _ in range(n):
            dd.dllm_attention_kv4_weights(q, cache, None, T, lse, weights, ws, causal=causal)
        if dd.dllm_get_status(ws) != dd.DLLM_OK:
            raise SystemExit("the accumulated weights reported a fault")
        return
    ws = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(cache, B, m, heads * group, T), dev)
    for _ in range(n):
        dd.dllm_attention_kv4(q, cache, None, T, out, ws, causal=causal)
    if dd.dllm_get_status(ws) != dd.DLLM_OK:
        raise SystemExit("attention reported a fault")


def main(argv) -> None:
    what = argv[0] if argv else "step"
    n = int(argv[1]) if len(argv) > 1 else 4
    if what in ("rope", "cache", "token", "block", "piece", "token_weights", "block_weights", "piece_weights",
                "evict"):
        refresh_operator(what, n)
        return
    draws = {"whole": dict(temperature=0.7), "nucleus": dict(temperature=0.7, top_p=0.9), "top_k": dict(top_k=50)}
    if what not in ("stats", "probs", "gemm", "step", "fused", *draws):
        raise SystemExit(f"unknown kernel family {what!r}")
    B, L = (int(argv[2]), int(argv[3])) if what in ("stats", *draws) and len(argv) > 3 else (B_, L_)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    shape = dd.make_shape(B, L, V, dd.DLLM_BF16)
    lg = torch.randn(B, L, V, device=dev, generator=g).mul_(2).to(torch.bfloat16)
    state, stats = dd.BlockState(B, L), dd.StatsBuffers(B * L)
    ws = dd.workspace(dd.dllm_workspace_bytes(shape))
    if what in draws:
        lg[..., :32] += 12.0 - torch.arange(32, device=dev) / 4  # a head over the bulk
        uniform = torch.rand(B * L, device=dev, generator=g)
        for _ in range(n):
            dd.dllm_sample(lg, shape, None, uniform, stats, **draws[what])
        torch.cuda.synchronize()
        return
    if what == "stats":
        for _ in range(n):
            state.reset()
            dd.dllm_commit_threshold(lg, shape, stats, state, TAU, -1, ws)
        torch.cuda.synchronize()
        return
    Et = torch.randn(dd.dllm_embedding_t_elems(V, D), device=dev, generator=g)
    Et = Et.mul_(0.02).to(torch.bfloat16)
    ws_s = dd.workspace(dd.dllm_smooth_workspace_bytes(shape, D))
    out = torch.empty(B * L, D, device=dev)
    row_ids = torch.empty(B * L, dtype=torch.int32, device=dev)
    M = torch.zeros(1, dtype=torch.int32, device=dev)
    T = PREFIX + L
    refresh = torch.empty(B * T, dtype=torch.uint8, device=dev)
    idx = torch.empty(B * T, dtype=torch.int32, device=dev)
    count = torch.empty(B, dtype=torch.int32, device=dev)
    state.reset()
    dd.dllm_commit_threshold(lg, shape, stats, state, TAU, -1, ws)
    if what == "gemm":
        dd.dllm_smooth_probs(lg, shape, stats, state, D, row_ids, M, ws_s)
    for _ in range(n):
        if what == "probs":
            dd.dllm_smooth_probs(lg, shape, stats, state, D, row_ids, M, ws_s)
        elif what == "gemm":
            dd.dllm_smooth_gemm(shape, Et, D, out, M, ws_s)
        elif what == "fused":
            state.reset()
            dd.dllm_commit_threshold_smooth(lg, shape, stats, state, TAU, -1, Et, D, out,
                                            row_ids, M, ws_s)
            dd.dllm_kv_refresh_mask(state, PREFIX, WINDOW, refresh, idx, count)
        else:
            state.reset()
            dd.dllm_commit_threshold(lg, shape, stats, state, TAU, -1, ws)
            dd.dllm_smooth_probs(lg, shape, stats, state, D, row_ids, M, ws_s)
            dd.dllm_smooth_gemm(shape, Et, D, out, M, ws_s)
            dd.dllm_kv_refresh_mask(state, PREFIX, WINDOW, refresh, idx, count)
    torch.cuda.synchronize()
    if dd.dllm_get_status(ws_s) != dd.DLLM_OK:
        raise SystemExit("smoothing reported an error status")


if __name__ == "__main__":
    main(sys.argv[1:])
    print("ok")

"""Refusals of sampling, accumulated weights and eviction: nothing is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import diffusion_decoding_gb300 as dd
from diffusion_decoding_gb300 import build as cuda_build

P = 1 << 20  # an address that is only checked


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return dd.lib()


INVALID, UNSUPPORTED = dd.DLLM_ERR_INVALID_ARG, dd.DLLM_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,want", [
    (dict(logits=None), INVALID), (dict(uniform=None), INVALID), (dict(how=None), INVALID),
    (dict(uniform=P + 2), INVALID), (dict(logits=P + 1), INVALID), (dict(argmax=None), INVALID),
    (dict(V=(1 << 20) + 1, row_stride=(1 << 20) + 1), UNSUPPORTED), (dict(B=0), INVALID),
    (dict(L=1025), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(row_stride=10), INVALID),
    (dict(temperature=-1.0), INVALID), (dict(temperature=2.0 ** -11), INVALID),
    (dict(temperature=2000.0), INVALID), (dict(temperature=float("nan")), INVALID),
    (dict(top_k=-1), INVALID), (dict(top_p=0.0), INVALID), (dict(top_p=1.5), INVALID),
    (dict(top_p=float("nan")), INVALID), (dict(min_p=-0.1), INVALID), (dict(min_p=1.1), INVALID),
    (dict(min_p=float("nan")), INVALID)])
def test_sample(lib, change, want):
    a = dict(logits=P, uniform=P, how=True, argmax=P, V=1000, row_stride=1000, B=2, L=8, dtype=dd.DLLM_BF16,
             temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    a.update(change)
    if "V" in change or "row_stride" in change:
        a["row_stride"] = change.get("row_stride", a["V"])
    sh = dd.dllm_shape(a["B"], a["L"], a["V"], a["dtype"], a["row_stride"])
    how = dd.dllm_sampling(a["temperature"], a["top_k"], a["top_p"], a["min_p"])
    st = dd.dllm_stats(P, P, P, a["argmax"])
    rc = lib.dllm_sample(a["logits"], ctypes.byref(sh), None, a["uniform"],
                         ctypes.byref(how) if a["how"] else None, ctypes.byref(st), None)
    assert rc == want and lib.dllm_last_error()


def cache(**kw):
    d = dict(pages=10, heads=2, page_size=64, head_dim=128, table_stride=4)
    d.update(kw)
    return dd.dllm_kv4_cache(P, P, P, P, P, d["pages"], d["heads"], d["page_size"], d["head_dim"],
                             d["table_stride"])


@pytest.mark.parametrize("change,want", [
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(weights=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 8), INVALID), (dict(ws_bytes=0), INVALID), (dict(dtype=dd.DLLM_F32), UNSUPPORTED),
    (dict(q_heads=3), INVALID), (dict(max_len=257), INVALID), (dict(max_len=-1), INVALID), (dict(n=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(scale=float("inf")), INVALID), (dict(keep=float("nan")), INVALID),
    (dict(weights_stride=100), INVALID), (dict(prior_stride=100), INVALID), (dict(mask_stride=100), INVALID),
    (dict(weights=P + 2), INVALID), (dict(prior=P + 1), INVALID), (dict(lse=P + 2), INVALID),
    (dict(lens=P + 2), INVALID), (dict(prior=P, weights=P, prior_stride=300), INVALID),
    (dict(B=1 << 20, max_len=1 << 20, table_stride=1 << 14, weights_stride=1 << 20, prior_stride=1 << 20),
     UNSUPPORTED)])
def test_weights(lib, change, want):
    a = dict(q=True, q_heads=4, dtype=dd.DLLM_BF16, lens=None, max_len=256, mask=P, mask_stride=256, scale=0.1, lse=P,
             prior=2 * P, prior_stride=256, keep=1.0, weights=P, weights_stride=256, B=2, n=3, ws=P,
             ws_bytes=1 << 40, head_dim=128, table_stride=4)
    a.update(change)
    c = cache(head_dim=a["head_dim"], table_stride=a["table_stride"])
    q = dd.dllm_heads(P, a["q_heads"], a["dtype"], 4 * 128 * 3, 4 * 128, 128)
    rc = lib.dllm_attention_kv4_weights(
        ctypes.byref(q) if a["q"] else None, ctypes.byref(c), a["lens"], a["max_len"], a["mask"], a["mask_stride"],
        a["scale"], 0, a["lse"], a["prior"], a["prior_stride"], a["keep"], a["weights"], a["weights_stride"], a["B"],
        a["n"], a["ws"], a["ws_bytes"], None)
    assert rc == want and lib.dllm_last_error()


def test_workspace_sizes(lib):
    c = cache()
    assert lib.dllm_attention_kv4_weights_workspace_bytes(ctypes.byref(c), 2, 3, 4, 256) > 0
    assert lib.dllm_attention_kv4_weights_workspace_bytes(ctypes.byref(c), 2, 3, 3, 256) == 0
    assert lib.dllm_attention_kv4_weights_workspace_bytes(ctypes.byref(c), 2, 3, 4, 257) == 0
    assert lib.dllm_kv4_evict_workspace_bytes(ctypes.byref(c), 2, 256) > 0
    assert lib.dllm_kv4_evict_workspace_bytes(ctypes.byref(c), 2, 257) == 0
    assert lib.dllm_kv4_evict_workspace_bytes(ctypes.byref(c), 0, 256) == 0


@pytest.mark.parametrize("change,want", [
    (dict(weights=None), INVALID), (dict(slots=None), INVALID), (dict(lens_out=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID), (dict(budget=-1), INVALID), (dict(first=-1), INVALID),
    (dict(last=-1), INVALID), (dict(first=60, last=41), INVALID), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID),
    (dict(max_len=257), INVALID), (dict(max_len=-1), INVALID), (dict(B=0), INVALID),
    (dict(B=(1 << 20) + 1), UNSUPPORTED), (dict(weights_stride=255), INVALID), (dict(slots_stride=255), INVALID),
    (dict(weights_out_stride=255), INVALID), (dict(weights_out=P, weights_out_stride=300), INVALID),
    (dict(weights=P + 1), INVALID), (dict(slots=P + 2), INVALID), (dict(lens=P + 2), INVALID),
    (dict(head_dim=48), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED)])
def test_evict(lib, change, want):
    a = dict(weights=P, weights_stride=256, lens=None, max_len=256, budget=100, first=4, last=8, slots=2 * P,
             slots_stride=256, lens_out=P, weights_out=3 * P, weights_out_stride=256, B=2, ws=P, ws_bytes=1 << 30,
             head_dim=128, page_size=64)
    a.update(change)
    c = cache(head_dim=a["head_dim"], page_size=a["page_size"])
    rc = lib.dllm_kv4_evict(ctypes.byref(c), a["weights"], a["weights_stride"], a["lens"], a["max_len"], a["budget"],
                            a["first"], a["last"], a["slots"], a["slots_stride"], a["lens_out"], a["weights_out"],
                            a["weights_out_stride"], a["B"], a["ws"], a["ws_bytes"], None)
    assert rc == want and lib.dllm_last_error()


def test_binding_refuses(lib):
    """Shapes and types that the C entry points cannot see."""
    kv = dd.Kv4Cache(4, 2, 16, 64, 2, 2, device="cpu")
    stats, shape = dd.StatsBuffers(8, device="cpu"), dd.make_shape(1, 8, 100, dd.DLLM_F32)
    f, i = torch.zeros, torch.zeros(2, 32, dtype=torch.int32)
    z, u, ws = f(8, 100), f(8), torch.zeros(1 << 16, dtype=torch.uint8)
    for bad in (f(7), f(8, dtype=torch.float64), f(16)[::2]):
        with pytest.raises(ValueError):
            dd.dllm_sample(z, shape, None, bad, stats)
    for bad in (f(8, dtype=torch.int32), f(7, dtype=torch.uint8), f(16, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            dd.dllm_sample(z, shape, bad, u, stats)
    q, lse, w = f(2, 3, 4, 64, dtype=torch.bfloat16), f(2, 4, 3), f(2, 32)
    lens = torch.zeros(2, dtype=torch.int32)

    def weights(q=q, lens=lens, max_len=32, lse=lse, w=w, **kw):
        with pytest.raises(ValueError):
            dd.dllm_attention_kv4_weights(q, kv, lens, max_len, lse, w, ws, **kw)
    weights(q=q[:1])
    weights(q=q[..., :32])
    weights(lse=lse[:, :3])
    weights(lse=lse.double())
    weights(lens=lens.long())
    weights(w=w[:, :31])
    weights(w=f(2, 64)[:, ::2])
    weights(w=w.double())
    weights(prior=w[:1])
    weights(key_mask=f(2, 31, dtype=torch.uint8))
    weights(key_mask=f(2, 32))

    def evict(w=w, lens=lens, max_len=32, slots=i, out=lens, **kw):
        with pytest.raises(ValueError):
            dd.dllm_kv4_evict(kv, w, lens, max_len, 10, slots, out, ws, **kw)
    evict(w=None)
    evict(slots=None)
    evict(out=None)
    evict(w=w[:, :20])
    evict(slots=i.float())
    evict(slots=i[:1])
    evict(lens=lens[:1])
    evict(out=lens.float())
    evict(weights_out=w[:, ::2])

"""Attention over the 4-bit cache with more (sequence, head) pairs than one dimension of a grid of
eight rows each can hold: every query gets its output, those behind the 2^28th pair too."""
import math

import pytest
import torch

import diffusion_decoding_gb300 as dd
import refresh_ref as ref
from test_gpu_refresh_ops import DEV, fill, gen, make_cache, randn

pytestmark = pytest.mark.gpu


def test_attention_of_more_segments_than_a_grid_of_rows():
    g = gen(21)
    B, H, D, T, long = 1 << 20, 264, 64, 1024, 1 << 14  # the last 2^14 sequences see T entries, others none
    one = make_cache(g, 1, T, H, D, T, spare=0)
    k, v = fill(g, one, T)
    q1 = (1.5 * randn(g, 1, 1, H, D)).to(torch.bfloat16)
    o, l, mag, top = ref.attention(q1, k, v, torch.ones(1, 1, T, dtype=torch.bool, device=DEV), D ** -0.5)
    c = dd.Kv4Cache.of(one.k_codes, one.k_params, one.v_codes, one.v_params,
                       one.table.expand(B, 1).contiguous())
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens[B - long:] = T
    out = torch.full((B, 1, H, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H, 1), 9.0, device=DEV)
    ws = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(c, B, 1, H, T))
    ws[256:] = 255
    dd.dllm_attention_kv4(q1.expand(B, 1, H, D), c, lens, T, out, ws, lse=lse)
    assert dd.dllm_get_status(ws) == dd.DLLM_OK
    del ws
    step = 1 << 13
    for b in range(0, B - long, step):
        assert not out[b:b + step].any() and (lse[b:b + step] == -math.inf).all()
    for b in range(B - long, B, step):
        err = (out[b:b + step].double() - o).abs()
        assert (err <= 2.0 ** -8 * 1.03 * (mag + o.abs()) + 1e-30).all()
        d = (lse[b:b + step].double() - l).abs()
        assert (d <= 1e-5 * l.abs().clamp(min=1) + 2.0 ** -20 * top).all()

"""How the attention shares its work out: several whole segments a CTA, equal stretches that start and end
within segments, more sequences than a warp looks at at once; lengths that differ, masks, causal.

Each tile of 64 entries has its value in a channel of its own, so an output channel is the weight of
its tiles: a part that is lost, doubled or given to another row is off by all of itself, where values
of both signs would hide it in the tolerance (which is that of the other sizes)."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
from test_gpu_refresh_ops import DEV, check_attention, entries, gen, make_cache, randn, run, seen_of

pytestmark = pytest.mark.gpu

WHOLE = [  # B, n, H, G, D, page, T: whole segments, several to a CTA (more segments than SMs)
    (60, 40, 3, 2, 128, 16, 202), (100, 17, 4, 2, 128, 64, 130), (50, 150, 4, 1, 64, 48, 200),
    (40, 33, 8, 6, 128, 32, 70), (90, 40, 4, 1, 64, 16, 333), (45, 20, 4, 2, 192, 16, 260),
    (60, 50, 3, 2, 256, 64, 150)]
STRETCHES = [  # 64 to 96 segments of 65 tiles and more: equal stretches of the line
    (32, 32, 2, 8, 128, 64, 4160), (16, 64, 2, 8, 128, 16, 4111), (64, 40, 1, 2, 128, 48, 4160),
    (32, 70, 2, 2, 64, 64, 4100), (64, 50, 1, 1, 64, 16, 4160), (32, 40, 2, 3, 256, 64, 4160),
    (16, 30, 4, 4, 192, 32, 4150), (12, 400, 2, 2, 128, 64, 8000)]
FEW = [  # the kernel for few rows: split, in tiles of 8 and 16 rows
    (50, 1, 2, 4, 128, 64, 3000), (40, 3, 2, 4, 128, 16, 2500), (20, 4, 2, 5, 64, 48, 2000),
    (40, 2, 1, 4, 256, 32, 1500), (35, 1, 3, 7, 192, 16, 1200), (70, 1, 8, 1, 64, 64, 700)]


def place(B, T, H, D):
    """Values [B, T, H, D]: 1 in the channel of the entry's tile, 0 in the others."""
    t = torch.arange(T, device=DEV) // 64
    ch = (t[:, None] + 7 * torch.arange(H, device=DEV)) % D
    return torch.nn.functional.one_hot(ch, D).to(torch.bfloat16).expand(B, T, H, D).contiguous()


@pytest.mark.parametrize("masked,causal", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("B,n,H,G,D,ps,T", WHOLE + STRETCHES + FEW)
def test_attention_by_tiles(B, n, H, G, D, ps, T, masked, causal):
    g = gen(B + n + D + T)
    c = make_cache(g, B, T, H, D, ps)
    k = randn(g, B, T, H, D).to(torch.bfloat16)
    dd.dllm_kv4_write(c, k, place(B, T, H, D), torch.arange(T, dtype=torch.int32, device=DEV).repeat(B, 1))
    kk, vv = entries(c, c.k_codes, c.k_params, T), entries(c, c.v_codes, c.v_params, T)
    q = randn(g, B, n, H * G, D).to(torch.bfloat16)
    lens = torch.randint(T // 2, T + 1, (B,), generator=torch.Generator().manual_seed(B + T)).tolist()
    lens[0], lens[1], lens[B // 2], lens[B - 1] = T, 0, 1, T - 64
    mask = None
    if masked:
        mask = (torch.rand(B, T, generator=g, device=DEV) < 0.6).to(torch.uint8)
        mask[2, : T // 2] = 0
    out, lse = run(c, q, lens, T, causal=causal, mask=mask)
    seen = seen_of(B, n, T, lens, mask, causal, c)
    for b in range(0, B, 4):  # a few sequences of the 64-bit statement at a time
        e = slice(b, b + 4)
        check_attention(out[e], lse[e], q[e], kk[e], vv[e], seen[e], D ** -0.5)


@pytest.mark.parametrize("B,n,H,G,D,ps,T", [WHOLE[0], WHOLE[2], STRETCHES[0], STRETCHES[5], FEW[1]])
def test_attention_of_equal_lengths_by_tiles(B, n, H, G, D, ps, T):
    g = gen(T)
    c = make_cache(g, B, T, H, D, ps)
    k = randn(g, B, T, H, D).to(torch.bfloat16)
    dd.dllm_kv4_write(c, k, place(B, T, H, D), torch.arange(T, dtype=torch.int32, device=DEV).repeat(B, 1))
    kk, vv = entries(c, c.k_codes, c.k_params, T), entries(c, c.v_codes, c.v_params, T)
    q = randn(g, B, n, H * G, D).to(torch.bfloat16)
    out, lse = run(c, q, None, T)
    seen = torch.ones(4, n, T, dtype=torch.bool, device=DEV)
    for b in range(0, B, 4):
        e = slice(b, b + 4)
        check_attention(out[e], lse[e], q[e], kk[e], vv[e], seen[: out[e].shape[0]], D ** -0.5)

"""Attention over the 4-bit cache where a query, a key or a value is NaN (a group of the cache that held
a NaN or an infinity reads back as NaN): by the formulas a row is NaN where a score that it sees is,
an output channel where a value that the row sees is, and nothing else is touched.  Everything that
is not NaN is held to the tolerances of the other sizes (test_gpu_refresh_ops.py)."""
import math

import pytest
import torch

import refresh_ref as ref
from test_gpu_refresh_ops import DEV, entries, gen, make_cache, randn, run, seen_of

pytestmark = pytest.mark.gpu


def check(out, lse, q, k, v, seen, scale):
    """Against the 64-bit statement of the finite parts; q, k, v may hold NaN."""
    B, n, H, D = q.shape
    G = H // k.shape[2]
    kn, vn = k.isnan().any(-1), v.isnan()  # [B, T, Hkv], [B, T, Hkv, D]
    zero = lambda x: torch.where(x.isnan(), torch.zeros_like(x), x)  # noqa: E731
    o, l, mag, top = ref.attention(zero(q), zero(k), zero(v), seen, scale)
    s = seen.double()
    bad_score = torch.einsum("bnt,bth->bnh", s, kn.double()).repeat_interleave(G, 2) > 0
    bad_score |= q.isnan().any(-1) & seen.any(-1)[:, :, None]
    bad = torch.einsum("bnt,bthd->bnhd", s, vn.double()).repeat_interleave(G, 2) > 0
    bad |= bad_score[..., None]
    assert torch.equal(out.isnan(), bad)
    err, tol = (out.double() - o).abs(), 2.0 ** -8 * 1.03 * (mag + o.abs())
    assert (err <= tol + 1e-30)[~bad].all()
    nan_l = bad_score.permute(0, 2, 1)
    assert torch.equal(lse.isnan(), nan_l)
    none = ~seen.any(-1)[:, None].expand_as(lse)
    assert (lse[none] == -math.inf).all() and (out.permute(0, 2, 1, 3)[none] == 0).all()
    rest = ~none & ~nan_l
    d = (lse.double() - l).abs()[rest]
    assert (d <= 1e-5 * l.abs().clamp(min=1)[rest] + 2.0 ** -20 * top[rest]).all()


def store(g, c, T, nan_k=(), nan_v=()):
    """Random keys and values of T entries, with NaN in one channel of the listed (sequence, entry,
    head, channel); what the cache then holds."""
    B = c.table.shape[0]
    k, v = (randn(g, B, T, c.heads, c.head_dim).to(torch.bfloat16) for _ in range(2))
    for x, where in ((k, nan_k), (v, nan_v)):
        for at in where:
            x[at] = math.nan
    import diffusion_decoding_gb300 as dd
    dd.dllm_kv4_write(c, k, v, torch.arange(T, dtype=torch.int32, device=DEV).repeat(B, 1))
    return entries(c, c.k_codes, c.k_params, T), entries(c, c.v_codes, c.v_params, T)


# few rows in tiles of 8 and 16, whole and split; many rows: the same in two groups, 256 in two groups,
# one group of 128 rows
ROWS = [(1, 2, 128, 16), (3, 4, 128, 64), (1, 5, 64, 16), (1, 3, 192, 32), (2, 3, 256, 16), (48, 2, 128, 16),
        (100, 3, 64, 64), (48, 1, 192, 16), (40, 1, 256, 64)]


@pytest.mark.parametrize("n,G,D,ps", ROWS)
@pytest.mark.parametrize("T", [1, 17, 331, 5000])
def test_nan_queries(n, G, D, ps, T):
    g = gen(T + n)
    B, H = 2, 2
    c = make_cache(g, B, T, H, D, ps)
    k, v = store(g, c, T)
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    q[0, 0, 0, 3] = math.nan
    q[1, n - 1, H * G - 1, D - 1] = math.nan
    mask = (torch.rand(B, T, generator=g, device=DEV) < 0.7).to(torch.uint8)
    for m in (None, mask):
        out, lse = run(c, q, None, T, mask=m)
        check(out, lse, q, k, v, seen_of(B, n, T, [T] * B, m, False, c), D ** -0.5)


@pytest.mark.parametrize("n,G,D,ps", ROWS)
@pytest.mark.parametrize("T,at", [(1, 0), (17, 16), (331, 330), (331, 200), (5000, 4999), (5000, 0)])
def test_nan_keys(n, G, D, ps, T, at):
    g = gen(T + n + at)
    B, H = 2, 2
    c = make_cache(g, B, T, H, D, ps)
    k, v = store(g, c, T, nan_k=[(1, at, 1, 40)])
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    out, lse = run(c, q, None, T)
    check(out, lse, q, k, v, seen_of(B, n, T, [T] * B, None, False, c), D ** -0.5)
    # hidden by the mask it is not used; alone in a stretch it is the only thing seen there
    mask = torch.ones(B, T, dtype=torch.uint8, device=DEV)
    mask[1, at] = 0
    out, lse = run(c, q, None, T, mask=mask)
    check(out, lse, q, k, v, seen_of(B, n, T, [T] * B, mask, False, c), D ** -0.5)
    lone = torch.ones(B, T, dtype=torch.uint8, device=DEV)
    lone[1, max(0, at - 300):at] = 0
    lone[1, at + 1:at + 300] = 0
    out, lse = run(c, q, None, T, mask=lone)
    check(out, lse, q, k, v, seen_of(B, n, T, [T] * B, lone, False, c), D ** -0.5)


@pytest.mark.parametrize("n,G,D,ps", ROWS + [(70, 8, 128, 32), (300, 1, 64, 16), (200, 2, 256, 48), (4, 4, 64, 48)])
@pytest.mark.parametrize("T", [310, 2500])
@pytest.mark.parametrize("masked", [False, True])
def test_nan_values_and_causal_rows(n, G, D, ps, T, masked):
    # a value that only later rows see leaves the earlier ones alone, whatever tile they share
    g = gen(T + n)
    B, H = 2, 2
    lens = [T, T - 41]
    c = make_cache(g, B, T, H, D, ps)
    first = T - n
    at = {lens[0] - 1, max(0, first), max(0, first) + n // 2, max(0, first - 1), max(0, first - 130), 5}
    nan_v = [(0, j, h, (37 * (i + h)) % D) for i, j in enumerate(sorted(at)) for h in (0, 1) if (i + h) % 3]
    nan_v += [(1, lens[1] - 1, 0, 0), (1, lens[1] - 1 - n // 3, 1, D - 1)]
    k, v = store(g, c, T, nan_v=nan_v)
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    mask = None
    if masked:
        mask = (torch.rand(B, T, generator=g, device=DEV) < 0.7).to(torch.uint8)
    for causal in (True, False):
        out, lse = run(c, q, lens, T, causal=causal, mask=mask)
        check(out, lse, q, k, v, seen_of(B, n, T, lens, mask, causal, c), D ** -0.5)


@pytest.mark.parametrize("n,G,D,ps", ROWS + [(300, 1, 64, 16)])
def test_nan_keys_and_causal_rows(n, G, D, ps):
    g = gen(n)
    B, H, T = 1, 2, 400
    c = make_cache(g, B, T, H, D, ps)
    k, v = store(g, c, T, nan_k=[(0, T - 1 - n // 2, 1, 7), (0, T - 1, 0, 0)])
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    out, lse = run(c, q, None, T, causal=True)
    check(out, lse, q, k, v, seen_of(B, n, T, [T], None, True, c), D ** -0.5)


@pytest.mark.parametrize("n,G,D", [(1, 4, 128), (48, 2, 128), (40, 1, 256), (90, 4, 64)])
def test_nan_value_of_a_vanishing_weight(n, G, D):
    # a value that is seen counts, however small its weight: 0 * NaN is NaN wherever the sum is joined
    g = gen(n)
    T = 700
    c = make_cache(g, 1, T, 1, D, 64)
    k = torch.zeros(1, T, 1, D, device=DEV, dtype=torch.bfloat16)
    k[:, 65] = 100.0  # one entry takes all of the weight
    v = randn(g, 1, T, 1, D).to(torch.bfloat16)
    v[0, 3, 0, 0] = v[0, 140, 0, D - 1] = math.nan
    import diffusion_decoding_gb300 as dd
    dd.dllm_kv4_write(c, k, v, torch.arange(T, dtype=torch.int32, device=DEV)[None])
    kk, vv = entries(c, c.k_codes, c.k_params, T), entries(c, c.v_codes, c.v_params, T)
    q = torch.ones(1, n, G, D, device=DEV, dtype=torch.bfloat16)
    out, lse = run(c, q, None, T, scale=1.0)
    check(out, lse, q, kk, vv, torch.ones(1, n, T, dtype=torch.bool, device=DEV), 1.0)

"""Norm + rotation, the 4-bit cache and the attention over it, on the GPU against 64-bit
statements (refresh_ref.py).

Tolerances.  norm_rope: fp32 sums and products, a hardware sine and cosine with at most 2^-21 of
absolute error and a phase of 24 bits: 4e-6 of the channel's pair; a bf16 result (8 significant
bits) adds half an ulp, at most 2^-8 of itself.  Cache: bf16 inputs bit for bit; fp32 inputs within half a step (a quotient next to
a tie may round either way).  Attention: each weight is rounded to bf16 (2^-8 of sum_j p_j |v_j|) and
so is the result (2^-8 of itself), and 3 % of that for the fp32 scores; lse: 1e-5 of max(1, |lse|)
plus 2^-20 of the largest sum |q_c k_c|, what fp32 sums of the products can lose."""
import math

import pytest
import torch

import refresh_ref as ref

import diffusion_decoding_gb300 as dd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def phases(R, **kw):
    t = torch.empty(max(R // 2, 1), dtype=torch.int64, device=DEV)
    dd.dllm_rope_phases(R, t, **kw)
    return t


# ---------------------------------------------------------------- norm + rotation

def strided(x, how):
    """The values of x [B, n, H, D] in another layout."""
    B, n, H, D = x.shape
    if how == "plain":
        return x
    if how == "packed":  # the heads of one projection among others
        big = torch.full((B, n, H + 3, D), 7.0, dtype=x.dtype, device=DEV)
        v = big[:, :, 1:H + 1]
    elif how == "heads_first":
        v = torch.empty(B, H, n, D, dtype=x.dtype, device=DEV).transpose(1, 2)
    else:  # odd: rows off 16-byte boundaries
        flat = torch.empty(B * n * H * (D + 1) + 1, dtype=x.dtype, device=DEV)
        v = flat[1:].view(B, n, H, D + 1)[..., :D]
    v.copy_(x)
    return v


def check_norm_rope(g, o, size):
    tol = 4e-6 * size + (2.0 ** -8 * o.abs() if g.dtype == torch.bfloat16 else 0)
    bad = (g.double() - o).abs() > tol + 1e-30
    assert not bad.any(), (bad.sum().item(), ((g.double() - o).abs() / (tol + 1e-30)).max().item())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,Hq,Hk,D,R,inter", [
    (1, 1, 16, 4, 128, 128, False), (2, 5, 3, 1, 64, 64, True), (1, 7, 5, 5, 80, 32, False),
    (2, 3, 4, 2, 256, 64, True), (1, 2, 1, 1, 16, 16, False), (3, 1, 7, 1, 96, 96, True),
    (1, 3, 2, 2, 512, 512, False), (1, 4, 2, 1, 50, 22, False), (1, 4, 2, 1, 33, 10, True),
    (1, 2, 3, 1, 576, 64, True), (1, 2, 1, 1, 1, 0, False), (2, 300, 12, 3, 128, 128, False),
    (1, 1, 1, 1, 1024, 1024, True), (1, 9, 2, 2, 128, 0, False)])
@pytest.mark.parametrize("layout", ["plain", "packed", "heads_first", "odd"])
def test_norm_rope(dtype, B, n, Hq, Hk, D, R, inter, layout):
    g = gen(B * 1000 + D + R)
    q, k = (randn(g, B, n, H, D).mul(1.7).to(dtype) for H in (Hq, Hk))
    wq, wk = ((1 + 0.3 * randn(g, D)).to(dtype) for _ in range(2))
    pos = torch.randint(0, 300, (B, n), generator=g, device=DEV, dtype=torch.int32)
    ph = phases(R, base=10000.0) if R else None
    qi, ki = strided(q, layout), strided(k, layout)
    qo, ko = strided(torch.zeros_like(q), layout), torch.zeros_like(k)
    dd.dllm_qk_norm_rope(qi, ki, qo, ko, pos, ph, wq, wk, 1e-6, inter)
    f = ref.frequencies(R, 10000.0) if R else None
    for x, w, out in ((q, wq, qo), (k, wk, ko)):
        check_norm_rope(out, *ref.norm_rope(x, pos, f, w, 1e-6, inter))


@pytest.mark.parametrize("kw,bands", [
    (dict(base=500000.0, factor=8.0), None),
    (dict(base=10000.0, factor=16.0, scaling=dd.DLLM_ROPE_BANDS, original_len=4096.0,
          slow_turns=1.0, fast_turns=32.0), (4096.0, 1.0, 32.0))])
def test_rotation_far_into_a_long_context(kw, bands):
    # positions up to 2^20: the phase must not lose bits with the angle
    g = gen(4)
    x = randn(g, 1, 64, 4, 128)
    pos = torch.randint(0, 1 << 20, (1, 64), generator=g, device=DEV, dtype=torch.int32)
    pos[0, 0], pos[0, 1] = (1 << 20) - 1, 0
    out = torch.empty_like(x)
    dd.dllm_qk_norm_rope(x, None, out, None, pos, phases(128, **kw), magnitude=1.25, norm=False)
    f = ref.frequencies(128, kw["base"], kw["factor"], bands)
    check_norm_rope(out, *ref.norm_rope(x, pos, f, None, 0.0, False, 1.25, norm=False))


def test_rotation_is_relative_and_keeps_length():
    # <R(p) q, R(p') k> depends on p - p' alone; the norm of every pair stays
    g = gen(5)
    q, k = randn(g, 1, 2, 1, 128), randn(g, 1, 2, 1, 128)
    q[0, 1], k[0, 1] = q[0, 0], k[0, 0]
    ph = phases(128)
    outs = []
    for x, p in ((q, [100, 70000]), (k, [37, 69937])):
        o = torch.empty_like(x)
        dd.dllm_qk_norm_rope(x, None, o, None, torch.tensor([p], dtype=torch.int32, device=DEV),
                             ph, norm=False)
        outs.append(o.double())
    d = (outs[0] * outs[1]).sum(-1).flatten()
    assert abs(d[0] - d[1]) < 1e-5 * (q.norm() * k.norm()).item()
    assert torch.allclose(outs[0].norm(dim=-1), q.double().norm(dim=-1), rtol=4e-6)


@pytest.mark.parametrize("D", [128, 50])
def test_norm_rope_skips_tokens_and_works_in_place(D):
    g = gen(6)
    x = randn(g, 2, 40, 3, D).to(torch.bfloat16)
    pos = torch.randint(0, 99, (2, 64), generator=g, device=DEV, dtype=torch.int32)
    pos[:, ::3] = -1
    w = (1 + 0.1 * randn(g, D)).to(torch.bfloat16)
    y = x.clone()
    dd.dllm_qk_norm_rope(None, y, None, y, pos, phases(D), k_weight=w)
    o, size = ref.norm_rope(x, pos[:, :40], ref.frequencies(D, 10000.0), w, 1e-6, False)
    keep = pos[:, :40] < 0
    assert torch.equal(y[keep], x[keep])
    check_norm_rope(y[~keep], o[~keep], size[~keep])


def test_norm_of_zeros_and_of_extremes():
    x = torch.zeros(1, 4, 1, 128, device=DEV)
    x[0, 1, 0, 3] = 1e18
    x[0, 2] = 1e-20
    x[0, 3, 0, 0] = math.nan
    y = torch.empty_like(x)
    dd.dllm_qk_norm_rope(x, None, y, None, None, None, eps=1e-6)
    assert torch.equal(y[0, 0], x[0, 0])
    assert abs(y[0, 1, 0, 3].item() - math.sqrt(128)) < 1e-4 and y[0, 1, 0, :3].abs().max() == 0
    assert torch.allclose(y[0, 2], torch.full_like(y[0, 2], 1e-17), rtol=1e-5)
    assert y[0, 3].isnan().all()


# ---------------------------------------------------------------- the 4-bit cache

def make_cache(g, B, T, H, D, ps, spare=3):
    per = max(1, -(-T // ps))
    c = dd.Kv4Cache(B * per + spare, H, ps, D, B, per)
    c.table.copy_((torch.randperm(B * per + spare, generator=g, device=DEV)[:B * per])
                  .view(B, per).to(torch.int32))
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV).to(torch.uint8))
    for t in (c.k_params, c.v_params):  # whatever memory held: NaN steps among them
        t.copy_(torch.randint(-32768, 32768, t.shape, generator=g, device=DEV).to(torch.int16))
    return c


def entries(c, codes, params, T):
    """Values [B, T, H, D] (float64) of the cache's entries by the documented format."""
    at = torch.arange(T, device=DEV)
    page, slot = c.table.long()[:, at // c.page_size], at % c.page_size
    return ref.unpack(codes[page, :, slot[None, :]], params[page, :, slot[None, :]])


@pytest.mark.parametrize("layout", ["plain", "packed", "heads_first", "odd"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,T,H,D,ps", [
    (1, 1, 1, 1, 32, 16), (2, 5, 40, 3, 128, 16), (1, 33, 33, 2, 96, 48), (3, 17, 129, 1, 512, 64),
    (2, 200, 200, 8, 64, 256), (1, 2100, 2100, 4, 128, 64), (1, 3, 5, 5, 256, 65536 // 64)])
def test_cache_write_then_read(dtype, B, n, T, H, D, ps, layout):
    g = gen(T + D)
    c = make_cache(g, B, T, H, D, ps)
    before = [t.clone() for t in (c.k_codes, c.k_params, c.v_codes, c.v_params)]
    k, v = (randn(g, B, n, H, D).mul(torch.exp(randn(g, D))).to(dtype) for _ in range(2))
    if n > 2:
        k[0, 0] = 0.0
        k[0, 1] = k[0, 1].abs()
        v[0, 1] = -v[0, 1].abs()
        v[0, 2] = 1.5
    pos = torch.rand(B, T, device=DEV, generator=g).argsort(1)[:, :n].to(torch.int32)
    if n > 4:
        pos[0, 3] = -1
    dd.dllm_kv4_write(c, strided(k, layout), strided(v, layout), pos)
    ko, vo = (strided(torch.full_like(k, 3.0), layout) for _ in range(2))
    dd.dllm_kv4_read(c, ko, vo, pos)
    here = (pos >= 0)[..., None, None]
    for x, got, codes, params in ((k, ko, c.k_codes, c.k_params), (v, vo, c.v_codes, c.v_params)):
        s, _ = ref.steps(x)
        s = s.repeat_interleave(32, -1)
        err = (got.double() - x.double()).abs()
        assert (torch.where(here, err, 0 * err) <= s / 2 * (1 + 2.0 ** -9)).all()
        if dtype == torch.bfloat16:
            assert torch.equal(got.double(), torch.where(here, ref.quantised(x), 0 * s))
        assert (got[~here.expand_as(got)] == 0).all()
        # the arrays themselves, by the documented format
        at = pos.clamp(min=0).long()
        raw = torch.gather(entries(c, codes, params, T), 1, at[..., None, None].expand_as(x))
        assert torch.equal(torch.where(here, raw, 0 * s), got.double())
    # nothing but those entries changed
    page = torch.gather(c.table.long(), 1, pos.clamp(min=0).long() // ps)
    for t, old in zip((c.k_codes, c.k_params, c.v_codes, c.v_params), before):
        written = torch.zeros(t.shape[0], t.shape[2], dtype=torch.bool, device=DEV)
        written[page[pos >= 0], (pos % ps).long()[pos >= 0]] = True
        same = (t == old).all(-1).all(1)
        assert (same | written).all()


def test_cache_ties_round_away_from_zero():
    # step 1 (0 .. 15), inputs on every half step, both signs of the zero point
    x = torch.zeros(1, 2, 1, 32, device=DEV, dtype=torch.bfloat16)
    x[0, 0, 0, :31] = torch.arange(31, device=DEV) / 2
    x[0, 1, 0, :31] = torch.arange(31, device=DEV) / 2 - 7
    for dt in (torch.bfloat16, torch.float32):
        g = gen(1)
        c = make_cache(g, 1, 16, 1, 32, 16)
        pos = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
        dd.dllm_kv4_write(c, x.to(dt), x.to(dt), pos)
        ko, vo = torch.empty_like(x), torch.empty_like(x)
        dd.dllm_kv4_read(c, ko, vo, pos)
        assert torch.equal(ko.double(), ref.quantised(x)) and torch.equal(vo, ko)


def test_cache_non_finite_and_tiny_groups():
    x = torch.ones(1, 6, 1, 64, device=DEV)
    x[0, 0, 0, 5] = math.inf
    x[0, 1, 0, 5] = -math.inf
    x[0, 2, 0, 5] = math.nan
    x[0, 3, 0, :32] = 2.0 ** -112
    x[0, 4, 0, 0], x[0, 4, 0, 1] = 3e38, -3e38
    x[0, 5, 0, 0] = 2.0 ** 122
    for dt in (torch.bfloat16, torch.float32):
        c = make_cache(gen(2), 1, 16, 1, 64, 16)
        pos = torch.arange(6, dtype=torch.int32, device=DEV)[None]
        dd.dllm_kv4_write(c, x.to(dt), x.to(dt), pos)
        ko, vo = torch.empty_like(x), torch.empty_like(x)
        dd.dllm_kv4_read(c, ko, vo, pos)
        for i in (0, 1, 2, 4):
            assert ko[0, i, 0, :32].isnan().all()
            assert torch.equal(ko[0, i, 0, 32:].double(), ref.quantised(x[0, i, 0, 32:]))  # its own group
        assert (ko[0, 3, 0, :32] == 0).all()
        assert abs(ko[0, 5, 0, 0].item() / 2.0 ** 122 - 1) < 0.1 and ko[0, 5, 0, 1:32].abs().max() == 0


def test_cache_skips_absent_pages_and_entries_beyond_the_table():
    g = gen(3)
    c = make_cache(g, 2, 64, 2, 64, 16)
    c.table[0, 1] = -1
    c.table[1, 2] = c.pages
    before = [t.clone() for t in (c.k_codes, c.k_params)]
    pos = torch.tensor([[16, 31, 64, 1 << 30], [32, 47, -5, -(1 << 31)]], dtype=torch.int32, device=DEV)
    x = randn(g, 2, 4, 2, 64)
    dd.dllm_kv4_write(c, x, x, pos)
    assert torch.equal(before[0], c.k_codes) and torch.equal(before[1], c.k_params)
    ko, vo = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    dd.dllm_kv4_read(c, ko, vo, pos)
    assert (ko == 0).all() and (vo == 0).all()


# ---------------------------------------------------------------- attention

def fill(g, c, T):
    """Random keys and values in all entries below T of every sequence; returns what they stand for."""
    B = c.table.shape[0]
    if T:
        k, v = (randn(g, B, T, c.heads, c.head_dim).to(torch.bfloat16) for _ in range(2))
        pos = torch.arange(T, dtype=torch.int32, device=DEV).repeat(B, 1)
        dd.dllm_kv4_write(c, k, v, pos)
    return entries(c, c.k_codes, c.k_params, T), entries(c, c.v_codes, c.v_params, T)


def seen_of(B, n, T, lens, mask, causal, c):
    j = torch.arange(T, device=DEV)
    last = torch.tensor([min(x, T) for x in lens], device=DEV)[:, None].expand(B, n)
    if causal:
        last = last - n + 1 + torch.arange(n, device=DEV)
    s = j < last[..., None]
    if mask is not None:
        s = s & (mask[:, None, :T] != 0)
    page = c.table.long()[:, j // c.page_size]
    return s & ((page >= 0) & (page < c.pages))[:, None]


def check_attention(out, lse, q, k, v, seen, scale):
    o, l, mag, top = ref.attention(q, k, v, seen, scale)
    assert not out.isnan().any()
    err = (out.double() - o).abs()
    tol = 2.0 ** -8 * 1.03 * (mag + o.abs())
    assert (err <= tol + 1e-30).all(), (err / (tol + 1e-30)).max().item()
    none = ~seen.any(-1)[:, None].expand_as(lse)
    assert (lse[none] == -math.inf).all() and (out.permute(0, 2, 1, 3)[none] == 0).all()
    if (~none).any():
        d, ll = (lse.double() - l).abs()[~none], l[~none]
        assert (d <= 1e-5 * ll.abs().clamp(min=1) + 2.0 ** -20 * top[~none]).all(), d.max().item()


def run(c, q, lens, T, causal=False, mask=None, scale=None, lse=True, out=None, ws=None, stream=None):
    B, n, H, _ = q.shape
    out = torch.full_like(q, 9.0, memory_format=torch.contiguous_format) if out is None else out
    l = torch.full((B, H, n), 9.0, device=DEV) if lse else None
    if ws is None:
        ws = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(c, B, n, H, T))
        ws[256:] = 255  # nothing but the status word has to be initialised
    ld = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    dd.dllm_attention_kv4(q, c, ld, T, out, ws, lse=l, key_mask=mask, scale=scale, causal=causal,
                          stream=stream)
    assert dd.dllm_get_status(ws, stream) == dd.DLLM_OK
    return out, l


SHAPES = [  # B, n, Hkv, G, D, page, T, lens
    (1, 1, 1, 1, 64, 16, 1, None), (1, 1, 2, 1, 128, 16, 17, None), (2, 1, 2, 3, 128, 64, 300, [300, 7]),
    (1, 1, 1, 8, 128, 48, 1000, None), (3, 1, 2, 5, 64, 16, 130, [0, 130, 64]),
    (1, 1, 1, 16, 256, 16, 200, None), (2, 2, 1, 7, 192, 32, 333, [333, 100]),
    (1, 1, 4, 4, 128, 256, 5000, None), (2, 1, 1, 20, 128, 16, 257, [257, 256]),
    (1, 32, 1, 1, 128, 64, 96, None), (2, 33, 3, 1, 64, 16, 200, [200, 150]),
    (1, 32, 2, 4, 128, 64, 1056, None), (2, 64, 1, 8, 128, 16, 500, [500, 437]),
    (1, 7, 1, 19, 128, 48, 129, None), (1, 17, 2, 5, 64, 64, 1000, None),
    (1, 40, 1, 3, 256, 64, 260, None), (1, 129, 1, 2, 128, 32, 640, None),
    (1, 300, 2, 1, 64, 64, 300, None), (2, 16, 1, 4, 192, 16, 90, [90, 16]),
    (1, 64, 1, 1, 128, 16, 127, None), (1, 1, 1, 1, 128, 16, 0, None), (2, 40, 1, 2, 64, 16, 0, None)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,n,H,G,D,ps,T,lens", SHAPES)
def test_attention(B, n, H, G, D, ps, T, lens, masked, causal):
    g = gen(n * 7 + T + D)
    c = make_cache(g, B, T, H, D, ps)
    k, v = fill(g, c, T)
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    mask = None
    if masked:
        mask = (torch.rand(B, T + 5, device=DEV, generator=g) < 0.6).to(torch.uint8) * 3
        mask[B - 1, : T // 2] = 0
    out, lse = run(c, q, lens, T, causal, mask)
    seen = seen_of(B, n, T, lens or [T] * B, mask, causal, c)
    check_attention(out, lse, q, k, v, seen, D ** -0.5)


@pytest.mark.parametrize("n,G", [(1, 4), (32, 4), (48, 1)])
def test_attention_masked_entries_may_hold_anything(n, G):
    # hidden by mask, by length, by an absent page: NaN steps and random codes there never matter
    g = gen(77)
    B, H, D, ps, T = 3, 2, 128, 16, 200
    c = make_cache(g, B, T, H, D, ps)  # params random: NaN and infinite steps in what is not written
    k, v = (randn(g, B, T, H, D).to(torch.bfloat16) for _ in range(2))
    mask = (torch.rand(B, T, device=DEV, generator=g) < 0.5).to(torch.uint8)
    mask[2] = 0  # sees nothing at all
    lens = [150, 200, 200]
    c.table[1, 3] = -1
    c.table[1, 5] = c.pages + 7
    pos = torch.arange(T, dtype=torch.int32, device=DEV).repeat(B, 1)
    pos[mask == 0] = -1
    pos[0, 150:] = -1
    c.k_params.fill_(0x7FE5)
    c.v_params.fill_(0x7FE5)
    dd.dllm_kv4_write(c, k, v, pos)
    seen = seen_of(B, n, T, lens, mask, False, c)
    q = (1.5 * randn(g, B, n, H * G, D)).to(torch.bfloat16)
    out, lse = run(c, q, lens, T, False, mask)
    table = c.table.clone()
    c.table.clamp_(0, c.pages - 1)
    kk, vv = entries(c, c.k_codes, c.k_params, T), entries(c, c.v_codes, c.v_params, T)
    c.table.copy_(table)
    check_attention(out, lse, q, kk, vv, seen, D ** -0.5)


@pytest.mark.parametrize("n,T,lens", [(1, 64, [1, 0]), (33, 64, [2, 40]), (80, 50, [50, 3])])
def test_attention_causal_rows_before_the_first_entry_see_nothing(n, T, lens):
    # more queries than entries: the first ones see nothing
    g = gen(n)
    c = make_cache(g, 2, T, 1, 128, 16)
    k, v = fill(g, c, T)
    q = randn(g, 2, n, 2, 128).to(torch.bfloat16)
    out, lse = run(c, q, lens, T, True)
    check_attention(out, lse, q, k, v, seen_of(2, n, T, lens, None, True, c), 128 ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_lengths_beyond_the_bound_are_cut(n):
    g = gen(8)
    c = make_cache(g, 2, 128, 2, 64, 16)
    k, v = fill(g, c, 128)
    q = randn(g, 2, n, 4, 64).to(torch.bfloat16)
    out, lse = run(c, q, [1 << 30, -3], 100)
    check_attention(out, lse, q, k[:, :100], v[:, :100], seen_of(2, n, 100, [100, 0], None, False, c), 0.125)


@pytest.mark.parametrize("n,G", [(1, 2), (48, 2)])
def test_attention_large_scores(n, G):
    # scores of several hundred: the running maximum keeps every exponential in range
    g = gen(9)
    c = make_cache(g, 1, 400, 1, 128, 64)
    k, v = fill(g, c, 400)
    for factor in (30.0, -30.0):
        q = (factor * randn(g, 1, n, G, 128)).to(torch.bfloat16)
        out, lse = run(c, q, None, 400)
        check_attention(out, lse, q, k, v, seen_of(1, n, 400, [400], None, False, c), 128 ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("layout", ["packed", "heads_first", "odd"])
def test_attention_strided_queries_and_outputs(n, layout):
    g = gen(10)
    c = make_cache(g, 2, 150, 2, 128, 16)
    k, v = fill(g, c, 150)
    q = randn(g, 2, n, 6, 128).to(torch.bfloat16)
    out = strided(torch.zeros_like(q), layout)
    mask = torch.ones(2, 333, dtype=torch.bool, device=DEV)[:, 3:]
    mask[0, 20:40] = False
    _, lse = run(c, strided(q, layout), None, 150, mask=mask, out=out, scale=0.2)
    check_attention(out, lse, q, k, v, seen_of(2, n, 150, [150] * 2, mask, False, c), 0.2)
    plain, _ = run(c, q, None, 150, mask=mask, scale=0.2, lse=False)
    assert torch.equal(plain, out)


@pytest.mark.parametrize("n,H,G,T", [(1, 4, 4, 3000), (64, 1, 4, 1500), (24, 2, 1, 2000)])
def test_attention_repeats_bit_for_bit_on_any_stream(n, H, G, T):
    g = gen(11)
    c = make_cache(g, 2, T, H, 128, 64)
    fill(g, c, T)
    q = randn(g, 2, n, H * G, 128).to(torch.bfloat16)
    first, l0 = run(c, q, [T, T - 77], T)
    ws = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(c, 2, n, H * G, T))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (None, side, None):
        out, l1 = run(c, q, [T, T - 77], T, ws=ws, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(l0, l1)


@pytest.mark.parametrize("n", [1, 64])
def test_cache_larger_than_32_bit_offsets(n):
    # a pool of 5.4 GB of codes: the pages used lie beyond 2^32 bytes
    pages, H, ps, D, T = 41000, 8, 256, 128, 600
    c = dd.Kv4Cache(pages, H, ps, D, 1, 3)
    assert c.k_codes.numel() > 1 << 32
    c.table.copy_(torch.tensor([[pages - 1, pages - 4000, pages - 2]], dtype=torch.int32))
    g = gen(12)
    x = randn(g, 1, T, H, D).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[None]
    dd.dllm_kv4_write(c, x, -x, pos)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    dd.dllm_kv4_read(c, ko, vo)
    assert torch.equal(ko.double(), ref.quantised(x)) and torch.equal(vo.double(), ref.quantised(-x))
    q = randn(g, 1, n, H, D).to(torch.bfloat16)
    out, lse = run(c, q, None, T)
    check_attention(out, lse, q, ko, vo, torch.ones(1, n, T, dtype=torch.bool, device=DEV), D ** -0.5)


def test_operators_captured_in_a_graph():
    g = gen(13)
    B, n, H, G, D, T = 2, 8, 2, 2, 128, 100
    c = make_cache(g, B, T, H, D, 16)
    fill(g, c, T)
    qkv = randn(g, B, n, H * G + 2 * H, D).to(torch.bfloat16)
    q, k, v = qkv[:, :, :H * G], qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:]
    pos = torch.arange(50, 50 + n, dtype=torch.int32, device=DEV).repeat(B, 1)
    ph = phases(D)
    qo, out = (torch.zeros(B, n, H * G, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ko = torch.zeros(B, n, H, D, dtype=torch.bfloat16, device=DEV)
    ws = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(c, B, n, H * G, T))

    def step():
        dd.dllm_qk_norm_rope(q, k, qo, ko, pos, ph)
        dd.dllm_kv4_write(c, ko, v, pos)
        dd.dllm_attention_kv4(qo, c, None, T, out, ws)

    step()
    torch.cuda.synchronize()
    eager = out.clone()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    qkv.mul_(0.5)
    q2 = q.clone()
    graph.replay()
    torch.cuda.synchronize()
    o, _ = ref.norm_rope(q2, pos, ref.frequencies(D, 10000.0), None, 1e-6, False)
    assert (qo.double() - o).abs().max() < 2.0 ** -6

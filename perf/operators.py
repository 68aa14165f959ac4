"""What the operators behind the KV refresh are measured on.

After a decode iteration the cache entries that `dllm_kv_refresh_mask` lists are recomputed: the
new keys (and the block's queries) are normalised per head and rotated to their positions, keys
and values are stored in a cache of 4-bit codes, and the block's queries attend over that cache.
Each case is one such operator at one size; `run` computes it in elementary torch operations, or
with `own` set through the library.

Cache format (see include/dllm.h): 32 channels of one token of one head share a step s (three
significant bits) and a zero point z; a code n in 0..15 stands for s * (n - z), which bf16 holds
exactly.  Codes: [pages, heads, page_size, head_dim / 2] bytes, low nibble first; params:
[pages, heads, page_size, head_dim / 32] words of 16 bits, bf16(s) with z in its low four bits.
"""
import math

import numpy as np
import torch

own = False

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    rope = {"op": "norm_rope", "interleaved": False, "packed": True, "dtype": "bf16",
            "base": 10000.0, "factor": 1.0}
    cache = {"op": "cache", "dtype": "bf16"}
    attn = {"op": "attention", "ragged": 0.0, "causal": False, "masked": False}
    return [
        # one new token of one sequence, 2048 channels in 16 heads: a plain decode step
        {"name": "rope_token", **rope, "B": 1, "n": 1, "q_heads": 16, "k_heads": 4,
         "head_dim": 128, "rotary_dim": 128, "start": 1024},
        # odd sizes in fp32: 80 channels of which 32 turn, pairs side by side, unpacked tensors
        {"name": "rope_odd", **rope, "B": 3, "n": 333, "q_heads": 7, "k_heads": 7,
         "head_dim": 80, "rotary_dim": 32, "interleaved": True, "packed": False, "dtype": "f32",
         "start": 5},
        # a whole prompt late in a long context, positions scaled, out of one packed projection
        {"name": "rope_prompt", **rope, "B": 2, "n": 8192, "q_heads": 32, "k_heads": 8,
         "head_dim": 128, "rotary_dim": 128, "start": 57000, "base": 500000.0, "factor": 8.0},
        # a refresh: 72 of the 1024 + 64 entries of each of 16 sequences, written and read back
        {"name": "cache_refresh", **cache, "B": 16, "n": 72, "heads": 4, "head_dim": 128,
         "page_size": 64, "length": 1088},
        # the prefix of 8 sequences as it first enters the cache
        {"name": "cache_prompt", **cache, "B": 8, "n": 4096, "heads": 8, "head_dim": 128,
         "page_size": 64, "length": 4096},
        # single tokens: one short sequence (latency), a ragged batch, one long context
        {"name": "token_short", **attn, "B": 1, "n": 1, "q_heads": 16, "kv_heads": 4,
         "head_dim": 128, "page_size": 64, "length": 331},
        {"name": "token_batch", **attn, "B": 32, "n": 1, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page_size": 64, "length": 8192, "ragged": 0.5},
        {"name": "token_long", **attn, "B": 1, "n": 1, "q_heads": 32, "kv_heads": 4,
         "head_dim": 128, "page_size": 256, "length": 65536},
        # blocks being decoded see their prefix and all of the block: 32 x 32 and 16 x 64 positions
        {"name": "block_32", **attn, "B": 32, "n": 32, "q_heads": 16, "kv_heads": 4,
         "head_dim": 128, "page_size": 64, "length": 1056},
        {"name": "block_64", **attn, "B": 16, "n": 64, "q_heads": 16, "kv_heads": 2,
         "head_dim": 128, "page_size": 64, "length": 4160},
        # odd sizes: small pages, a key mask that leaves one sequence nothing, no shared heads
        {"name": "block_odd", **attn, "B": 3, "n": 33, "q_heads": 6, "kv_heads": 6,
         "head_dim": 64, "page_size": 16, "length": 777, "ragged": 0.6, "masked": True},
        # a piece of a long prompt, causal, ragged
        {"name": "prompt_piece", **attn, "B": 2, "n": 1024, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page_size": 64, "length": 16384, "ragged": 0.2, "causal": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.25:
        B, D = rng.choice([1, 2, 3, 8, 32]), rng.choice([64, 80, 96, 128, 128, 256])
        kh = rng.randint(1, 8)
        qh = kh * rng.choice([1, 2, 3, 4])
        n = _log(rng, 1, max(1, min(8192, (16384 * 40 * 128) // (B * (qh + kh) * D))))
        rot = rng.choice([D, D, D // 2, 32])
        return {"op": "norm_rope", "B": B, "n": n, "q_heads": qh, "k_heads": kh, "head_dim": D,
                "rotary_dim": rot, "interleaved": rng.random() < 0.4, "packed": rng.random() < 0.6,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "base": rng.choice([1e4, 5e5]),
                "factor": rng.choice([1.0, 4.0]), "start": _log(rng, 1, 8000)}
    if kind < 0.45:
        B, D, H = rng.choice([1, 2, 3, 8, 32]), rng.choice([64, 96, 128, 128, 256]), rng.randint(1, 8)
        length = _log(rng, 8, min(8192, (8 * 4096 * 8 * 128) // (B * H * D)))
        return {"op": "cache", "B": B, "n": _log(rng, 1, length), "heads": H, "head_dim": D,
                "page_size": rng.choice([16, 32, 48, 64, 256]), "length": length,
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    D = rng.choice([64, 128, 128, 128, 256])
    kh, g = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 7, 8])
    kind = rng.choice(["token", "token", "block", "block", "piece"])
    n = 1 if kind == "token" else _log(rng, 2, 128) if kind == "block" else _log(rng, 128, 1024)
    B = rng.choice([1, 2, 3, 8, 32]) if kind != "piece" else rng.choice([1, 2])
    most = min(65536, int(32 * 8 * 8192 * 128 / (B * kh * D)),
               int(2 ** 30 * 128 / (B * kh * g * n * D)))
    length = _log(rng, max(n, 16), max(n, 16, most))
    return {"op": "attention", "B": B, "n": n, "q_heads": kh * g, "kv_heads": kh, "head_dim": D,
            "page_size": rng.choice([16, 48, 64, 256]), "length": length,
            "ragged": rng.choice([0.0, 0.0, 0.5, 0.9]) if length > 4 * n else 0.0,
            "causal": kind == "piece" or rng.random() < 0.2, "masked": rng.random() < 0.3}


def _lengths(c):
    """Entries of each sequence: spread over the last `ragged` part of the full length."""
    spread = c["ragged"] * (c["length"] - c["n"])
    return [c["length"] - int(spread * ((0.618034 * b) % 1.0)) for b in range(c["B"])]


def work(c):
    B, n = c["B"], c["n"]
    if c["op"] == "norm_rope":
        D, heads, es = c["head_dim"], c["q_heads"] + c["k_heads"], 2 if c["dtype"] == "bf16" else 4
        values = B * n * heads * D
        return {"bytes": 2 * values * es + 4 * B * n + 2 * es * D + 4 * c["rotary_dim"],
                "flops": values * 4 + B * n * heads * c["rotary_dim"] * 3}
    if c["op"] == "cache":
        es = 2 if c["dtype"] == "bf16" else 4
        values = 2 * B * n * c["heads"] * c["head_dim"]
        # each input read once, the cache entries written once, the values written once
        return {"bytes": values * (2 * es + 9 / 16) + 4 * B * n, "flops": values * 8}
    D, total = c["head_dim"], sum(_lengths(c))
    pairs = n * total - (B * n * (n - 1) // 2 if c["causal"] else 0)
    return {"bytes": total * c["kv_heads"] * 2 * (D * 9 // 16) + (total if c["masked"] else 0)
            + 4 * B * n * c["q_heads"] * (D + 1), "flops": 4 * D * c["q_heads"] * pairs}


# ---------------------------------------------------------------- the cache format, in 32 bits

def quantise(x):
    """Codes [..., D / 2] (uint8) and params [..., D / 32] (int16) of x [..., D] (fp32)."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    s = (hi - lo) / torch.full_like(hi, 15.0)  # a true division: by a number it is a product
    s = torch.where(s < 2.0 ** -110, 0.0, s)
    s = ((s.view(torch.int32) + 0x1FFFFF) & ~0x1FFFFF).view(torch.float32)  # up to 3 bits
    inv = torch.where(s > 0, s, 1.0)
    z = torch.floor(-lo / inv + 0.5).clamp(0, 15)
    r = g / inv.unsqueeze(-1)
    r = torch.where(s.unsqueeze(-1) > 0, torch.sign(r) * torch.floor(r.abs() + 0.5), 0.0)
    n = (r + z.unsqueeze(-1)).clamp(0, 15).to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    params = (s.view(torch.int32) >> 16) | z.to(torch.int32)
    return n[..., 0] | (n[..., 1] << 4), params.to(torch.int16)


def dequantise(codes, params):
    """The values [..., D] (fp32) that codes and params stand for."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.float32)
    p = params.to(torch.int32)
    s, z = ((p & 0x7FE0) << 16).view(torch.float32), (p & 15).to(torch.float32)
    return ((n.unflatten(-1, (-1, GROUP)) - z.unsqueeze(-1)) * s.unsqueeze(-1)).flatten(-2)


def _frequencies(c):
    i = np.arange(c["rotary_dim"] // 2, dtype=np.float64)
    return c["base"] ** (-2.0 * i / c["rotary_dim"]) / c["factor"]


# ---------------------------------------------------------------- inputs

def _pages(B, length, page_size, g, dev):
    """A page table [B, pages of a sequence] in no order, and the number of pages (one is spare)."""
    per = -(-length // page_size)
    order = torch.randperm(B * per, generator=g, device=dev).to(torch.int32)
    return order.view(B, per).contiguous(), B * per + 1


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device=dev, generator=g)  # noqa: E731
    B, n, D = c["B"], c["n"], c["head_dim"]
    st = {"case": c}
    if c["op"] == "norm_rope":
        dt, qh, kh = DTYPES[c["dtype"]], c["q_heads"], c["k_heads"]
        if c["packed"]:  # queries, keys and values of one projection side by side
            qkv = (rand(B, n, qh + 2 * kh, D) * 1.7).to(dt)
            st["q"], st["k"] = qkv[:, :, :qh], qkv[:, :, qh:qh + kh]
        else:
            st["q"], st["k"] = (rand(B, n, qh, D) * 1.7).to(dt), (rand(B, n, kh, D) * 1.7).to(dt)
        st["q_weight"], st["k_weight"] = ((1 + 0.2 * rand(D)).to(dt) for _ in range(2))
        first = torch.randint(0, c["start"] + 1, (B, 1), generator=g, device=dev)
        st["pos"] = (first + torch.arange(n, device=dev)).to(torch.int32).contiguous()
        # fraction of a turn per position, in 2^-64 turns
        turns = np.round(_frequencies(c) / (2 * math.pi) * 2.0 ** 64).astype(np.int64)
        st["phases"] = torch.from_numpy(turns).to(dev)
        st["q_out"] = torch.zeros(B, n, qh, D, dtype=dt, device=dev)
        st["k_out"] = torch.zeros(B, n, kh, D, dtype=dt, device=dev)
        return st
    ps = c["page_size"]
    st["table"], pages = _pages(B, c["length"], ps, g, dev)
    if c["op"] == "cache":
        dt, H = DTYPES[c["dtype"]], c["heads"]
        channel = torch.exp(0.5 * rand(H, D))  # some channels of a head are larger than others
        st["k"], st["v"] = (rand(B, n, H, D) * channel).to(dt), rand(B, n, H, D).to(dt)
        rank = torch.rand(B, c["length"], device=dev, generator=g).argsort(1)[:, :n]
        pos = rank.sort(1).values.to(torch.int32)
        if n > 8 and n < c["length"]:  # a refresh list ends in -1 where fewer entries changed
            pos[:, n - n // 8:] = -1
        st["pos"] = pos.contiguous()
        st["k_codes"], st["v_codes"] = (torch.zeros(pages, H, ps, D // 2, dtype=torch.uint8, device=dev)
                                        for _ in range(2))
        st["k_params"], st["v_params"] = (torch.zeros(pages, H, ps, D // GROUP, dtype=torch.int16, device=dev)
                                          for _ in range(2))
        st["k_out"], st["v_out"] = (torch.zeros(B, n, H, D, dtype=dt, device=dev) for _ in range(2))
    else:
        kh = c["kv_heads"]
        # queries and keys are normalised (unit mean square); sharper queries than a flat softmax
        st["q"] = (1.5 * rand(B, n, c["q_heads"], D)).to(torch.bfloat16)
        st["k_codes"], st["k_params"] = quantise(rand(pages, kh, ps, D))
        st["v_codes"], st["v_params"] = quantise(rand(pages, kh, ps, D))
        st["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
        st["key_mask"] = None
        if c["masked"]:
            st["key_mask"] = (torch.rand(B, c["length"], device=dev, generator=g) < 0.8).to(torch.uint8)
            if B > 1:
                st["key_mask"][1] = 0  # a sequence that sees nothing
        st["scale"] = D ** -0.5
        st["out"] = torch.zeros(B, n, c["q_heads"], D, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(B, c["q_heads"], n, dtype=torch.float32, device=dev)
    return st


# ---------------------------------------------------------------- plain forms

def _norm_rope_one(x, weight, cos, sin, c):
    x = x.to(torch.float32)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.to(torch.float32)
    R = c["rotary_dim"]
    r = y[..., :R]
    r = r.unflatten(-1, (-1, 2)) if c["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
    a, b = r[..., 0], r[..., 1]
    r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1)
    r = r.flatten(-2) if c["interleaved"] else r.transpose(-1, -2).flatten(-2)
    return torch.cat((r, y[..., R:]), -1)


def _plain_norm_rope(st):
    c, dt = st["case"], st["q"].dtype
    phase = (st["pos"].to(torch.int64).unsqueeze(-1) * st["phases"]) >> 32  # 2^-32 turns, wrapped
    angle = phase.to(torch.float32) * (2 * math.pi / 2.0 ** 32)
    cos, sin = torch.cos(angle).unsqueeze(2), torch.sin(angle).unsqueeze(2)
    return {"q": _norm_rope_one(st["q"], st["q_weight"], cos, sin, c).to(dt),
            "k": _norm_rope_one(st["k"], st["k_weight"], cos, sin, c).to(dt)}


def _plain_cache(st):
    ps, pos = st["case"]["page_size"], st["pos"].to(torch.int64)
    spare = st["k_codes"].shape[0] - 1
    page = torch.gather(st["table"].to(torch.int64), 1, (pos // ps).clamp(min=0))
    page, slot = torch.where(pos >= 0, page, spare), pos.clamp(min=0) % ps
    out = {}
    for x, dt in (("k", st["k"].dtype), ("v", st["v"].dtype)):
        codes, params = quantise(st[x].to(torch.float32))
        st[x + "_codes"][page, :, slot] = codes
        st[x + "_params"][page, :, slot] = params
        back = dequantise(st[x + "_codes"][page, :, slot], st[x + "_params"][page, :, slot])
        out[x] = torch.where((pos >= 0)[..., None, None], back, 0.0).to(dt)
    return out


def _plain_attention(st):
    c, n = st["case"], st["case"]["n"]
    table = st["table"].to(torch.int64)
    k, v = (dequantise(st[x + "_codes"][table], st[x + "_params"][table])
            .transpose(1, 2).flatten(2, 3)[:, :, :c["length"]] for x in "kv")
    B, kh = k.shape[:2]
    q = st["q"].to(torch.float32).transpose(1, 2).reshape(B, kh, -1, c["head_dim"])
    j = torch.arange(c["length"], device=k.device)
    last = st["lens"].to(torch.int64)[:, None].expand(B, n)
    if c["causal"]:
        last = last - n + 1 + torch.arange(n, device=k.device)
    seen = j < last.unsqueeze(-1)
    if st["key_mask"] is not None:
        seen = seen & (st["key_mask"] != 0).unsqueeze(1)
    seen = seen.unsqueeze(1).unsqueeze(1)  # [B, 1, 1, n, length]
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).unflatten(2, (-1, n))
    s = s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, n))
    out = torch.where(total > 0, out / total, 0.0)
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": out.flatten(1, 2).transpose(1, 2).to(torch.bfloat16), "lse": lse.flatten(1, 2)}


# ---------------------------------------------------------------- the library's operators

def _own_norm_rope(st):
    import diffusion_decoding_gb300 as dd
    c = st["case"]
    dd.dllm_qk_norm_rope(st["q"], st["k"], st["q_out"], st["k_out"], st["pos"], st["phases"],
                         q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6,
                         interleaved=c["interleaved"])
    return {"q": st["q_out"], "k": st["k_out"]}


def _handle(st):
    """The cache's descriptor (and the attention's workspace): made once, kept with the cache."""
    import diffusion_decoding_gb300 as dd
    c = st["case"]
    st["cache"] = dd.Kv4Cache.of(st["k_codes"], st["k_params"], st["v_codes"], st["v_params"],
                                 st["table"])
    if c["op"] == "attention":
        st["ws"] = dd.workspace(dd.dllm_attention_kv4_workspace_bytes(
            st["cache"], c["B"], c["n"], c["q_heads"], c["length"]))


def _own_cache(st):
    import diffusion_decoding_gb300 as dd
    if "cache" not in st:
        _handle(st)
    dd.dllm_kv4_write(st["cache"], st["k"], st["v"], st["pos"])
    dd.dllm_kv4_read(st["cache"], st["k_out"], st["v_out"], st["pos"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_attention(st):
    import diffusion_decoding_gb300 as dd
    c = st["case"]
    if "cache" not in st:
        _handle(st)
    dd.dllm_attention_kv4(st["q"], st["cache"], st["lens"], c["length"], st["out"], st["ws"],
                          lse=st["lse"], key_mask=st["key_mask"], scale=st["scale"],
                          causal=c["causal"])
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "cache": _own_cache, "attention": _own_attention}[op](state)
    return {"norm_rope": _plain_norm_rope, "cache": _plain_cache, "attention": _plain_attention}[op](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm_rope(st, c):
    angle = st["pos"].double().unsqueeze(-1) * torch.from_numpy(_frequencies(c)).to(st["pos"].device)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(2)
    R, out = c["rotary_dim"], {}
    for x in "qk":
        y = st[x].double()
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["head_dim"] + 1e-6) * st[x + "_weight"].double()
        first, second = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
        both = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = both.real, both.imag
        out[x] = y
    return out


def _exact_cache(st, c):
    out = {}
    for x in "kv":
        groups = st[x].double().reshape(-1, GROUP)
        zero = torch.zeros_like(groups[:, :1])
        lo = torch.cat((groups, zero), 1).min(1, keepdim=True).values
        hi = torch.cat((groups, zero), 1).max(1, keepdim=True).values
        part, power = torch.frexp((hi - lo) / 15)
        step = torch.ceil(part * 8) / 8 * torch.exp2(power.double())
        safe = torch.where(step == 0, torch.ones_like(step), step)
        z = torch.floor(-lo / safe + 0.5)
        near = torch.copysign(torch.floor((groups / safe).abs() + 0.5), groups)
        value = (torch.minimum(torch.maximum(near + z, torch.zeros_like(z)), torch.full_like(z, 15)) - z) * step
        out[x] = value.reshape(st[x].shape) * (st["pos"] >= 0)[:, :, None, None]
    return out


def _exact_values(codes, params):
    word = params.long()
    exponent, mantissa, z = word // 128, word % 128 // 32, word % 16  # bf16(s): 8 + 7 bits
    step = torch.where(word < 32, 0.0, (1 + mantissa.double() / 4) * torch.exp2(exponent.double() - 127))
    pair = codes.long().unsqueeze(-1)
    n = torch.cat((pair % 16, pair // 16), -1).reshape(*codes.shape[:-1], -1, GROUP)
    return ((n - z.unsqueeze(-1)).double() * step.unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _exact_attention(st, c):
    if work(c)["flops"] > 4e12:
        return None
    n, G = c["n"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(c["B"], n, c["q_heads"], c["head_dim"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["q_heads"], n), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(_lengths(c)):
        at = torch.arange(length, device="cuda")
        page, slot = st["table"][b].long()[at // c["page_size"]], at % c["page_size"]
        hidden = torch.zeros(n, length, dtype=torch.bool, device="cuda")
        if st["key_mask"] is not None:
            hidden |= st["key_mask"][b, :length] == 0
        if c["causal"]:
            hidden |= at > length - n + torch.arange(n, device="cuda")[:, None]
        for h in range(c["kv_heads"]):
            k = _exact_values(st["k_codes"][page, h, slot], st["k_params"][page, h, slot])
            v = _exact_values(st["v_codes"][page, h, slot], st["v_params"][page, h, slot])
            for i in range(h * G, (h + 1) * G):
                s = (st["q"][b, :, i].double() @ k.T) * st["scale"]
                s[hidden] = -math.inf
                total = torch.logsumexp(s, 1)
                lse[b, i] = total
                some = total > -math.inf
                out[b, some, i] = torch.exp(s[some] - total[some, None]) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "cache": _exact_cache,
            "attention": _exact_attention}[case["op"]](st, case)

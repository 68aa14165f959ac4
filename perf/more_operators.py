"""What the operators of a sampled decode loop over a bounded cache are measured on.

A decode step that samples draws each open position's token from the filtered distribution of its
logits (`sample`); a loop that keeps its cache within a budget adds up how much attention every
entry received (`weights`) and now and then drops the entries that received least (`evict`).  Each
case is one such operator at one size; `run` computes it in elementary torch operations, or with
`own` set through the library.

The cache holds 4-bit codes in pages (see include/dllm.h): 32 channels of one token of one head
share a step s (three significant bits) and a zero point z; a code n stands for s * (n - z).  Codes:
[pages, heads, page_size, head_dim / 2] bytes, low nibble first; params: [pages, heads, page_size,
head_dim / 32] words of 16 bits, bf16(s) with z in its low four bits.
"""
import math

import torch

own = False

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    sample = {"op": "sample", "dtype": "bf16", "top_k": 0, "top_p": 1.0, "min_p": 0.0,
              "open": 1.0, "pad": 0, "sure": 0.0}
    weights = {"op": "weights", "ragged": 0.0, "causal": False, "masked": False, "keep": 0.0}
    evict = {"op": "evict", "ragged": 0.0, "first": 4, "last": 32}
    return [
        # one short block with a small vocabulary: latency
        {"name": "sample_step", **sample, "B": 1, "L": 32, "V": 4096, "dtype": "f32",
         "temperature": 1.0, "top_k": 50, "top_p": 0.95},
        # one block of one sequence, the usual filters of a chat request
        {"name": "sample_block", **sample, "B": 1, "L": 32, "V": 126464, "temperature": 0.8,
         "top_k": 40, "top_p": 0.95},
        # a full batch with a nucleus only: where the model is unsure it holds much of the vocabulary
        {"name": "sample_nucleus", **sample, "B": 32, "L": 32, "V": 126464, "temperature": 0.7,
         "top_p": 0.9},
        # a full batch, the whole distribution at a temperature
        {"name": "sample_whole", **sample, "B": 16, "L": 64, "V": 126464, "temperature": 0.7},
        # odd sizes in fp32, rows on no boundary, half of the positions decided already
        {"name": "sample_odd", **sample, "B": 3, "L": 21, "V": 50257, "dtype": "f32",
         "temperature": 1.3, "min_p": 0.05, "open": 0.5, "pad": 6},
        # single tokens of a ragged batch, added to what earlier steps left
        {"name": "weights_token", **weights, "B": 32, "n": 1, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page_size": 64, "length": 8192, "ragged": 0.5, "keep": 1.0},
        # blocks of 64 positions over prefix and block
        {"name": "weights_block", **weights, "B": 16, "n": 64, "q_heads": 16, "kv_heads": 2,
         "head_dim": 128, "page_size": 64, "length": 4160, "keep": 0.9},
        # odd sizes: small pages, a key mask that hides one sequence whole, no shared heads
        {"name": "weights_odd", **weights, "B": 3, "n": 33, "q_heads": 6, "kv_heads": 6,
         "head_dim": 64, "page_size": 16, "length": 777, "ragged": 0.6, "masked": True},
        # a piece of a long prompt, causal, ragged: what its entries received from it
        {"name": "weights_piece", **weights, "B": 2, "n": 1024, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page_size": 64, "length": 16384, "ragged": 0.2, "causal": True},
        # one short sequence cut to a budget: latency
        {"name": "evict_single", **evict, "B": 1, "kv_heads": 4, "head_dim": 128, "page_size": 64,
         "length": 331, "budget": 256},
        # a ragged batch cut to half its longest
        {"name": "evict_batch", **evict, "B": 32, "kv_heads": 8, "head_dim": 128, "page_size": 64,
         "length": 8192, "budget": 4096, "ragged": 0.5},
        # one long context cut to a quarter
        {"name": "evict_long", **evict, "B": 1, "kv_heads": 4, "head_dim": 128, "page_size": 256,
         "length": 65536, "budget": 16384},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.4:
        V = _log(rng, 1000, 160000)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 1024 * 126464 // (V if dtype == "bf16" else 2 * V)
        rows = _log(rng, 1, min(1024, most))
        L = min(rows, rng.choice([1, 7, 32, 64]))
        return {"op": "sample", "B": rows // L, "L": L, "V": V, "dtype": dtype,
                "temperature": rng.choice([0.3, 0.7, 1.0, 1.0, 1.5]),
                "top_k": rng.choice([0, 0, 1, 20, 50, 200, 900]),
                "top_p": rng.choice([1.0, 1.0, 0.95, 0.9, 0.5]),
                "min_p": rng.choice([0.0, 0.0, 0.02, 0.1]), "open": rng.choice([1.0, 1.0, 0.4]),
                "pad": rng.choice([0, 0, 8, 3]), "sure": rng.choice([-1.0, 0.0, 0.0, 3.0])}
    if kind < 0.75:
        D = rng.choice([64, 128, 128, 128, 256])
        kh, g = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 7, 8])
        kind = rng.choice(["token", "token", "block", "block", "piece"])
        n = 1 if kind == "token" else _log(rng, 2, 128) if kind == "block" else _log(rng, 128, 1024)
        B = rng.choice([1, 2, 3, 8, 32]) if kind != "piece" else rng.choice([1, 2])
        most = min(65536, int(32 * 8 * 8192 * 128 / (B * kh * D)),
                   int(2 ** 30 * 128 / (B * kh * g * n * D)))
        length = _log(rng, max(n, 16), max(n, 16, most))
        return {"op": "weights", "B": B, "n": n, "q_heads": kh * g, "kv_heads": kh, "head_dim": D,
                "page_size": rng.choice([16, 48, 64, 256]), "length": length,
                "ragged": rng.choice([0.0, 0.0, 0.5, 0.9]) if length > 4 * n else 0.0,
                "causal": kind == "piece" or rng.random() < 0.2, "masked": rng.random() < 0.3,
                "keep": rng.choice([0.0, 0.9, 1.0])}
    B, D, kh = rng.choice([1, 1, 2, 3, 8, 32]), rng.choice([64, 96, 128, 128, 256]), rng.randint(1, 8)
    length = _log(rng, 64, min(65536, int(32 * 8 * 8192 * 128 / (B * kh * D))))
    budget = max(16, int(length * rng.uniform(0.1, 0.95)))
    return {"op": "evict", "B": B, "kv_heads": kh, "head_dim": D,
            "page_size": rng.choice([16, 48, 64, 256]), "length": length, "budget": budget,
            "ragged": rng.choice([0.0, 0.0, 0.5, 0.9]), "first": rng.choice([0, 1, 4]),
            "last": min(rng.choice([0, 7, 32]), budget // 4)}


def _lengths(c):
    """Entries of each sequence: spread over the last `ragged` part of the full length."""
    spread = c["ragged"] * (c["length"] - c.get("n", 16))
    return [c["length"] - int(spread * ((0.618034 * b) % 1.0)) for b in range(c["B"])]


def work(c):
    B = c["B"]
    if c["op"] == "sample":
        rows, es = int(B * c["L"] * c["open"]), 2 if c["dtype"] == "bf16" else 4
        return {"bytes": rows * c["V"] * es + B * c["L"] * 21, "flops": rows * c["V"] * 5}
    D, total = c["head_dim"], sum(_lengths(c))
    if c["op"] == "weights":
        n = c["n"]
        pairs = n * total - (B * n * (n - 1) // 2 if c["causal"] else 0)
        return {"bytes": total * c["kv_heads"] * (D * 9 // 16) + (total if c["masked"] else 0)
                + 4 * total * (2 if c["keep"] else 1) + B * n * c["q_heads"] * (2 * D + 4),
                "flops": (2 * D + 2) * c["q_heads"] * pairs}
    bytes_ = 0.0
    for length in _lengths(c):
        new, fixed = min(length, c["budget"]), c["first"] + c["last"]
        # entries beyond the new length that stay: the last ones, and their share of the others
        stay = (new - fixed) / max(1, length - fixed)
        moved = c["last"] + stay * max(0, length - new - c["last"]) if length > new else 0
        bytes_ += 2 * moved * c["kv_heads"] * 2 * (D * 9 // 16) + 8 * length + 4 * c["length"]
    return {"bytes": bytes_, "flops": total * 4}


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


# ---------------------------------------------------------------- inputs

def _pages(B, length, page_size, g, dev):
    """A page table [B, pages of a sequence] in no order, and the number of pages (one is spare)."""
    per = -(-length // page_size)
    order = torch.randperm(B * per, generator=g, device=dev).to(torch.int32)
    return order.view(B, per).contiguous(), B * per + 1


def _prepare_sample(c, g, dev):
    B, L, V = c["B"], c["L"], c["V"]
    R = B * L
    rand = lambda *shape: torch.rand(*shape, device=dev, generator=g)  # noqa: E731
    store = torch.empty(R, V + c["pad"], dtype=DTYPES[c["dtype"]], device=dev)
    # a bulk of N(0, 2) and a head of 64 tokens that falls off like 1 / rank^1.2; `sure` to
    # `sure` + 6 is the log of the first token's odds against the whole bulk
    z = 2.0 * torch.randn(R, V, device=dev, generator=g)
    first = math.log(V) + 2.0 + c["sure"] + 6.0 * rand(R, 1)
    head = min(64, V)
    rank = rand(R, head).argsort(1).to(torch.float32)
    at = torch.arange(head, device=dev) * (V // head)
    at = at + torch.randint(0, V // head, (R, head), generator=g, device=dev)
    z.scatter_(1, at, first - 1.2 * torch.log1p(rank) + 0.3 * torch.randn(R, head, device=dev, generator=g))
    store[:, :V] = z
    store[:, V:] = 50.0
    masked = (rand(R) < c["open"]).to(torch.uint8)
    masked[0] = 1
    return {"logits": store, "masked": masked, "uniform": rand(R)}


def _prepare_cache(c, g, dev):
    kh, D, ps = c["kv_heads"], c["head_dim"], c["page_size"]
    st = {}
    st["table"], pages = _pages(c["B"], c["length"], ps, g, dev)
    for x in "kv":
        st[x + "_codes"], st[x + "_params"] = quantise(
            torch.randn(pages, kh, ps, D, device=dev, generator=g))
    st["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
    return st


def _prepare_weights(c, g, dev):
    st = _prepare_cache(c, g, dev)
    B, n, D, length = c["B"], c["n"], c["head_dim"], c["length"]
    # queries and keys are normalised (unit mean square); sharper queries than a flat softmax
    st["q"] = (1.5 * torch.randn(B, n, c["q_heads"], D, device=dev, generator=g)).to(torch.bfloat16)
    st["key_mask"] = None
    if c["masked"]:
        st["key_mask"] = (torch.rand(B, length, device=dev, generator=g) < 0.8).to(torch.uint8)
        if B > 1:
            st["key_mask"][1] = 0  # a sequence that sees nothing
    st["scale"] = D ** -0.5
    st["prior"] = torch.rand(B, length, device=dev, generator=g) if c["keep"] else None
    st["weights"] = torch.zeros(B, length, device=dev)
    st["lse"] = torch.empty(B, c["q_heads"], n, device=dev)  # as the attention leaves it
    for b in range(B):
        s = _scores({**st, "case": {**c, "B": 1}, "q": st["q"][b:b + 1], "table": st["table"][b:b + 1],
                     "lens": st["lens"][b:b + 1],
                     "key_mask": None if st["key_mask"] is None else st["key_mask"][b:b + 1]})
        st["lse"][b] = torch.logsumexp(s, -1).flatten(0, 2)
    return st


def _prepare_evict(c, g, dev):
    st = _prepare_cache(c, g, dev)
    B, length = c["B"], c["length"]
    # attention received: over several orders of magnitude, and nothing for one entry in twenty
    w = torch.exp(1.5 * torch.randn(B, length, device=dev, generator=g))
    st["weights"] = w * (torch.rand(B, length, device=dev, generator=g) > 0.05)
    st["slots"] = torch.zeros(B, length, dtype=torch.int32, device=dev)
    st["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    st["new_weights"] = torch.zeros(B, length, device=dev)
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    make = {"sample": _prepare_sample, "weights": _prepare_weights, "evict": _prepare_evict}
    return {"case": case, **make[case["op"]](case, g, dev)}


# ---------------------------------------------------------------- plain forms

def _f32(x):
    """A parameter as the library receives it."""
    return float(torch.tensor(x, dtype=torch.float32))


def _plain_sample(st):
    c = st["case"]
    V, T = c["V"], _f32(c["temperature"])
    z = st["logits"][:, :V].to(torch.float32)
    m = z.amax(1, keepdim=True)
    lse = (m + torch.log(torch.exp(z - m).sum(1, keepdim=True))).squeeze(1)
    w = torch.exp((z.double() - m) / T)  # sums over a vocabulary, and values next to a border
    if c["top_k"] or c["top_p"] < 1.0 or c["min_p"] > 0.0:
        falling, order = torch.sort(z, dim=1, descending=True, stable=True)
        upto = w.gather(1, order).cumsum(1)
        n = torch.full_like(order[:, :1], min(c["top_k"] or V, V))
        if c["top_p"] < 1.0:
            need = _f32(c["top_p"]) * upto.gather(1, n - 1)
            n = torch.minimum(n, (upto < need).sum(1, keepdim=True) + 1)
        if c["min_p"] > 0.0:
            least = m.double() + T * math.log(_f32(c["min_p"]))
            n = torch.minimum(n, (falling >= least).sum(1, keepdim=True))
        kept = torch.arange(V, device=z.device) < n
        w = w * torch.zeros_like(w).scatter_(1, order, kept.double())
    upto = w.cumsum(1)
    token = (upto <= st["uniform"].double().unsqueeze(1) * upto[:, -1:]).sum(1).clamp(max=V - 1)
    conf = torch.exp(z.gather(1, token.unsqueeze(1)).squeeze(1) - lse)
    open_ = st["masked"] != 0
    return {"row_max": torch.where(open_, m.squeeze(1), -math.inf),
            "lse": torch.where(open_, lse, -math.inf), "conf": torch.where(open_, conf, 0.0),
            "token": torch.where(open_, token, -1).to(torch.int32)}


def _scores(st):
    """Scaled scores [B, kv_heads, queries of a head, n, length], -inf where an entry is not seen."""
    c, n = st["case"], st["case"]["n"]
    table = st["table"].to(torch.int64)
    k = dequantise(st["k_codes"][table], st["k_params"][table])
    k = k.transpose(1, 2).flatten(2, 3)[:, :, :c["length"]]
    B, kh = k.shape[:2]
    q = st["q"].to(torch.float32).transpose(1, 2).reshape(B, kh, -1, c["head_dim"])
    j = torch.arange(c["length"], device=k.device)
    last = st["lens"].to(torch.int64)[:, None].expand(B, n)
    if c["causal"]:
        last = last - n + 1 + torch.arange(n, device=k.device)
    seen = j < last.unsqueeze(-1)
    if st["key_mask"] is not None:
        seen = seen & (st["key_mask"] != 0).unsqueeze(1)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).unflatten(2, (-1, n))
    return s.masked_fill_(~seen.unsqueeze(1).unsqueeze(1), -math.inf)


def _plain_weights(st):
    c = st["case"]
    s = _scores(st)
    lse = st["lse"].unflatten(1, (c["kv_heads"], -1)).unsqueeze(-1)
    lse = torch.where(lse == -math.inf, math.inf, lse)  # a query that saw nothing gives nothing
    got = s.sub_(lse).exp_().flatten(1, 3).sum(1)
    if st["prior"] is not None:
        got = got + _f32(c["keep"]) * st["prior"]
    there = torch.arange(c["length"], device=s.device) < st["lens"].unsqueeze(1)
    st["weights"].copy_(torch.where(there, got, st["weights"]))
    return {"weights": st["weights"]}


def _plain_evict(st):
    c = st["case"]
    length, ps, dev = c["length"], c["page_size"], st["weights"].device
    j = torch.arange(length, device=dev)
    lens = st["lens"].to(torch.int64).unsqueeze(1)
    new = lens.clamp(max=c["budget"])
    # those that stay whatever they weigh first, those that are not there last; ties in order
    rank = torch.where((j < c["first"]) | (j >= lens - c["last"]), math.inf, st["weights"])
    order = torch.sort(torch.where(j < lens, rank, -math.inf), dim=1, descending=True, stable=True)[1]
    stays = torch.zeros(c["B"], length, dtype=torch.bool, device=dev).scatter_(1, order, j < new)
    hole, tail = ~stays & (j < new), stays & (j >= new)
    # the k-th entry that stays beyond the new length takes the place of the k-th hole below it
    hole_rank = torch.where(hole, hole.cumsum(1) - 1, length)
    tail_rank = torch.where(tail, tail.cumsum(1) - 1, length)
    holes = torch.zeros(c["B"], length + 1, dtype=torch.int64, device=dev)
    holes.scatter_(1, hole_rank, j.expand_as(hole_rank))
    tails = torch.zeros_like(holes).scatter_(1, tail_rank, j.expand_as(tail_rank))
    slots = torch.where(stays, torch.where(tail, holes.gather(1, tail_rank), j), -1)
    origin = torch.where(hole, tails.gather(1, hole_rank), j)
    st["slots"].copy_(slots)
    st["new_lens"].copy_(new.squeeze(1))
    st["new_weights"].copy_(torch.where(j < new, st["weights"].gather(1, origin), 0.0))
    table = st["table"].to(torch.int64)
    most = min(length, c["budget"])
    page, slot = table.gather(1, origin[:, :most] // ps), origin[:, :most] % ps
    to_page, to_slot = table[:, j[:most] // ps], (j[:most] % ps).expand_as(page)
    for x in ("k_codes", "k_params", "v_codes", "v_params"):
        st[x][to_page, :, to_slot] = st[x][page, :, slot]
    return _evicted(st)


def _evicted(st):
    return {x: st[x] for x in ("slots", "new_lens", "new_weights", "k_codes", "k_params", "v_codes",
                               "v_params")}


# ---------------------------------------------------------------- the library's operators

def _own_sample(st):
    import diffusion_decoding_gb300 as dd
    c = st["case"]
    if "stats" not in st:  # descriptors and buffers that a decode loop makes once
        st["shape"] = dd.make_shape(c["B"], c["L"], c["V"],
                                    dd.DLLM_BF16 if c["dtype"] == "bf16" else dd.DLLM_F32,
                                    c["V"] + c["pad"])
        st["stats"] = dd.StatsBuffers(c["B"] * c["L"])
    s = st["stats"]
    dd.dllm_sample(st["logits"], st["shape"], st["masked"], st["uniform"], s,
                   temperature=c["temperature"], top_k=c["top_k"], top_p=c["top_p"],
                   min_p=c["min_p"])
    return {"row_max": s.row_max, "lse": s.lse, "conf": s.conf, "token": s.argmax}


def _own_weights(st):
    import diffusion_decoding_gb300 as dd
    c = st["case"]
    if "cache" not in st:  # the cache's descriptor and the workspace: made once, kept with the cache
        st["cache"] = dd.Kv4Cache.of(st["k_codes"], st["k_params"], st["v_codes"], st["v_params"],
                                     st["table"])
        st["ws"] = dd.workspace(dd.dllm_attention_kv4_weights_workspace_bytes(
            st["cache"], c["B"], c["n"], c["q_heads"], c["length"]))
    dd.dllm_attention_kv4_weights(st["q"], st["cache"], st["lens"], c["length"], st["lse"],
                                  st["weights"], st["ws"], prior=st["prior"], keep=c["keep"],
                                  key_mask=st["key_mask"], scale=st["scale"], causal=c["causal"])
    return {"weights": st["weights"]}


def _own_evict(st):
    import diffusion_decoding_gb300 as dd
    c = st["case"]
    if "cache" not in st:
        st["cache"] = dd.Kv4Cache.of(st["k_codes"], st["k_params"], st["v_codes"], st["v_params"],
                                     st["table"])
        st["ws"] = dd.workspace(dd.dllm_kv4_evict_workspace_bytes(st["cache"], c["B"], c["length"]))
    dd.dllm_kv4_evict(st["cache"], st["weights"], st["lens"], c["length"], c["budget"], st["slots"],
                      st["new_lens"], st["ws"], first=c["first"], last=c["last"],
                      weights_out=st["new_weights"])
    return _evicted(st)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"sample": _own_sample, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"sample": _plain_sample, "weights": _plain_weights, "evict": _plain_evict}[op](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_sample(st, c):
    V, T = c["V"], _f32(c["temperature"])
    R, dev = c["B"] * c["L"], st["uniform"].device
    out = {x: torch.full((R,), v, dtype=torch.float64, device=dev)
           for x, v in (("row_max", -math.inf), ("lse", -math.inf), ("conf", 0.0))}
    out["token"] = torch.full((R,), -1, dtype=torch.int32, device=dev)
    for r in torch.nonzero(st["masked"]).flatten().tolist():
        z = st["logits"][r, :V].double()
        lse = torch.logsumexp(z, 0)
        # candidates: probability falling, lower ids first among equals
        ids = torch.argsort(-z, stable=True)
        p = torch.softmax(z / T, 0)
        if c["top_k"]:
            ids = ids[:c["top_k"]]
        mass = torch.cumsum(p[ids], 0)
        count = ids.numel()
        if c["top_p"] < 1.0:
            reach = torch.searchsorted(mass, mass[-1:] * _f32(c["top_p"]), right=False)
            count = min(count, int(reach) + 1)
        if c["min_p"] > 0.0:
            ratio = (z[ids] - z.max()) / T - math.log(_f32(c["min_p"]))
            count = max(1, min(count, int((ratio >= 0.0).sum())))
        ids = torch.sort(ids[:count]).values
        mass = torch.cumsum(p[ids], 0)
        at = torch.searchsorted(mass, mass[-1:] * st["uniform"][r].double(), right=True)
        token = ids[min(int(at), ids.numel() - 1)]
        out["row_max"][r], out["lse"][r], out["conf"][r] = z.max(), lse, torch.exp(z[token] - lse)
        out["token"][r] = token.to(torch.int32)
    return out


def _exact_values(codes, params):
    word = params.long()
    exponent, mantissa, z = word // 128, word % 128 // 32, word % 16  # bf16(s): 8 + 7 bits
    step = torch.where(word < 32, 0.0, (1 + mantissa.double() / 4) * torch.exp2(exponent.double() - 127))
    pair = codes.long().unsqueeze(-1)
    n = torch.cat((pair % 16, pair // 16), -1).reshape(*codes.shape[:-1], -1, GROUP)
    return ((n - z.unsqueeze(-1)).double() * step.unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _exact_weights(st, c):
    if work(c)["flops"] > 4e12:
        return None
    n, G = c["n"], c["q_heads"] // c["kv_heads"]
    out = st["weights"].double()
    for b, length in enumerate(_lengths(c)):
        at = torch.arange(length, device="cuda")
        page, slot = st["table"][b].long()[at // c["page_size"]], at % c["page_size"]
        shown = torch.ones(n, length, dtype=torch.bool, device="cuda")
        if st["key_mask"] is not None:
            shown &= st["key_mask"][b, :length] != 0
        if c["causal"]:
            shown &= at <= length - n + torch.arange(n, device="cuda")[:, None]
        total = torch.zeros(length, dtype=torch.float64, device="cuda")
        if c["keep"]:
            total += _f32(c["keep"]) * st["prior"][b, :length].double()
        for h in range(c["kv_heads"]):
            k = _exact_values(st["k_codes"][page, h, slot], st["k_params"][page, h, slot])
            for i in range(h * G, (h + 1) * G):
                share = torch.exp((st["q"][b, :, i].double() @ k.T) * st["scale"]
                                  - st["lse"][b, i].double()[:, None])
                total += torch.where(shown, share, 0.0).sum(0)
        out[b, :length] = total
    return {"weights": out}


def _exact_evict(st, c):
    ps = c["page_size"]
    for b, length in enumerate(_lengths(c)):
        new = min(length, c["budget"])
        w = st["weights"][b].double().tolist()
        fixed = [e for e in range(length) if e < c["first"] or e >= length - c["last"]]
        others = sorted(range(c["first"], max(c["first"], length - c["last"])), key=lambda e: (-w[e], e))
        stays = set(range(length)) if new == length else set(fixed + others[:new - len(fixed)])
        holes = [e for e in range(new) if e not in stays]
        moved = [e for e in range(new, length) if e in stays]
        slots, weights = [-1] * c["length"], [0.0] * c["length"]
        for e in stays:
            if e < new:
                slots[e], weights[e] = e, w[e]
        table = st["table"][b].tolist()
        for e, hole in zip(moved, holes):
            slots[e], weights[hole] = hole, w[e]
        if moved:
            there = torch.tensor([(table[e // ps], e % ps) for e in moved], device="cuda").T
            here = torch.tensor([(table[e // ps], e % ps) for e in holes], device="cuda").T
            for x in ("k_codes", "k_params", "v_codes", "v_params"):
                st[x][here[0], :, here[1]] = st[x][there[0], :, there[1]]
        st["slots"][b] = torch.tensor(slots)
        st["new_lens"][b] = new
        st["new_weights"][b] = torch.tensor(weights, dtype=torch.float64)
    return _evicted(st)


def exact(case, seed):
    st = prepare(case, seed)
    return {"sample": _exact_sample, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](st, case)

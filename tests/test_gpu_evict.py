"""dllm_kv4_evict against a plain statement of it: every array equal."""
import math

import pytest
import torch

import diffusion_decoding_gb300 as dd
from bounded_ref import evict

pytestmark = pytest.mark.gpu

ARRAYS = ("k_codes", "k_params", "v_codes", "v_params")


def make_cache(B, per, heads, ps, D, seed, spare=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = B * per + spare
    cache = dd.Kv4Cache(pages, heads, ps, D, B, per)
    for x in ARRAYS:
        t = getattr(cache, x)
        t.copy_(torch.randint(0, 256 if t.dtype == torch.uint8 else 30000, t.shape, device="cuda", generator=g))
    cache.table.copy_(torch.randperm(pages, device="cuda", generator=g)[:B * per].view(B, per))
    return cache


def check(cache, w, lens, max_len, budget, first=0, last=0, in_place=False, pad=0):
    B, ps = cache.B, cache.page_size
    wide = torch.full((B, max_len + pad), 9.0, device="cuda")
    wide[:, :max_len] = w
    w = wide[:, :max_len]
    before = {x: getattr(cache, x).clone().cpu() for x in ARRAYS}
    wl = w.cpu().double().tolist()
    slots = torch.full((B, max_len + 2 * pad), 55, dtype=torch.int32, device="cuda")[:, :max_len]
    lens_in = None if lens is None else lens.clone()
    lens_out = lens_in if in_place and lens is not None else torch.full((B,), 77, dtype=torch.int32, device="cuda")
    w_out = w if in_place else torch.full((B, max_len), 66.0, device="cuda")
    ws = dd.workspace(dd.dllm_kv4_evict_workspace_bytes(cache, B, max_len))
    dd.dllm_kv4_evict(cache, w, lens_in, max_len, budget, slots, lens_out, ws, first=first, last=last,
                      weights_out=w_out)
    table = cache.table.cpu().tolist()
    for b in range(B):
        n = max_len if lens is None else max(0, min(int(lens[b]), max_len))
        new = min(n, budget)
        want, moves = evict(wl[b], n, budget, first, last)
        assert slots[b].tolist() == want + [-1] * (max_len - n)
        assert lens_out[b] == new
        weights = [0.0] * max_len
        for j, s in enumerate(want):
            if s >= 0:
                weights[s] = wl[b][j]
        got = w_out[b].cpu().double().tolist()
        assert all(x == y or (math.isnan(x) and math.isnan(y)) for x, y in zip(got, weights))
        for a, to in moves:
            pa, pt = table[b][a // ps], table[b][to // ps]
            if 0 <= pa < cache.pages and 0 <= pt < cache.pages:
                for x in ARRAYS:
                    before[x][pt, :, to % ps] = before[x][pa, :, a % ps]
    for x in ARRAYS:
        assert torch.equal(getattr(cache, x).cpu(), before[x]), x
    if pad:
        assert bool((wide[:, max_len:] == 9.0).all())


def rand(B, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(B, n, device="cuda", generator=g)


@pytest.mark.parametrize("ps,D,heads", [(16, 32, 1), (64, 128, 2), (48, 96, 3), (16, 512, 1), (32, 64, 5)])
def test_formats(ps, D, heads):
    cache = make_cache(2, 5, heads, ps, D, 1)
    n = 5 * ps - 3
    check(cache, rand(2, n, 1), torch.tensor([n, n // 2], dtype=torch.int32, device="cuda"), n, n // 3, 2, 3)


@pytest.mark.parametrize("budget,first,last", [(0, 0, 0), (1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 3, 4), (50, 0, 50),
                                               (50, 50, 0), (99, 2, 2), (100, 0, 0), (101, 5, 5), (5000, 1, 1)])
def test_budgets(budget, first, last):
    cache = make_cache(4, 7, 2, 16, 64, 2)
    lens = torch.tensor([100, 0, 1, 112], dtype=torch.int32, device="cuda")
    check(cache, rand(4, 112, budget), lens, 112, budget, first, last)


@pytest.mark.parametrize("max_len", [1, 31, 33, 600, 5000, 20011])
@pytest.mark.parametrize("in_place", [False, True])
def test_lengths(max_len, in_place):
    per = -(-max_len // 32)
    cache = make_cache(2, per, 1, 32, 32, 3)
    w = torch.round(rand(2, max_len, max_len) * 40) / 40  # many ties
    lens = torch.tensor([max_len, max(0, max_len - 17)], dtype=torch.int32, device="cuda")
    check(cache, w, lens, max_len, max_len // 2, min(2, max_len // 4), min(5, max_len // 4), in_place=in_place, pad=3)


def test_values():
    """Equal weights, NaN, infinities, zeros of both signs, subnormals, negatives."""
    cache = make_cache(7, 4, 1, 16, 32, 4)
    w = rand(7, 64, 4)
    w[0] = 0.25
    w[1, ::3] = math.nan
    w[2, ::2] = math.inf
    w[2, 1::4] = -math.inf
    w[3] = torch.where(torch.arange(64, device="cuda") % 2 == 0, 0.0, -0.0)
    w[4] = w[4] * 1e-42
    w[5] = w[5] - 0.5
    w[6] = math.nan
    for budget in (5, 20, 40, 63):
        check(cache, w, None, 64, budget, 1, 2)


def test_lens_beyond_max_len_and_negative():
    cache = make_cache(3, 4, 1, 16, 32, 5)
    lens = torch.tensor([200, -4, 64], dtype=torch.int32, device="cuda")
    check(cache, rand(3, 50, 5), lens, 50, 20, 1, 1)


def test_absent_pages_are_neither_read_nor_written():
    cache = make_cache(2, 6, 2, 16, 64, 6)
    cache.table[0, 1] = -1
    cache.table[0, 5] = cache.pages
    cache.table[1, 3] = 1 << 30
    check(cache, rand(2, 96, 6), None, 96, 40)


def test_many_sequences():
    cache = make_cache(300, 2, 1, 16, 32, 7)
    lens = torch.randint(0, 33, (300,), device="cuda").to(torch.int32)
    check(cache, rand(300, 32, 7), lens, 32, 11, 1, 2, in_place=True)


def test_no_weights_out_and_replay():
    cache = make_cache(2, 8, 2, 16, 64, 8)
    w, slots = rand(2, 128, 8), torch.empty(2, 128, dtype=torch.int32, device="cuda")
    lens_out = torch.empty(2, dtype=torch.int32, device="cuda")
    ws = dd.workspace(dd.dllm_kv4_evict_workspace_bytes(cache, 2, 128))
    dd.dllm_kv4_evict(cache, w, None, 128, 60, slots, lens_out, ws)
    want, kept = slots.clone(), {x: getattr(cache, x).clone() for x in ARRAYS}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dd.dllm_kv4_evict(cache, w, None, 128, 60, slots, lens_out, ws)
    slots.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    # the sources were left as they were: the same moves again change nothing
    assert torch.equal(slots, want) and lens_out.tolist() == [60, 60]
    for x in ARRAYS:
        assert torch.equal(getattr(cache, x), kept[x])

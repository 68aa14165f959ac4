"""dllm_sample against a 64-bit statement of it, row by row: tokens equal, statistics to their
rounding errors."""
import math

import numpy as np
import pytest
import torch

import diffusion_decoding_gb300 as dd
from bounded_ref import log_sum_exp, sample_row

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, dd.DLLM_BF16), "f32": (torch.float32, dd.DLLM_F32)}


def call(z, dtype, u, masked=None, pad=0, offset=0, **how):
    """z [R, V] float -> (stats, logits as the library sees them in float64)."""
    R, V = z.shape
    t, dt = DT[dtype]
    store = torch.full((offset + R * (V + pad) + 8,), 77.0, dtype=t, device="cuda")
    rows = store[offset:offset + R * (V + pad)].view(R, V + pad)
    rows[:, :V] = z.to(t)
    stats = dd.StatsBuffers(R)
    dd.dllm_sample(rows, dd.make_shape(1 if R <= 1024 else R // 64, R if R <= 1024 else 64, V, dt, V + pad),
                   masked, u, stats, **how)
    return stats, rows[:, :V].double().cpu().numpy()


def check(stats, z, u, masked=None, **how):
    token, conf, lse, top = (x.cpu().numpy() for x in (stats.argmax, stats.conf, stats.lse, stats.row_max))
    for r in range(z.shape[0]):
        if masked is not None and not masked[r]:
            assert (token[r], conf[r], lse[r], top[r]) == (-1, 0.0, -math.inf, -math.inf)
            continue
        want = sample_row(z[r], u[r].item(), **how)
        assert token[r] == want, (r, token[r], want)
        exact = log_sum_exp(z[r])
        assert top[r] == z[r].max()
        if want < 0:
            assert conf[r] == 0.0 and lse[r] == exact
            continue
        # at most 2^10 additions a lane, each half an ulp, and the terms' own errors; then the
        # rounding of lse itself
        tol = 2.0 ** -13 + abs(exact) * 2.0 ** -23
        assert abs(lse[r] - exact) <= tol
        p = math.exp(z[r][want] - exact)
        assert abs(conf[r] - p) <= p * (2 * tol + abs(z[r][want] - exact) * 2.0 ** -22) + 1e-37


def uniform(R, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(R, device="cuda", generator=g)


def logits(R, V, seed, head=3.0):
    """A bulk and a few likely tokens, more or less so from row to row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = 2.0 * torch.randn(R, V, device="cuda", generator=g)
    k = min(V, 12)
    at = torch.rand(R, V, device="cuda", generator=g).argsort(1)[:, :k]
    up = math.log(V) + head * torch.rand(R, 1, device="cuda", generator=g) - torch.arange(k, device="cuda")
    return z.scatter(1, at, up.expand(R, k))


FILTERS = [dict(), dict(top_k=1), dict(top_k=7), dict(top_k=50, top_p=0.9), dict(top_p=0.5),
           dict(top_p=0.97), dict(min_p=0.1), dict(top_k=300, top_p=0.999, min_p=0.001),
           dict(top_p=0.9, min_p=0.02)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 30011])
def test_filters(dtype, V):
    z = logits(6, V, V)
    for i, f in enumerate(FILTERS):
        u = uniform(6, 10 * V + i)
        how = dict(temperature=[1.0, 0.5, 1.7][i % 3], **f)
        stats, seen = call(z, dtype, u, **how)
        check(stats, seen, u, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 3, 40, 700])
def test_rows_and_clusters(dtype, R):
    """The same rows give the same tokens in any company (a row takes one CTA or up to eight)."""
    V = 40009
    z, u = logits(R, V, R), uniform(R, R)
    for how in (dict(temperature=0.8), dict(temperature=0.8, top_p=0.92), dict(temperature=1.0, top_k=40)):
        stats, seen = call(z, dtype, u, **how)
        few = min(R, 5)
        check(dd.StatsBuffers(1) if few == 0 else _head(stats, few), seen[:few], u[:few], **how)
        alone, _ = call(z[R - 1:], dtype, u[R - 1:].contiguous(), **how)
        assert alone.argmax[0] == stats.argmax[R - 1]
        again, _ = call(z, dtype, u, **how)
        assert torch.equal(again.argmax, stats.argmax)
        assert torch.equal(again.lse, stats.lse) and torch.equal(again.conf, stats.conf)


def _head(stats, n):
    out = dd.StatsBuffers(n)
    for x in ("row_max", "lse", "conf", "argmax"):
        getattr(out, x).copy_(getattr(stats, x)[:n])
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (5, 4)])
def test_rows_on_no_boundary(dtype, pad, offset):
    z, u = logits(5, 2051, 3), uniform(5, pad)
    for how in (dict(temperature=1.0), dict(temperature=1.0, top_p=0.9)):
        stats, seen = call(z, dtype, u, pad=pad, offset=offset, **how)
        check(stats, seen, u, **how)


def test_masked_rows_are_not_read():
    z, u = logits(8, 3001, 4), uniform(8, 4)
    z[2] = float("nan")
    masked = torch.tensor([1, 0, 0, 1, 1, 0, 1, 0], dtype=torch.uint8, device="cuda")
    stats, seen = call(z, "f32", u, masked=masked, temperature=0.9, top_p=0.8)
    check(stats, seen, u, masked=masked.tolist(), temperature=0.9, top_p=0.8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hidden_tokens(dtype):
    """-inf: never drawn, whatever the filters; rows with one token left, and with none."""
    V = 5000
    z = logits(6, V, 6)
    z[0, ::2] = -math.inf
    z[1, 1:] = -math.inf
    z[2, :] = -math.inf
    z[3, :V - 1] = -math.inf
    z[4, 100:] = -math.inf
    u = uniform(6, 6)
    for how in (dict(temperature=1.0), dict(temperature=1.0, top_k=4000), dict(temperature=1.0, top_p=0.99),
                dict(temperature=0.0), dict(temperature=2.0, min_p=1e-6)):
        stats, seen = call(z, dtype, u, **how)
        check(stats, seen, u, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [64, 1024, 40000])
def test_equal_logits(dtype, V):
    """All weights are 1, so that every sum and border is exact: u * n on and beside whole numbers."""
    z = torch.full((7, V), -3.25, device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.5 - 2.0 ** -25, 0.999, 1.0 - 2.0 ** -24], device="cuda")
    for how in (dict(temperature=0.7), dict(temperature=0.7, top_k=V // 2), dict(temperature=1.0, top_p=0.5),
                dict(temperature=1.0, top_k=V // 2, top_p=0.25), dict(temperature=1.0, min_p=1.0)):
        stats, seen = call(z, dtype, u, **how)
        check(stats, seen, u, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_ties(dtype):
    """Few distinct values, so that a cut falls among thousands of equals; both zeros are one value."""
    g = torch.Generator(device="cuda").manual_seed(9)
    V = 30000
    z = torch.randint(-3, 1, (6, V), device="cuda", generator=g).float()
    z[:, ::7] *= -1.0  # -0 among the zeros, and a few positive
    u = uniform(6, 9)
    for how in (dict(temperature=1.0, top_k=2500), dict(temperature=1.0, top_k=9000), dict(temperature=1.0, top_p=0.3),
                dict(temperature=0.6, top_p=0.85), dict(temperature=1.0, top_k=20000, top_p=0.7),
                dict(temperature=0.0)):
        stats, seen = call(z, dtype, u, **how)
        check(stats, seen, u, **how)


def test_close_values():
    """Thousands of different values within a small part of an octave."""
    g = torch.Generator(device="cuda").manual_seed(11)
    z = 5.0 + 0.003 * torch.rand(4, 20000, device="cuda", generator=g)
    u = uniform(4, 11)
    for how in (dict(temperature=1.0, top_k=2777), dict(temperature=1.0, top_p=0.37), dict(temperature=0.5)):
        stats, seen = call(z, "f32", u, **how)
        check(stats, seen, u, **how)


@pytest.mark.parametrize("temperature", [2.0 ** -10, 0.01, 0.1, 30.0, 1024.0])
def test_temperatures(temperature):
    z, u = logits(8, 3000, 12), uniform(8, 12)
    for f in (dict(), dict(top_p=0.8), dict(top_k=20)):
        stats, seen = call(z, "bf16", u, temperature=temperature, **f)
        check(stats, seen, u, temperature=temperature, **f)


def test_large_logits():
    z = logits(4, 3000, 13)
    z[1] = z[1] * 1e4
    z[2] = z[2] + 3e4
    z[3] = z[3] * 1e36
    u = uniform(4, 13)
    for how in (dict(temperature=1.0), dict(temperature=1.0, top_p=0.9), dict(temperature=0.0)):
        stats, seen = call(z, "f32", u, **how)
        token = stats.argmax.cpu()
        for r in range(4):
            assert token[r] == sample_row(seen[r], u[r].item(), **how)


def test_uniform_out_of_range():
    z = logits(6, 777, 14)
    u = torch.tensor([-1.0, 1.0, 7.0, math.inf, -math.inf, math.nan], device="cuda")
    for how in (dict(temperature=1.0), dict(temperature=1.0, top_k=30)):
        stats, seen = call(z, "f32", u, **how)
        check(stats, seen, u, **how)


def test_largest_vocabulary():
    V = 1 << 20
    z, u = logits(2, V, 15), uniform(2, 15)
    for dtype in ("bf16", "f32"):
        for how in (dict(temperature=1.0), dict(temperature=1.0, top_p=0.9), dict(temperature=1.0, top_k=100)):
            stats, seen = call(z, dtype, u, **how)
            check(stats, seen, u, **how)


def test_frequencies():
    """Draws at evenly spread numbers hit every token as often as its weight says."""
    p = torch.tensor([0.5, 0.25, 0.125, 0.125])
    R = 1024
    z = torch.log(p).repeat(R, 1).cuda()
    u = (torch.arange(R, device="cuda") + 0.5) / R
    stats, _ = call(z, "f32", u, temperature=1.0)
    count = torch.bincount(stats.argmax.cpu().long(), minlength=4)
    assert (count - (p * R).long()).abs().max() <= 1  # log(p) is rounded


def test_commit_of_sampled_tokens():
    """The statistics feed the commit: sampled tokens where their probability passes the threshold."""
    B, L, V = 2, 16, 999
    z, u = logits(B * L, V, 16), uniform(B * L, 16)
    state, stats = dd.BlockState(B, L), dd.StatsBuffers(B * L)
    shape = dd.make_shape(B, L, V, dd.DLLM_F32)
    dd.dllm_sample(z, shape, state.masked, u, stats, temperature=1.0, top_k=20)
    dd.dllm_commit_threshold(None, shape, stats, state, 0.3, -1, None)
    token, conf = stats.argmax.view(B, L).cpu(), stats.conf.view(B, L).cpu()
    got, left = state.tokens.view(B, L).cpu(), state.masked.view(B, L).cpu()
    for b in range(B):
        fixed = (conf[b] > 0.3).nonzero().flatten().tolist() or [int(conf[b].argmax())]
        for i in range(L):
            assert left[b, i] == (0 if i in fixed else 1)
            assert got[b, i] == (token[b, i] if i in fixed else -1)


def test_captured_and_on_another_stream():
    z, u = logits(40, 9000, 17), uniform(40, 17)
    shape, stats = dd.make_shape(1, 40, 9000, dd.DLLM_F32), dd.StatsBuffers(40)
    want, _ = call(z, "f32", u, temperature=0.9, top_p=0.9)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dd.dllm_sample(z, shape, None, u, stats, temperature=0.9, top_p=0.9)
    side.synchronize()
    assert torch.equal(stats.argmax, want.argmax)
    stats.argmax.fill_(-5)
    with torch.cuda.graph(graph):
        dd.dllm_sample(z, shape, None, u, stats, temperature=0.9, top_p=0.9)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(stats.argmax, want.argmax) and torch.equal(stats.conf, want.conf)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1, 100, 129, 300, 513, 700, 1500, 2047, 2049, 5000])
def test_kept_by_number(dtype, size):
    """Nuclei and top-k sets of as many candidates as lists hold, a few more and far more: `size` tokens
    stand out of 9001, alone or with a few chunks full of them."""
    V, R = 9001, 6
    g = torch.Generator(device="cuda").manual_seed(size)
    z = torch.randn(R, V, device="cuda", generator=g) - 12.0
    up = torch.rand(R, size, device="cuda", generator=g)
    at = torch.rand(R, V, device="cuda", generator=g).argsort(1)[:, :size]
    at[R // 2:] = torch.arange(size, device="cuda") + 17
    z.scatter_(1, at, up)
    for i, how in enumerate([dict(top_p=0.9), dict(top_k=size), dict(top_k=size, top_p=0.95),
                             dict(top_p=0.999, min_p=0.4), dict(min_p=0.2)]):
        u = uniform(R, 100 * size + i)
        stats, seen = call(z, dtype, u, temperature=1.0, **how)
        check(stats, seen, u, temperature=1.0, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(2, 1000), (40, 5000), (330, 12345)])
def test_flat_rows(dtype, R, V):
    """Rows that the sums of chunks leave open: no token weighs more than their error."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = 0.3 * torch.randn(R, V, device="cuda", generator=g)
    for i, how in enumerate([dict(), dict(top_p=0.9), dict(top_p=0.1), dict(top_k=V - 1, top_p=0.5)]):
        u = uniform(R, V + i)
        stats, seen = call(z, dtype, u, temperature=1.5, **how)
        check(stats, seen, u, temperature=1.5, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_flat_rows_by_two(dtype):
    """The same where two CTAs share a row: borders in doubt go to the second kernel, long lists do not."""
    R, V = 200, 15001
    g = torch.Generator(device="cuda").manual_seed(4)
    z = torch.randn(R, V, device="cuda", generator=g)
    z[: R // 2] *= 0.2
    z[::3, 77] += 9.0
    for i, how in enumerate([dict(), dict(top_p=0.9), dict(top_p=0.3, min_p=0.001)]):
        u = uniform(R, 50 + i)
        stats, seen = call(z, dtype, u, temperature=1.2, **how)
        check(stats, seen, u, temperature=1.2, **how)

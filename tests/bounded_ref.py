"""64-bit statements of sampling, accumulated attention weights and eviction, for the tests: plain
numpy and torch, no code of the library."""
import math

import numpy as np
import torch

from refresh_ref import unpack


def sample_row(z, u, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """Token of one row z (float64 numpy), or -1."""
    z = np.asarray(z, dtype=np.float64)
    temperature, top_p, min_p = (float(np.float32(x)) for x in (temperature, top_p, min_p))
    if not np.isfinite(z.max()):
        return -1
    if temperature == 0.0:
        return int(np.argmax(z))
    order = np.lexsort((np.arange(z.size), -z))  # falling, lower ids first among equals
    w = np.exp((z - z.max()) / temperature)
    n = min(top_k, z.size) if top_k else z.size
    if top_p < 1.0:
        upto = np.cumsum(w[order][:n])
        n = min(n, int(np.searchsorted(upto, top_p * upto[-1], side="left")) + 1)
    if min_p > 0.0:
        n = min(n, int((z[order] >= z.max() + temperature * math.log(min_p)).sum()))
    ids = np.sort(order[:n])
    upto = np.cumsum(w[ids])
    u = float(np.float32(u))
    u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1.0 - 2.0 ** -24)
    return int(ids[np.searchsorted(upto, u * upto[-1], side="right")])


def log_sum_exp(z):
    m = z.max()
    return m + math.log(np.exp(z - m).sum()) if np.isfinite(m) else -math.inf


def cache_values(cache, x, b, h):
    """Keys ("k") or values ("v") of head h of sequence b, [entries of the table, D] float64; entries on
    an absent page are 0.  Also whether each entry's page is there."""
    codes, params = getattr(cache, x + "_codes"), getattr(cache, x + "_params")
    ps, table = cache.page_size, cache.table[b].tolist()
    rows, there = [], []
    for page in table:
        ok = 0 <= page < cache.pages
        rows.append(unpack(codes[page if ok else 0, h], params[page if ok else 0, h]) * (1.0 if ok else 0.0))
        there += [ok] * ps
    return torch.cat(rows), torch.tensor(there, device=codes.device)


def received(q, cache, lens, lse, seen, scale, keep=0.0, prior=None):
    """weights [B, T] float64 of the attention that entries receive, the number of terms and the largest
    sum_c |scale q_c k_c| of each entry (scales of the rounding errors).  seen [B, n, T] bool."""
    B, n, Hq, D = q.shape
    T = seen.shape[2]
    out = torch.zeros(B, T, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    for b in range(B):
        for h in range(Hq):
            k, there = cache_values(cache, "k", b, h // (Hq // cache.heads))
            k, there = k[:T], there[:T]
            on = seen[b] & there & (lse[b, h] != -math.inf)[:, None]
            k = torch.where(on.any(0)[:, None], k, 0.0)
            x = q[b, :, h].double()
            term = torch.exp(scale * (x @ k.T) - lse[b, h].double()[:, None])
            out[b] += torch.where(on, term, 0.0).sum(0)
            size[b] = torch.maximum(size[b], (abs(scale) * (x.abs() @ k.abs().T)).amax(0))
    if prior is not None:
        out = out + float(np.float32(keep)) * prior[:, :T].double()
    return out, size


def evict(w, length, budget, first, last):
    """New entry number of each of the `length` entries (-1: dropped) and the moves [(from, to)]."""
    new = min(length, budget)
    if length <= budget:
        return list(range(length)), []
    fixed = [j for j in range(length) if j < first or j >= length - last]
    others = [j for j in range(length) if first <= j < length - last]
    value = lambda j: -math.inf if math.isnan(w[j]) else w[j]  # noqa: E731
    # a NaN is less than every number, -inf too
    others.sort(key=lambda j: (math.isnan(w[j]), -value(j), j))
    stays = set(fixed + others[:new - len(fixed)])
    holes = [j for j in range(new) if j not in stays]
    moved = [j for j in range(new, length) if j in stays]
    slots = [j if j in stays and j < new else -1 for j in range(length)]
    for a, b in zip(moved, holes):
        slots[a] = b
    return slots, list(zip(moved, holes))

"""dllm_sample where top_p lies beside a border of its order: the cut falls as in 64 bits."""
import numpy as np
import pytest
import torch

import diffusion_decoding_gb300 as dd

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, dd.DLLM_BF16), "f32": (torch.float32, dd.DLLM_F32)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,R", [(16, 300), (900, 700), (40003, 50), (40003, 250), (40003, 700)])
@pytest.mark.parametrize("bulk", [7.0, 13.0])
@pytest.mark.parametrize("top_k", [0, 30])
def test_cut(V, R, dtype, bulk, top_k):
    """Rows of the same logits in other orders, so that one top_p lies beside a border of all of them.  The
    sums up to the border and top_p times the total are off by 2^-36 of themselves and V 2^-43 each."""
    rng = np.random.default_rng(V + R)
    heavy = min(V, 12)
    one = np.concatenate([1.2 * rng.standard_normal(heavy), -bulk + rng.random(V - heavy)])
    one = torch.from_numpy(one).to(DT[dtype][0])
    order = np.argsort(rng.random((R, V)), 1)
    z = one[torch.from_numpy(order)].cuda()
    seen, t = one.double().numpy(), float(np.float32(0.8))
    w = np.sort(np.exp((seen - seen.max()) / t))[::-1]
    upto = np.cumsum(w[:top_k] if top_k else w)
    u = rng.random(R).astype(np.float32)
    shape, stats = dd.make_shape(1, R, V, DT[dtype][1]), dd.StatsBuffers(R)
    first = min(R, 60)  # rows that are looked at
    row_w = np.exp((z[:first].double().cpu().numpy() - seen.max()) / t)
    by_fall = np.argsort(-row_w, axis=1, kind="stable")
    for k in range(heavy - 1):
        if k + 1 < heavy and w[k] == w[k + 1]:
            continue  # (which of two equals is cut off depends on the row's order alone)
        for step in (-2, -1, 0, 1, 2):
            top_p = np.float32(upto[k] / upto[-1])
            for _ in range(abs(step)):
                top_p = np.nextafter(top_p, np.float32(1.0 if step > 0 else 0.0))
            if not 0.0 < top_p < 1.0 or abs(float(top_p) - upto[k] / upto[-1]) < 2.0 ** -35 + V * 2.0 ** -42 / upto[-1]:
                continue
            kept = int(np.searchsorted(upto, float(top_p) * upto[-1], side="left")) + 1
            dd.dllm_sample(z, shape, None, torch.from_numpy(u).cuda(), stats, temperature=0.8, top_k=top_k,
                           top_p=float(top_p))
            got = stats.argmax.cpu().numpy()
            for r in range(first):
                ids = np.sort(by_fall[r, :kept])
                c = np.cumsum(row_w[r, ids])
                goal = float(u[r]) * c[-1]
                if np.abs(c - goal).min() < 2.0 ** -30 * c[-1]:
                    continue
                assert got[r] == ids[np.searchsorted(c, goal, side="right")], (k, step, r, float(top_p))

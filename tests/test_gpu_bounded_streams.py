"""Sampling, accumulated weights and eviction on several streams at once, each with its own buffers: as alone."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
from test_gpu_received import setup

pytestmark = pytest.mark.gpu


class Work:
    def __init__(self, seed, D, n, G, B=6, per=12):
        self.cache, self.q, g = setup(B, per, 2, 64, D, n, G, seed)
        self.T, H = per * 64, 2 * G
        self.lens = torch.randint(200, self.T + 1, (B,), device="cuda", generator=g).to(torch.int32)
        self.z = 3.0 * torch.randn(40, 30001, device="cuda", generator=g)
        self.u = torch.rand(40, device="cuda", generator=g)
        self.shape = dd.make_shape(1, 40, 30001, dd.DLLM_F32)
        self.ws = [dd.workspace(x) for x in (
            dd.dllm_attention_kv4_workspace_bytes(self.cache, B, n, H, self.T),
            dd.dllm_attention_kv4_weights_workspace_bytes(self.cache, B, n, H, self.T),
            dd.dllm_kv4_evict_workspace_bytes(self.cache, B, self.T))]
        self.lse = torch.empty(B, H, n, device="cuda")
        self.out = torch.empty_like(self.q)
        self.k_codes, self.v_codes = self.cache.k_codes.clone(), self.cache.v_codes.clone()
        self.k_params, self.v_params = self.cache.k_params.clone(), self.cache.v_params.clone()

    def run(self, rounds, sink):
        for x in ("k_codes", "k_params", "v_codes", "v_params"):
            getattr(self.cache, x).copy_(getattr(self, x))
        lens = self.lens.clone()
        weights = torch.zeros(self.q.shape[0], self.T, device="cuda")
        slots = torch.empty(self.q.shape[0], self.T, dtype=torch.int32, device="cuda")
        for k in range(rounds):
            stats = dd.StatsBuffers(40)
            dd.dllm_attention_kv4(self.q, self.cache, lens, self.T, self.out, self.ws[0], lse=self.lse)
            dd.dllm_attention_kv4_weights(self.q, self.cache, lens, self.T, self.lse, weights, self.ws[1],
                                          prior=weights, keep=0.9)
            dd.dllm_kv4_evict(self.cache, weights, lens, self.T, self.T - 50 * (k + 1), slots, lens, self.ws[2],
                              first=2, last=5, weights_out=weights)
            dd.dllm_sample(self.z, self.shape, None, self.u, stats, temperature=1.0 + 0.1 * k, top_p=0.95)
            sink += [lens.clone(), weights.clone(), slots.clone(), self.out.clone(), stats.argmax, stats.conf]


def test_three_streams():
    works = [Work(1, 128, 40, 4), Work(2, 64, 1, 4), Work(3, 256, 33, 2)]
    alone = []
    for w in works:
        sink = []
        w.run(8, sink)
        torch.cuda.synchronize()
        alone.append([x.clone() for x in sink])
    streams = [torch.cuda.Stream() for _ in works]
    together = [[] for _ in works]
    for w, stream, sink in zip(works, streams, together):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            w.run(8, sink)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        for i, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), i
    for w in works:
        assert all(dd.dllm_get_status(x) == dd.DLLM_OK for x in w.ws[:2])

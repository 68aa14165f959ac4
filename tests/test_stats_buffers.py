"""Statistics buffers of fewer rows than a call writes are refused before anything is launched (no GPU
needed)."""
from types import SimpleNamespace

import pytest
import torch

import diffusion_decoding_gb300 as dd
from diffusion_decoding_gb300 import build as cuda_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()


@pytest.mark.parametrize("short", [None, "row_max", "lse", "conf", "argmax"])
def test_short_buffers(short):
    shape, z, u = dd.make_shape(2, 4, 100, dd.DLLM_F32), torch.zeros(8, 100), torch.zeros(8)
    stats = dd.StatsBuffers(7 if short is None else 8, device="cpu")
    if short is not None:
        setattr(stats, short, getattr(stats, short)[:7])
    with pytest.raises(ValueError, match="statistics"):
        dd.dllm_sample(z, shape, None, u, stats)
    with pytest.raises(ValueError, match="statistics"):
        dd.dllm_decode_stats(z, shape, None, stats, None)
    state = dd.BlockState(2, 4, 2, device="cpu")
    for call in (lambda: dd.dllm_commit_threshold(z, shape, stats, state, 0.9, -1, None),
                 lambda: dd.dllm_commit_threshold(None, shape, stats, state, 0.9, -1, None),
                 lambda: dd.dllm_commit_threshold_static(z, shape, stats, state, 0.9, -1),
                 lambda: dd.dllm_commit_hierarchical(z, shape, stats, state, 0.5, 2, -1, None),
                 lambda: dd.dllm_commit_hierarchical_levels(z, shape, stats, state, 0.5, 2, -1, None),
                 lambda: dd.dllm_commit_credit(z, shape, stats, state, 2, 0.7, 0.3, 0.9, -1, None),
                 lambda: dd.dllm_commit_credit_tracked(z, shape, stats, state, 2, 0.7, 0.3, 0.9, -1, None)):
        with pytest.raises(ValueError, match="statistics"):
            call()


def test_buffers_of_more_rows_pass():
    """(as far as the next refusal, a temperature that the library does not take)"""
    stats = dd.StatsBuffers(9, device="cpu")
    with pytest.raises(dd.DllmError, match="temperature"):
        dd.dllm_sample(torch.zeros(8, 100), dd.make_shape(2, 4, 100, dd.DLLM_F32), None, torch.zeros(8), stats,
                       temperature=-1.0, stream=SimpleNamespace(cuda_stream=0))

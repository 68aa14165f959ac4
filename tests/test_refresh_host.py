"""Host-side checks of the refresh operators: every bad argument is refused before a launch (no
GPU needed), and the binding checks its tensors."""
import ctypes
import math

import pytest
import torch

import diffusion_decoding_gb300 as dd
from diffusion_decoding_gb300 import build as cuda_build

INV, UNS = dd.DLLM_ERR_INVALID_ARG, dd.DLLM_ERR_UNSUPPORTED
BAD = 4096  # an address that is never read: every call below is refused


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return dd.lib()


def heads(data=BAD, heads=4, dtype=dd.DLLM_BF16, strides=(4096, 512, 128)):
    return dd.dllm_heads(data, heads, dtype, *strides)


def cache(**kw):
    d = dict(k_codes=BAD, k_params=BAD, v_codes=BAD, v_params=BAD, page_table=BAD, pages=8, heads=4,
             page_size=64, head_dim=128, table_stride=4)
    d.update(kw)
    return dd.dllm_kv4_cache(*d.values())


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("kw,expect", [
    (dict(rotary_dim=3), INV), (dict(rotary_dim=0), INV), (dict(rotary_dim=2048), UNS),
    (dict(scaling=2), UNS), (dict(base=1.0), INV), (dict(base=math.nan), INV),
    (dict(factor=0.5), INV), (dict(factor=math.inf), INV),
    (dict(scaling=1, original_len=0.0), INV), (dict(scaling=1, fast_turns=1.0), INV),
    (dict(scaling=1, slow_turns=-1.0), INV)])
def test_rope_phases_refuses(lib, kw, expect):
    d = dict(rotary_dim=64, scaling=0, base=1e4, factor=2.0, original_len=4096.0, slow_turns=1.0,
             fast_turns=32.0)
    d.update(kw)
    assert lib.dllm_rope_phases(ctypes.byref(dd.dllm_rope(*d.values())), BAD, None) == expect
    assert lib.dllm_last_error()


def norm_rope(lib, q=heads(), qo=heads(), k=heads(), ko=heads(), B=2, n=3, D=128, pos=BAD,
              phases=BAD, R=128, norm=1, wq=None, wk=None, eps=1e-6):
    return lib.dllm_qk_norm_rope(ref(q), ref(qo), ref(k), ref(ko), B, n, D, pos, 3, phases, R, 0,
                                 1.0, norm, wq, wk, eps, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(ko=None), INV), (dict(q=None, qo=None, k=None, ko=None), INV),
    (dict(q=heads(data=None)), INV), (dict(q=heads(data=BAD + 1)), INV),
    (dict(q=heads(dtype=9)), UNS), (dict(k=heads(dtype=dd.DLLM_F32)), INV),
    (dict(q=heads(heads=0)), INV), (dict(qo=heads(heads=3)), INV), (dict(B=0), INV),
    (dict(n=0), INV), (dict(B=2048, n=1024), UNS), (dict(D=0), INV), (dict(D=1025, R=0), UNS),
    (dict(R=7), INV), (dict(R=130), INV), (dict(pos=None), INV), (dict(phases=None), INV),
    (dict(R=0, norm=0), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(norm=0, wq=BAD), INV), (dict(wk=BAD + 1), INV), (dict(pos=BAD + 2), INV)])
def test_norm_rope_refuses(lib, kw, expect):
    assert norm_rope(lib, **kw) == expect
    assert lib.dllm_last_error()


CACHE_FAULTS = [
    (dict(k_codes=None), INV), (dict(page_table=None), INV), (dict(pages=0), INV),
    (dict(heads=0), INV), (dict(table_stride=0), INV), (dict(page_size=8), UNS),
    (dict(page_size=24), UNS), (dict(page_size=1 << 17), UNS), (dict(head_dim=48), UNS),
    (dict(head_dim=544), UNS), (dict(k_codes=BAD + 8), INV), (dict(v_params=BAD + 2), INV),
    (dict(table_stride=1 << 26, page_size=64), UNS)]


@pytest.mark.parametrize("kw,expect", CACHE_FAULTS)
def test_cache_calls_refuse_bad_caches(lib, kw, expect):
    c = cache(**kw)
    h = heads()
    for fn in (lib.dllm_kv4_write, lib.dllm_kv4_read):
        assert fn(ref(c), ref(h), ref(h), 2, 3, BAD, 3, None) == expect
    assert lib.dllm_attention_kv4(ref(h), ref(c), None, 64, None, 0, 1.0, 0, ref(h), None, 2, 3, BAD,
                                  1 << 40, None) == expect
    assert lib.dllm_attention_kv4_workspace_bytes(ref(c), 2, 3, 4, 64) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INV), (dict(v=heads(data=None)), INV), (dict(k=heads(heads=3)), INV),
    (dict(v=heads(dtype=dd.DLLM_F32)), INV), (dict(B=0), INV), (dict(n=1 << 21), UNS),
    (dict(pos=BAD + 1), INV)])
def test_cache_calls_refuse_bad_rows(lib, kw, expect):
    d = dict(k=heads(), v=heads(), B=2, n=3, pos=BAD)
    d.update(kw)
    c = cache()
    for fn in (lib.dllm_kv4_write, lib.dllm_kv4_read):
        assert fn(ref(c), ref(d["k"]), ref(d["v"]), d["B"], d["n"], d["pos"], 3, None) == expect
    assert lib.dllm_kv4_write(ref(c), ref(heads()), ref(heads()), 2, 3, None, 3, None) == INV


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(out=heads(heads=8)), INV), (dict(q=heads(heads=6), out=heads(heads=6)), INV),
    (dict(q=heads(dtype=dd.DLLM_F32)), UNS), (dict(out=heads(dtype=dd.DLLM_F32)), UNS),
    (dict(c=cache(head_dim=96)), UNS), (dict(max_len=-1), INV), (dict(max_len=257), INV),
    (dict(scale=math.inf), INV), (dict(scale=math.nan), INV), (dict(mask=BAD, mask_stride=63), INV),
    (dict(ws=None), INV), (dict(ws=BAD + 128), INV), (dict(ws_bytes=0), INV),
    (dict(lens=BAD + 1), INV), (dict(lse=BAD + 2), INV), (dict(B=0), INV), (dict(n=1 << 21), UNS)])
def test_attention_refuses(lib, kw, expect):
    d = dict(q=heads(), c=cache(), lens=None, max_len=64, mask=None, mask_stride=0, scale=1.0,
             out=heads(), lse=None, B=2, n=3, ws=BAD, ws_bytes=1 << 40)
    d.update(kw)
    assert lib.dllm_attention_kv4(ref(d["q"]), ref(d["c"]), d["lens"], d["max_len"], d["mask"],
                                  d["mask_stride"], d["scale"], 0, ref(d["out"]), d["lse"], d["B"],
                                  d["n"], d["ws"], d["ws_bytes"], None) == expect
    assert lib.dllm_last_error()


def test_workspace_is_the_same_for_every_call_of_a_size(lib):
    c = cache()
    a = lib.dllm_attention_kv4_workspace_bytes(ref(c), 2, 1, 8, 256)
    assert a >= 256 and a == lib.dllm_attention_kv4_workspace_bytes(ref(c), 2, 1, 8, 256)


def cpu_cache():
    return dd.Kv4Cache(4, 2, 16, 64, 2, 2, device="cpu")


def test_binding_checks_its_tensors():
    c = cpu_cache()
    assert c.c().head_dim == 64 and c.c().table_stride == 2 and (c.table == -1).all()
    x = torch.zeros(2, 3, 2, 64)
    pos = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        dd.dllm_kv4_write(c, x, x[:, :2], pos)
    with pytest.raises(ValueError):
        dd.dllm_kv4_write(c, x, x, pos.long())
    with pytest.raises(ValueError):
        dd.dllm_kv4_write(c, x, x, pos[:, :2])
    with pytest.raises(TypeError):
        dd.heads_of(x.half())
    with pytest.raises(ValueError):
        dd.heads_of(x.transpose(2, 3))
    with pytest.raises(ValueError):
        dd.dllm_qk_norm_rope(x, None, x[:1], None, pos, None)
    with pytest.raises(ValueError):
        dd.dllm_qk_norm_rope(x, None, x, None, pos, None, q_weight=torch.ones(32))
    with pytest.raises(ValueError):
        dd.dllm_attention_kv4(x, c, torch.zeros(2), 16, x, None)
    with pytest.raises(ValueError):
        dd.dllm_attention_kv4(x, c, None, 16, x, None, lse=torch.zeros(2, 3, 2))
    with pytest.raises(ValueError):
        dd.dllm_attention_kv4(x, c, None, 16, x, None, key_mask=torch.zeros(2, 15, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dd.dllm_rope_phases(64, torch.zeros(16, dtype=torch.int64))
    with pytest.raises(ValueError):
        dd.Kv4Cache.of(c.k_codes, c.k_params[:2], c.v_codes, c.v_params, c.table)

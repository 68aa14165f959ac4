"""Host-side checks of the refresh operators beyond test_refresh_host.py: sizes at the far end of the
limits, and tensors that the binding must not take (no GPU needed: every call is refused or only asks
for sizes)."""
import pytest
import torch

import diffusion_decoding_gb300 as dd
from test_refresh_host import BAD, INV, UNS, cache, heads, lib, norm_rope, ref  # noqa: F401


@pytest.mark.parametrize("q,k,B,n", [
    (65536, 65536, 1 << 10, 1 << 6),   # 2^33 heads
    (65536, 65536, 1 << 20, 1), (8192, None, 1 << 20, 1), (None, 8192, 1, 1 << 20),
    (8191, 1, 1 << 10, 1 << 10)])
@pytest.mark.parametrize("D,R", [(1, 0), (64, 64), (1024, 0)])
def test_norm_rope_refuses_more_heads_than_a_grid_has_warps(lib, q, k, B, n, D, R):
    hq, hk = (None if h is None else heads(heads=h) for h in (q, k))
    assert norm_rope(lib, q=hq, qo=hq, k=hk, ko=hk, B=B, n=n, D=D, R=R) == UNS
    assert b"heads" in lib.dllm_last_error()


def test_phase_tables_are_whole_and_of_their_type():
    x, pos = torch.zeros(2, 3, 2, 64), torch.zeros(2, 3, dtype=torch.int32)
    table = torch.zeros(64, dtype=torch.int64)
    for bad in (table[:33], table[::2], table[:32].int(), table[:32].double()):  # 64 channels: 32 words
        with pytest.raises(ValueError):
            dd.dllm_rope_phases(64, bad)
    for bad in (table[::2], table[:32].int(), table[:32].double(), table[:32].float()):
        with pytest.raises(ValueError):
            dd.dllm_qk_norm_rope(x, None, x, None, pos, bad)


def test_a_cache_follows_the_table_it_is_given():
    c = dd.Kv4Cache(4, 2, 16, 64, 2, 2, device="cpu")
    other = torch.zeros(3, 5, dtype=torch.int32)
    c.table = other
    assert c.table is other and c.B == 3
    assert c.c().page_table == other.data_ptr() and c.c().table_stride == 5
    assert c.ref._obj.page_table == other.data_ptr()
    for bad in (other.float(), other.long(), other[:, ::2], other[0], other.t()):
        with pytest.raises(ValueError):
            c.table = bad
    assert c.table is other
    for name in ("k_codes", "k_params", "v_codes", "v_params"):  # a cache over others is made by `of`
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name).clone())
    c.k_codes += 1  # in place is no other tensor


def test_a_cache_over_arrays_of_other_types_is_refused():
    c = dd.Kv4Cache(4, 2, 16, 64, 2, 2, device="cpu")
    arrays = dict(k_codes=c.k_codes, k_params=c.k_params, v_codes=c.v_codes, v_params=c.v_params,
                  table=c.table)
    dd.Kv4Cache.of(**arrays)
    for name, dtype in (("k_codes", torch.bool), ("v_codes", torch.int8), ("k_params", torch.bfloat16),
                        ("v_params", torch.float16), ("table", torch.float32)):
        with pytest.raises(ValueError):
            dd.Kv4Cache.of(**{**arrays, name: arrays[name].to(dtype)})
    for name in ("k_params", "v_params"):  # the same words, unsigned
        dd.Kv4Cache.of(**{**arrays, name: arrays[name].view(torch.uint16)})


def test_norm_rope_of_nothing_is_refused():
    with pytest.raises(ValueError):
        dd.dllm_qk_norm_rope(None, None, None, None, None, None)

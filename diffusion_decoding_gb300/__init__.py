"""Python binding of ``libdllm`` — the GB300 (sm_103a) parallel-decode step of a diffusion LM.

Each ``dllm_*`` function here marshals its arguments and calls the C entry point of the same
name (``include/dllm.h``); every step of the computation runs in the library's CUDA kernels.
Tensors must live on the current CUDA device; PyTorch provides device memory and streams only.

The library is built in-tree by ``diffusion_decoding_gb300.build.build()``.  Importing works
without it (so that host-side code and the CPU tests run), but every call raises if the shared
library is missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdllm.so")

DLLM_OK, DLLM_ERR_INVALID_ARG, DLLM_ERR_UNSUPPORTED, DLLM_ERR_CUDA, DLLM_ERR_TIMEOUT = range(5)
DLLM_F32, DLLM_BF16 = 0, 1
DLLM_ROPE_LINEAR, DLLM_ROPE_BANDS = 0, 1

_c_i32, _c_i64, _c_f32, _c_vp, _c_sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                        ctypes.c_void_p, ctypes.c_size_t)


class DllmError(RuntimeError):
    def __init__(self, status: int, name: str, msg: str):
        super().__init__(f"{name} -> status {status}: {msg}")
        self.status = status


class dllm_shape(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("L", _c_i32), ("V", _c_i32), ("dtype", _c_i32),
                ("row_stride", _c_i64)]


class dllm_block_state(ctypes.Structure):
    _fields_ = [("masked", _c_vp), ("tokens", _c_vp), ("committed_now", _c_vp),
                ("n_commit", _c_vp), ("eos_hit", _c_vp)]


class dllm_stats(ctypes.Structure):
    _fields_ = [("row_max", _c_vp), ("lse", _c_vp), ("conf", _c_vp), ("argmax", _c_vp)]


class dllm_shard_stats(ctypes.Structure):
    _fields_ = [("stats", dllm_stats), ("vocab_offset", _c_i64)]


class dllm_heads(ctypes.Structure):
    _fields_ = [("data", _c_vp), ("heads", _c_i32), ("dtype", _c_i32), ("batch_stride", _c_i64),
                ("token_stride", _c_i64), ("head_stride", _c_i64)]


class dllm_rope(ctypes.Structure):
    _fields_ = [("rotary_dim", _c_i32), ("scaling", _c_i32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("slow_turns", ctypes.c_double), ("fast_turns", ctypes.c_double)]


class dllm_sampling(ctypes.Structure):
    _fields_ = [("temperature", _c_f32), ("top_k", _c_i32), ("top_p", _c_f32), ("min_p", _c_f32)]


class dllm_kv4_cache(ctypes.Structure):
    _fields_ = [("k_codes", _c_vp), ("k_params", _c_vp), ("v_codes", _c_vp), ("v_params", _c_vp),
                ("page_table", _c_vp), ("pages", _c_i32), ("heads", _c_i32),
                ("page_size", _c_i32), ("head_dim", _c_i32), ("table_stride", _c_i32)]


_byref = ctypes.byref
_P_HEADS = _c_vp  # const dllm_heads*: byref of the structure, or its bytes
_P_CACHE = ctypes.POINTER(dllm_kv4_cache)

_SIGS = {
    "dllm_last_error": (ctypes.c_char_p, []),
    "dllm_workspace_bytes": (_c_sz, [ctypes.POINTER(dllm_shape)]),
    "dllm_decode_stats": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape), _c_vp,
                                   ctypes.POINTER(dllm_stats), _c_vp, _c_vp]),
    "dllm_sample": (_c_i32, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "dllm_commit_threshold": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                       ctypes.POINTER(dllm_stats),
                                       ctypes.POINTER(dllm_block_state), _c_f32, _c_i32, _c_vp,
                                       _c_vp]),
    "dllm_commit_hierarchical": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                          ctypes.POINTER(dllm_stats),
                                          ctypes.POINTER(dllm_block_state), _c_f32, _c_i32,
                                          _c_i32, _c_vp, _c_vp]),
    "dllm_commit_hierarchical_levels": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                                 ctypes.POINTER(dllm_stats),
                                                 ctypes.POINTER(dllm_block_state), _c_f32,
                                                 _c_i32, _c_i32, _c_vp, _c_vp]),
    "dllm_commit_credit_tracked": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                            ctypes.POINTER(dllm_stats),
                                            ctypes.POINTER(dllm_block_state), _c_vp, _c_vp,
                                            _c_i32, _c_f32, _c_f32, _c_f32, _c_i32, _c_vp,
                                            _c_vp]),
    "dllm_commit_credit": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                    ctypes.POINTER(dllm_stats), ctypes.POINTER(dllm_block_state),
                                    _c_vp, _c_vp, _c_i32, _c_f32, _c_f32, _c_f32, _c_i32, _c_vp,
                                    _c_vp]),
    "dllm_embedding_t_elems": (_c_sz, [_c_i32, _c_i32]),
    "dllm_prepare_embedding": (_c_i32, [_c_vp, _c_i32, _c_i32, _c_vp, _c_vp]),
    "dllm_smooth_workspace_bytes": (_c_sz, [ctypes.POINTER(dllm_shape), _c_i32]),
    "dllm_smooth_embed": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape), ctypes.POINTER(dllm_stats),
                                   ctypes.POINTER(dllm_block_state), _c_vp, _c_i32, _c_vp, _c_vp,
                                   _c_vp, _c_vp, _c_sz, _c_vp]),
    "dllm_smooth_plan_info": (_c_i32, [ctypes.POINTER(dllm_shape), _c_i32, _c_vp]),
    "dllm_commit_threshold_smooth": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                              ctypes.POINTER(dllm_stats),
                                              ctypes.POINTER(dllm_block_state), _c_f32, _c_i32,
                                              _c_vp, _c_i32, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz,
                                              _c_vp]),
    "dllm_smooth_probs": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape), ctypes.POINTER(dllm_stats),
                                   ctypes.POINTER(dllm_block_state), _c_i32, _c_vp, _c_vp, _c_vp,
                                   _c_sz, _c_vp]),
    "dllm_smooth_gemm": (_c_i32, [ctypes.POINTER(dllm_shape), _c_vp, _c_i32, _c_vp, _c_vp, _c_vp,
                                  _c_sz, _c_vp]),
    "dllm_block_state_reset": (_c_i32, [ctypes.POINTER(dllm_block_state), _c_i32, _c_i32, _c_vp,
                                        _c_vp, _c_i32, _c_vp]),
    "dllm_kv_refresh_mask": (_c_i32, [ctypes.POINTER(dllm_block_state), _c_i32, _c_i32, _c_i32,
                                      _c_i32, _c_vp, _c_vp, _c_vp, _c_vp]),
    "dllm_rope_phases": (_c_i32, [ctypes.POINTER(dllm_rope), _c_vp, _c_vp]),
    "dllm_qk_norm_rope": (_c_i32, [_P_HEADS, _P_HEADS, _P_HEADS, _P_HEADS, _c_i32, _c_i32, _c_i32,
                                   _c_vp, _c_i64, _c_vp, _c_i32, _c_i32, _c_f32, _c_i32, _c_vp,
                                   _c_vp, _c_f32, _c_vp]),
    "dllm_kv4_write": (_c_i32, [_P_CACHE, _P_HEADS, _P_HEADS, _c_i32, _c_i32, _c_vp, _c_i64,
                                _c_vp]),
    "dllm_kv4_read": (_c_i32, [_P_CACHE, _P_HEADS, _P_HEADS, _c_i32, _c_i32, _c_vp, _c_i64,
                               _c_vp]),
    "dllm_attention_kv4_workspace_bytes": (_c_sz, [_P_CACHE, _c_i32, _c_i32, _c_i32, _c_i32]),
    "dllm_attention_kv4": (_c_i32, [_P_HEADS, _P_CACHE, _c_vp, _c_i32, _c_vp, _c_i64, _c_f32,
                                    _c_i32, _P_HEADS, _c_vp, _c_i32, _c_i32, _c_vp, _c_sz,
                                    _c_vp]),
    "dllm_attention_kv4_weights_workspace_bytes": (_c_sz, [_P_CACHE, _c_i32, _c_i32, _c_i32, _c_i32]),
    "dllm_attention_kv4_weights": (_c_i32, [_P_HEADS, _P_CACHE, _c_vp, _c_i32, _c_vp, _c_i64, _c_f32,
                                            _c_i32, _c_vp, _c_vp, _c_i64, _c_f32, _c_vp, _c_i64,
                                            _c_i32, _c_i32, _c_vp, _c_sz, _c_vp]),
    "dllm_kv4_evict_workspace_bytes": (_c_sz, [_P_CACHE, _c_i32, _c_i32]),
    "dllm_kv4_evict": (_c_i32, [_P_CACHE, _c_vp, _c_i64, _c_vp, _c_i32, _c_i32, _c_i32, _c_i32, _c_vp,
                                _c_i64, _c_vp, _c_vp, _c_i64, _c_i32, _c_vp, _c_sz, _c_vp]),
    "dllm_get_status": (_c_i32, [_c_vp, _c_vp, ctypes.POINTER(_c_i32)]),
    "dllm_merge_shard_stats": (_c_i32, [ctypes.POINTER(dllm_shard_stats), _c_i32, _c_i64,
                                        ctypes.POINTER(dllm_stats), _c_vp]),
    "dllm_selftest_wait_timeout": (_c_i32, [_c_vp, ctypes.c_uint32, _c_vp]),
    "dllm_commit_threshold_static": (_c_i32, [_c_vp, ctypes.POINTER(dllm_shape),
                                              ctypes.POINTER(dllm_stats),
                                              ctypes.POINTER(dllm_block_state), _c_f32, _c_i32,
                                              _c_vp]),
    "dllm_capture_condition": (_c_i32, [_c_vp, ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint64)]),
    "dllm_capture_if_begin": (_c_i32, [_c_vp, _c_vp, ctypes.c_uint64]),
    "dllm_capture_if_end": (_c_i32, [_c_vp]),
    "dllm_loop_continue": (_c_i32, [ctypes.POINTER(dllm_block_state), _c_i32, _c_i32,
                                    ctypes.c_uint64, _c_vp]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "diffusion_decoding_gb300.build.build() (no CPU fallback exists)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# The current stream's handle without a Stream object around it (a quarter of the time).
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               if hasattr(torch._C, "_cuda_getDevice") else None)


def _check(status: int, name: str) -> None:
    if status != DLLM_OK:
        raise DllmError(status, name, lib().dllm_last_error().decode())


# ------------------------------------------------------------------ descriptors

def make_shape(B: int, L: int, V: int, dtype: int, row_stride: int | None = None) -> dllm_shape:
    return dllm_shape(B, L, V, dtype, V if row_stride is None else row_stride)


def shape_of(logits: torch.Tensor) -> dllm_shape:
    """Shape descriptor of a [B, L, V] (or [B, L, row_stride] sliced to V) logits tensor."""
    B, L, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = DLLM_BF16
    elif logits.dtype == torch.float32:
        dt = DLLM_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    if logits.stride(2) != 1 or logits.stride(0) != L * logits.stride(1):
        raise ValueError("logits rows must be contiguous and evenly strided")
    return dllm_shape(B, L, V, dt, logits.stride(1))


class StatsBuffers:
    """Device arrays for row_max, lse, conf and argmax ([B*L] each)."""

    def __init__(self, R: int, device=None):
        dev = device or torch.device("cuda")
        self.row_max = torch.empty(R, dtype=torch.float32, device=dev)
        self.lse = torch.empty(R, dtype=torch.float32, device=dev)
        self.conf = torch.empty(R, dtype=torch.float32, device=dev)
        self.argmax = torch.empty(R, dtype=torch.int32, device=dev)

    def c(self) -> dllm_stats:
        return dllm_stats(_ptr(self.row_max), _ptr(self.lse), _ptr(self.conf), _ptr(self.argmax))


class BlockState:
    """Device decode state of B blocks of L positions (fresh: everything masked)."""

    def __init__(self, B: int, L: int, K: int = 0, device=None):
        dev = device or torch.device("cuda")
        self.B, self.L, self.K = B, L, K
        self.masked = torch.ones(B * L, dtype=torch.uint8, device=dev)
        self.tokens = torch.full((B * L,), -1, dtype=torch.int32, device=dev)
        self.committed_now = torch.zeros(B * L, dtype=torch.uint8, device=dev)
        self.n_commit = torch.zeros(B, dtype=torch.int32, device=dev)
        self.eos_hit = torch.zeros(B, dtype=torch.int32, device=dev)
        self.cand_id = torch.full((B * L, max(K, 1)), -1, dtype=torch.int32, device=dev)
        self.cand_credit = torch.zeros((B * L, max(K, 1)), dtype=torch.float32, device=dev)

    def c(self) -> dllm_block_state:
        return dllm_block_state(_ptr(self.masked), _ptr(self.tokens), _ptr(self.committed_now),
                                _ptr(self.n_commit), _ptr(self.eos_hit))

    def reset(self, stream=None) -> None:
        """A new block, by one kernel (dllm_block_state_reset), credit slots included."""
        dllm_block_state_reset(self, stream=stream)


def _kept(i: int) -> property:
    """Array i of a cache: its descriptor holds the address, so no other tensor can be assigned."""
    def put(self, t):
        if t is not self._arrays[i]:
            raise AttributeError("a cache keeps its arrays; Kv4Cache.of makes one over others")
    return property(lambda self: self._arrays[i], put)


class Kv4Cache:
    """Device arrays of a paged 4-bit key/value cache (format: include/dllm.h) and its page table.

    pages: pages in the pool; table: [B, pages per sequence] int32 page ids (a word outside
    [0, pages) is an absent page).  The table's words may be changed between calls, and `table` may be
    set to another tensor; codes and params need no initial values and stay the same tensors."""

    def __init__(self, pages: int, heads: int, page_size: int, head_dim: int, B: int,
                 pages_per_seq: int, device=None):
        dev = device or torch.device("cuda")
        codes, params = (pages, heads, page_size, head_dim // 2), (pages, heads, page_size,
                                                                   head_dim // 32)
        self._set(torch.empty(codes, dtype=torch.uint8, device=dev),
                  torch.empty(params, dtype=torch.int16, device=dev),
                  torch.empty(codes, dtype=torch.uint8, device=dev),
                  torch.empty(params, dtype=torch.int16, device=dev),
                  torch.full((B, pages_per_seq), -1, dtype=torch.int32, device=dev))

    @classmethod
    def of(cls, k_codes, k_params, v_codes, v_params, table) -> "Kv4Cache":
        """A cache over existing contiguous device tensors (shapes as the constructor makes)."""
        self = cls.__new__(cls)
        pages, heads, page_size, half = k_codes.shape
        codes, params = (torch.uint8,), (torch.int16, torch.uint16)
        for name, t, shape, types in (
                ("k_codes", k_codes, k_codes.shape, codes), ("v_codes", v_codes, k_codes.shape, codes),
                ("k_params", k_params, (pages, heads, page_size, half // 16), params),
                ("v_params", v_params, (pages, heads, page_size, half // 16), params)):
            if tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.dtype not in types:
                raise ValueError(f"{name} must be contiguous, {tuple(shape)}, {types[0]}")
        self._set(k_codes, k_params, v_codes, v_params, table)
        return self

    def _set(self, k_codes, k_params, v_codes, v_params, table) -> None:
        self._arrays = (k_codes, k_params, v_codes, v_params)
        pages, heads, page_size, half = k_codes.shape
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, page_size, 2 * half
        self._c = dllm_kv4_cache(*map(_ptr, self._arrays), None, pages, heads, page_size, 2 * half, 0)
        self.ref = _byref(self._c)
        self.table = table

    k_codes, k_params, v_codes, v_params = map(_kept, range(4))

    @property
    def table(self) -> torch.Tensor:
        return self._table

    @table.setter
    def table(self, table: torch.Tensor) -> None:
        if table.dtype is not torch.int32 or table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be [B, pages of a sequence] int32, contiguous")
        self._table, self.B = table, table.shape[0]
        self._c.page_table, self._c.table_stride = _ptr(table), table.shape[1]

    def c(self) -> dllm_kv4_cache:
        return self._c


_DTYPES = {torch.float32: DLLM_F32, torch.bfloat16: DLLM_BF16}
_pack_heads = struct.Struct("Pii3q").pack  # dllm_heads
assert struct.calcsize("Pii3q") == ctypes.sizeof(dllm_heads)
_pack_stats = struct.Struct("4P").pack  # dllm_stats
_pack_sampling = struct.Struct("fi2f").pack  # dllm_sampling
assert struct.calcsize("fi2f") == ctypes.sizeof(dllm_sampling)


def heads_of(t: torch.Tensor) -> dllm_heads:
    """Descriptor of a [B, n, heads, head_dim] bf16 or fp32 tensor with contiguous channels."""
    if t.dim() != 4:
        raise ValueError("need a [B, n, heads, head_dim] tensor")
    return dllm_heads.from_buffer_copy(_rows(t, t.shape[0], t.shape[1], t.shape[3]))


def _rows(t: torch.Tensor, B: int, n: int, D: int) -> bytes:
    """The bytes of heads_of a tensor that has to be [B, n, any, D] (a ctypes structure takes longer
    to make than they do, and a small call takes as long as the host needs to make it)."""
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError("need bfloat16 or float32")
    stride = t.stride()
    if len(stride) != 4:
        raise ValueError("need [B, n, heads, head_dim] tensors")
    b, m, h, d = t.shape
    sb, st, sh, sc = stride
    if b != B or m != n or d != D:
        raise ValueError("the tensors differ in B, n or head_dim")
    if sc != 1 and d != 1:
        raise ValueError("channels must be contiguous")
    return _pack_heads(t.data_ptr(), h, dt, sb, st, sh)


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zero-filled device workspace (256-byte aligned: torch allocations are 512-aligned)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------ entry points

def dllm_workspace_bytes(shape: dllm_shape) -> int:
    return int(lib().dllm_workspace_bytes(ctypes.byref(shape)))


def _check_stats(stats: StatsBuffers, rows: int) -> None:
    """Calls write (or read) as many rows as the shape has, whatever the buffers hold."""
    if stats.row_max.numel() < rows or stats.lse.numel() < rows or stats.conf.numel() < rows \
            or stats.argmax.numel() < rows:
        raise ValueError("the statistics buffers hold fewer than B*L rows")


def _stats_c(stats: StatsBuffers, shape: dllm_shape) -> dllm_stats:
    _check_stats(stats, shape.B * shape.L)
    return stats.c()


def dllm_decode_stats(logits, shape, masked, stats: StatsBuffers, ws, stream=None) -> None:
    st = _stats_c(stats, shape)
    _check(lib().dllm_decode_stats(_ptr(logits), ctypes.byref(shape), _ptr(masked),
                                   ctypes.byref(st), _ptr(ws), _stream(stream)),
           "dllm_decode_stats")


def dllm_sample(logits, shape, masked, uniform, stats: StatsBuffers, temperature: float = 1.0,
                top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0, stream=None) -> None:
    """Draw a token per row (into stats.argmax, its model probability into stats.conf); uniform:
    [B*L] fp32 numbers in [0, 1); masked: [B*L] uint8 or None; filters: see include/dllm.h."""
    rows, open_ = shape.B * shape.L, None
    if uniform.dtype is not torch.float32 or uniform.numel() != rows or not uniform.is_contiguous():
        raise ValueError("uniform must be [B*L] float32, contiguous")
    if masked is not None:
        if masked.element_size() != 1 or masked.numel() != rows or not masked.is_contiguous():
            raise ValueError("masked must be [B*L] uint8, contiguous")
        open_ = masked.data_ptr()
    _check_stats(stats, rows)
    out = _pack_stats(stats.row_max.data_ptr(), stats.lse.data_ptr(), stats.conf.data_ptr(),
                      stats.argmax.data_ptr())
    status = lib().dllm_sample(_ptr(logits), _byref(shape), open_, uniform.data_ptr(),
                               _pack_sampling(temperature, top_k, top_p, min_p), out, _stream(stream))
    if status:
        _check(status, "dllm_sample")


def dllm_commit_threshold(logits, shape, stats: StatsBuffers, state: BlockState, tau: float,
                          eos_id: int, ws, stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_threshold(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                       ctypes.byref(bs), tau, eos_id, _ptr(ws), _stream(stream)),
           "dllm_commit_threshold")


def dllm_commit_hierarchical(logits, shape, stats: StatsBuffers, state: BlockState,
                             tau_low: float, min_width: int, eos_id: int, ws,
                             stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_hierarchical(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                          ctypes.byref(bs), tau_low, min_width, eos_id, _ptr(ws),
                                          _stream(stream)),
           "dllm_commit_hierarchical")


def dllm_commit_hierarchical_levels(logits, shape, stats: StatsBuffers, state: BlockState,
                                    tau_low: float, min_width: int, eos_id: int, ws,
                                    stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_hierarchical_levels(_ptr(logits), ctypes.byref(shape),
                                                 ctypes.byref(st), ctypes.byref(bs), tau_low,
                                                 min_width, eos_id, _ptr(ws), _stream(stream)),
           "dllm_commit_hierarchical_levels")


def dllm_commit_credit_tracked(logits, shape, stats: StatsBuffers, state: BlockState, K: int,
                               decay: float, boost: float, tau: float, eos_id: int, ws,
                               stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_credit_tracked(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                            ctypes.byref(bs), _ptr(state.cand_id),
                                            _ptr(state.cand_credit), K, decay, boost, tau, eos_id,
                                            _ptr(ws), _stream(stream)),
           "dllm_commit_credit_tracked")


def dllm_commit_credit(logits, shape, stats: StatsBuffers, state: BlockState, K: int,
                       decay: float, boost: float, tau: float, eos_id: int, ws,
                       stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_credit(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                    ctypes.byref(bs), _ptr(state.cand_id),
                                    _ptr(state.cand_credit), K, decay, boost, tau, eos_id,
                                    _ptr(ws), _stream(stream)),
           "dllm_commit_credit")


def dllm_embedding_t_elems(V: int, d: int) -> int:
    return int(lib().dllm_embedding_t_elems(V, d))


def dllm_prepare_embedding(E: torch.Tensor, Et: torch.Tensor, stream=None) -> None:
    """E: [V, d] bf16 (or int16 bit patterns); Et: dllm_embedding_t_elems(V, d) elements."""
    V, d = E.shape
    _check(lib().dllm_prepare_embedding(_ptr(E), V, d, _ptr(Et), _stream(stream)),
           "dllm_prepare_embedding")


def dllm_smooth_workspace_bytes(shape: dllm_shape, d: int) -> int:
    return int(lib().dllm_smooth_workspace_bytes(ctypes.byref(shape), d))


def dllm_smooth_embed(logits, shape, stats: StatsBuffers, state: BlockState, Et, d: int, out,
                      row_ids, M, ws, stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_smooth_embed(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                   ctypes.byref(bs), _ptr(Et), d, _ptr(out), _ptr(row_ids),
                                   _ptr(M), _ptr(ws), ws.numel(), _stream(stream)),
           "dllm_smooth_embed")


def dllm_commit_threshold_smooth(logits, shape, stats: StatsBuffers, state: BlockState,
                                 tau: float, eos_id: int, Et, d: int, out, row_ids, M, ws,
                                 stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_threshold_smooth(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                              ctypes.byref(bs), tau, eos_id, _ptr(Et), d,
                                              _ptr(out), _ptr(row_ids), _ptr(M), _ptr(ws),
                                              ws.numel(), _stream(stream)),
           "dllm_commit_threshold_smooth")


def dllm_smooth_plan_info(shape, d: int) -> dict:
    info = (_c_i32 * 6)()
    _check(lib().dllm_smooth_plan_info(ctypes.byref(shape), d, info), "dllm_smooth_plan_info")
    keys = ("m_tiles", "n_tiles", "bn_max", "split_k", "stages", "launches")
    return dict(zip(keys, (int(x) for x in info)))


def dllm_smooth_probs(logits, shape, stats: StatsBuffers, state: BlockState, d: int, row_ids, M,
                      ws, stream=None) -> None:
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_smooth_probs(_ptr(logits), ctypes.byref(shape), ctypes.byref(st),
                                   ctypes.byref(bs), d, _ptr(row_ids), _ptr(M), _ptr(ws),
                                   ws.numel(), _stream(stream)),
           "dllm_smooth_probs")


def dllm_smooth_gemm(shape, Et, d: int, out, M, ws, stream=None) -> None:
    _check(lib().dllm_smooth_gemm(ctypes.byref(shape), _ptr(Et), d, _ptr(out), _ptr(M), _ptr(ws),
                                  ws.numel(), _stream(stream)),
           "dllm_smooth_gemm")


def dllm_block_state_reset(state: BlockState, credit: bool = True, stream=None) -> None:
    bs = state.c()
    K = state.cand_id.shape[1]
    _check(lib().dllm_block_state_reset(ctypes.byref(bs), state.B, state.L,
                                        _ptr(state.cand_id) if credit else None,
                                        _ptr(state.cand_credit) if credit else None,
                                        K if credit else 0, _stream(stream)),
           "dllm_block_state_reset")


def dllm_kv_refresh_mask(state: BlockState, prefix_len: int, window: int, refresh, idx, count,
                         stream=None) -> None:
    bs = state.c()
    _check(lib().dllm_kv_refresh_mask(ctypes.byref(bs), state.B, state.L, prefix_len, window,
                                      _ptr(refresh), _ptr(idx), _ptr(count), _stream(stream)),
           "dllm_kv_refresh_mask")


def dllm_commit_threshold_static(logits, shape, stats: StatsBuffers, state: BlockState, tau: float,
                                 eos_id: int, stream=None) -> None:
    """dllm_commit_threshold for callers that cannot allocate: no workspace argument, the
    scratch is a fixed static array inside the library (see include/dllm.h)."""
    st, bs = _stats_c(stats, shape), state.c()
    _check(lib().dllm_commit_threshold_static(_ptr(logits), ctypes.byref(shape),
                                              ctypes.byref(st), ctypes.byref(bs), tau, eos_id,
                                              _stream(stream)),
           "dllm_commit_threshold_static")


def dllm_rope_phases(rotary_dim: int, phases: torch.Tensor, base: float = 10000.0,
                     factor: float = 1.0, scaling: int = DLLM_ROPE_LINEAR,
                     original_len: float = 0.0, slow_turns: float = 1.0, fast_turns: float = 32.0,
                     stream=None) -> None:
    """Fill phases ([rotary_dim / 2] int64) with each pair's turns per position in 2^-64."""
    # as many words as pairs: dllm_qk_norm_rope rotates two channels for every word it is given
    if phases.dtype is not torch.int64 or phases.numel() != rotary_dim // 2 \
            or not phases.is_contiguous():
        raise ValueError("phases must be rotary_dim / 2 int64 words, contiguous")
    r = dllm_rope(rotary_dim, scaling, base, factor, original_len, slow_turns, fast_turns)
    _check(lib().dllm_rope_phases(ctypes.byref(r), _ptr(phases), _stream(stream)),
           "dllm_rope_phases")


def _pos_stride(pos, B: int, n: int) -> int:
    if pos is None:
        return 0
    if pos.dtype is not torch.int32 or pos.dim() != 2:
        raise ValueError("pos must be [B, >= n] int32")
    b, m = pos.shape
    stride, unit = pos.stride()
    if b != B or m < n or (unit != 1 and m != 1):
        raise ValueError("pos must be [B, >= n] int32 with contiguous rows")
    return stride


def dllm_qk_norm_rope(q, k, q_out, k_out, pos, phases, q_weight=None, k_weight=None,
                      eps: float = 1e-6, interleaved: bool = False, magnitude: float = 1.0,
                      norm: bool = True, stream=None) -> None:
    """q, k and their outputs: [B, n, heads, head_dim] (any strides with contiguous channels; q or
    k with its output may be None); pos: [B, >= n] int32, < 0: token skipped; phases: the
    dllm_rope_phases table, two channels per entry are rotated (None: no rotation)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("need q with q_out, or k with k_out, or both pairs")
    B, n, _, D = x.shape
    dtype = x.dtype
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not dtype or w.numel() != D or not w.is_contiguous()):
            raise ValueError("weights must be contiguous, [head_dim], of the tensors' dtype")
    if phases is not None and (phases.dtype is not torch.int64 or not phases.is_contiguous()):
        raise ValueError("phases must be a contiguous int64 table")
    hq = hqo = hk = hko = None
    if q is not None:
        hq = _rows(q, B, n, D)
    if q_out is not None:
        hqo = _rows(q_out, B, n, D)
    if k is not None:
        hk = _rows(k, B, n, D)
    if k_out is not None:
        hko = _rows(k_out, B, n, D)
    status = lib().dllm_qk_norm_rope(
        hq, hqo, hk, hko, B, n, D, _ptr(pos), _pos_stride(pos, B, n), _ptr(phases),
        0 if phases is None else 2 * phases.numel(), interleaved, magnitude, norm, _ptr(q_weight),
        _ptr(k_weight), eps, _stream(stream))
    if status:
        _check(status, "dllm_qk_norm_rope")


def _cache_rows(cache: Kv4Cache, k, v, pos):
    B, n, _, D = k.shape
    if D != cache.head_dim or B != cache.B:
        raise ValueError("k and v must be [B, n, heads, head_dim] of the cache")
    return (cache.ref, _rows(k, B, n, D), _rows(v, B, n, D), B, n, _ptr(pos),
            _pos_stride(pos, B, n))


def dllm_kv4_write(cache: Kv4Cache, k, v, pos, stream=None) -> None:
    """Quantise k, v ([B, n, heads, head_dim]) into the entries pos ([B, >= n] int32, < 0: skip)."""
    status = lib().dllm_kv4_write(*_cache_rows(cache, k, v, pos), _stream(stream))
    if status:
        _check(status, "dllm_kv4_write")


def dllm_kv4_read(cache: Kv4Cache, k, v, pos=None, stream=None) -> None:
    """Read the entries pos (None: 0 .. n-1) back into k, v ([B, n, heads, head_dim])."""
    status = lib().dllm_kv4_read(*_cache_rows(cache, k, v, pos), _stream(stream))
    if status:
        _check(status, "dllm_kv4_read")


def dllm_attention_kv4_workspace_bytes(cache: Kv4Cache, B: int, n: int, q_heads: int,
                                       max_len: int) -> int:
    return int(lib().dllm_attention_kv4_workspace_bytes(cache.ref, B, n, q_heads, max_len))


def dllm_attention_kv4(q, cache: Kv4Cache, lens, max_len: int, out, ws, lse=None, key_mask=None,
                       scale: float | None = None, causal: bool = False, stream=None) -> None:
    """q, out: [B, n, heads, head_dim] bf16; lens: [B] int32 (None: max_len everywhere); lse:
    [B, heads, n] fp32 or None; key_mask: [B, >= max_len] uint8 or bool with contiguous rows (it may
    be one row expanded to all sequences), 0 = hidden; scale: None for head_dim ** -0.5."""
    B, n, H, D = q.shape
    if D != cache.head_dim or B != cache.B:
        raise ValueError("q and out must be [B, n, heads, head_dim] of the cache")
    if lens is not None and (lens.dtype is not torch.int32 or lens.numel() != B
                             or not lens.is_contiguous()):
        raise ValueError("lens must be [B] int32, contiguous")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (B, H, n)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be [B, heads, n] float32, contiguous")
    mask_stride = 0
    if key_mask is not None:
        if key_mask.element_size() != 1 or key_mask.dim() != 2 or key_mask.shape[0] != B \
                or key_mask.shape[1] < max_len or (key_mask.stride(1) != 1 and key_mask.shape[1] != 1):
            raise ValueError("key_mask must be [B, >= max_len] uint8 or bool with contiguous rows")
        mask_stride = key_mask.stride(0)
    status = lib().dllm_attention_kv4(
        _rows(q, B, n, D), cache.ref, _ptr(lens), max_len, _ptr(key_mask), mask_stride,
        D ** -0.5 if scale is None else scale, causal, _rows(out, B, n, D), _ptr(lse), B, n,
        _ptr(ws), ws.numel(), _stream(stream))
    if status:
        _check(status, "dllm_attention_kv4")


def _word_rows(t, name: str, B: int, max_len: int, dtype=torch.float32) -> int:
    """Stride of the rows of a [B, >= max_len] tensor of 32-bit words (0: none)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.dim() != 2 or t.shape[0] != B or t.shape[1] < max_len \
            or (t.stride(1) != 1 and t.shape[1] != 1):
        raise ValueError(f"{name} must be [B, >= max_len] {dtype} with contiguous rows")
    return t.stride(0)


def _lens(lens, name: str, B: int):
    if lens is not None and (lens.dtype is not torch.int32 or lens.numel() != B
                             or not lens.is_contiguous()):
        raise ValueError(f"{name} must be [B] int32, contiguous")
    return _ptr(lens)


def dllm_attention_kv4_weights_workspace_bytes(cache: Kv4Cache, B: int, n: int, q_heads: int,
                                               max_len: int) -> int:
    return int(lib().dllm_attention_kv4_weights_workspace_bytes(cache.ref, B, n, q_heads, max_len))


def dllm_attention_kv4_weights(q, cache: Kv4Cache, lens, max_len: int, lse, weights, ws, prior=None,
                               keep: float = 1.0, key_mask=None, scale: float | None = None,
                               causal: bool = False, stream=None) -> None:
    """weights[b, j] = keep * prior[b, j] + the attention that entry j receives from all queries and
    heads; q, lens, max_len, key_mask, scale, causal as given to dllm_attention_kv4, lse ([B, heads, n])
    as it wrote it; weights, prior: [B, >= max_len] fp32 (prior may be weights, or None)."""
    B, n, H, D = q.shape
    if D != cache.head_dim or B != cache.B:
        raise ValueError("q must be [B, n, heads, head_dim] of the cache")
    if lse.dtype is not torch.float32 or lse.shape != (B, H, n) or not lse.is_contiguous():
        raise ValueError("lse must be [B, heads, n] float32, contiguous")
    mask_stride = 0
    if key_mask is not None:
        if key_mask.element_size() != 1 or key_mask.dim() != 2 or key_mask.shape[0] != B \
                or key_mask.shape[1] < max_len or (key_mask.stride(1) != 1 and key_mask.shape[1] != 1):
            raise ValueError("key_mask must be [B, >= max_len] uint8 or bool with contiguous rows")
        mask_stride = key_mask.stride(0)
    status = lib().dllm_attention_kv4_weights(
        _rows(q, B, n, D), cache.ref, _lens(lens, "lens", B), max_len, _ptr(key_mask), mask_stride,
        D ** -0.5 if scale is None else scale, causal, _ptr(lse), _ptr(prior),
        _word_rows(prior, "prior", B, max_len), keep, _ptr(weights),
        _word_rows(weights, "weights", B, max_len), B, n, _ptr(ws), ws.numel(), _stream(stream))
    if status:
        _check(status, "dllm_attention_kv4_weights")


def dllm_kv4_evict_workspace_bytes(cache: Kv4Cache, B: int, max_len: int) -> int:
    return int(lib().dllm_kv4_evict_workspace_bytes(cache.ref, B, max_len))


def dllm_kv4_evict(cache: Kv4Cache, weights, lens, max_len: int, budget: int, slots, lens_out, ws,
                   first: int = 0, last: int = 0, weights_out=None, stream=None) -> None:
    """Cut every sequence to its `budget` entries of largest weight ([B, >= max_len] fp32; the first
    `first` and last `last` always stay).  slots ([B, >= max_len] int32): where each entry is now, -1
    if dropped; lens_out ([B] int32; may be lens): the new lengths; weights_out (may be weights): the
    weights in the new order."""
    B = cache.B
    if weights is None or slots is None or lens_out is None:
        raise ValueError("weights, slots and lens_out are needed")
    status = lib().dllm_kv4_evict(
        cache.ref, _ptr(weights), _word_rows(weights, "weights", B, max_len), _lens(lens, "lens", B),
        max_len, budget, first, last, _ptr(slots), _word_rows(slots, "slots", B, max_len, torch.int32),
        _lens(lens_out, "lens_out", B), _ptr(weights_out),
        _word_rows(weights_out, "weights_out", B, max_len), B, _ptr(ws), ws.numel(), _stream(stream))
    if status:
        _check(status, "dllm_kv4_evict")


def dllm_capture_condition(default_value: int = 0, stream=None) -> int:
    """A condition handle in the graph `stream` is capturing (see include/dllm.h)."""
    h = ctypes.c_uint64(0)
    _check(lib().dllm_capture_condition(_stream(stream), int(default_value), ctypes.byref(h)),
           "dllm_capture_condition")
    return int(h.value)


def dllm_capture_if_begin(handle: int, body_stream, stream=None) -> None:
    """Conditional IF node on `handle` in the graph `stream` is capturing; its body is captured
    on body_stream until dllm_capture_if_end."""
    _check(lib().dllm_capture_if_begin(_stream(stream), body_stream.cuda_stream, int(handle)),
           "dllm_capture_if_begin")


def dllm_capture_if_end(body_stream) -> None:
    _check(lib().dllm_capture_if_end(body_stream.cuda_stream), "dllm_capture_if_end")


def dllm_loop_continue(state: BlockState, handle: int, stream=None) -> None:
    """Inside a capture: sets `handle` to whether some sequence of the block still decodes."""
    bs = state.c()
    _check(lib().dllm_loop_continue(ctypes.byref(bs), state.B, state.L, int(handle),
                                    _stream(stream)), "dllm_loop_continue")


def dllm_selftest_wait_timeout(ws, limit_us: int, stream=None) -> None:
    _check(lib().dllm_selftest_wait_timeout(_ptr(ws), limit_us, _stream(stream)),
           "dllm_selftest_wait_timeout")


def dllm_merge_shard_stats(shards, rows: int, out: StatsBuffers, stream=None) -> None:
    """shards: list of (statistics of one vocabulary shard, its first vocabulary id); each
    statistics object has row_max, lse, conf (float32) and argmax (int32) device tensors."""
    arr = (dllm_shard_stats * len(shards))(*[
        dllm_shard_stats(dllm_stats(_ptr(st.row_max), _ptr(st.lse), _ptr(st.conf),
                                    _ptr(st.argmax)), int(off))
        for st, off in shards])
    _check(lib().dllm_merge_shard_stats(arr, len(shards), int(rows), ctypes.byref(out.c()),
                                        _stream(stream)), "dllm_merge_shard_stats")


def dllm_get_status(ws, stream=None) -> int:
    out = _c_i32(0)
    _check(lib().dllm_get_status(_ptr(ws), _stream(stream), ctypes.byref(out)), "dllm_get_status")
    return int(out.value)

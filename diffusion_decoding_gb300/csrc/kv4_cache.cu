// The 4-bit key/value cache: quantising entries as they are written, and reading them back (dInfer
// explainer, KV-cache manager: refreshed entries replace the stale ones in the cache).  The format
// is described in kv4.cuh and include/dllm.h.
//
// Both kernels are HBM-bound (bf16: 2 bytes of values and 9/16 bytes of cache per value), with
// little to spare: the write has about a dozen instructions a value.  A lane handles 16 channels
// (32 bytes of bf16 in one access, 8 bytes of codes), so the two lanes of a group find its extremes
// with one shuffle and work out its step together with 16 values each.  A warp takes up to kItems
// such pieces of one token and issues all their loads before it uses the first, the values' before
// it even knows their place in the cache.
//
// Measured, 32768 entries of 8 heads of 128 channels, keys and values in bf16 (153 MB each way): write
// 33.6 us, 80 % of the issue slots busy; read 29.3 us, 66 %; one after the other 59 us, 5.2 TB/s, 0.77
// of the card's copy rate.  One piece a lane: 74 us; four: 69.5 (registers).
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 2;

struct Kv4Params {
  char* x[2];  // keys, values; strides in bytes
  int64_t xb[2], xt[2], xh[2];
  uint8_t* codes[2];
  uint16_t* params[2];
  const int32_t* table;
  int table_stride, pages, heads, page_size, D;
  const int32_t* pos;
  int64_t pos_stride;
  int n;
  unsigned tokens;
  uint32_t head_magic;
  int lanes_log2;  // lanes of a token: 32, or fewer where its pieces are few
};

// One warp's work: a token, keys or values, and pieces [first, first + 32 * ITEMS) of its heads.
// The grid is (warps over the tokens, segments of 32 * ITEMS pieces, keys and values).
struct Unit {
  int b, i, first;
  int entry;  // cache entry, -1: none
  int page, slot;
  int lane;  // of the token's
  bool valid;
};

template <int ITEMS>
__device__ __forceinline__ Unit unit_of(const Kv4Params& p) {
  const int lanes_log2 = ITEMS == 1 ? p.lanes_log2 : 5;  // with more, a token has a warp at least
  const unsigned token = (blockIdx.x * static_cast<unsigned>(kThreads) + threadIdx.x) >> lanes_log2;
  Unit u;
  u.first = static_cast<int>(blockIdx.y) * 32 * ITEMS;
  u.valid = token < p.tokens;
  u.lane = static_cast<int>(threadIdx.x) & ((1 << lanes_log2) - 1);
  u.b = static_cast<int>(token / static_cast<unsigned>(p.n));
  u.i = static_cast<int>(token) - u.b * p.n;
  u.entry = u.page = -1;
  u.slot = 0;
  if (u.valid) u.entry = p.pos ? p.pos[u.b * p.pos_stride + u.i] : u.i;
  return u;
}

// Page and slot of the unit's entry.
__device__ __forceinline__ void find_page(const Kv4Params& p, Unit& u) {
  if (u.entry >= 0) {
    const int t = static_cast<int>(static_cast<unsigned>(u.entry) / static_cast<unsigned>(p.page_size));
    u.slot = u.entry - t * p.page_size;
    if (t < p.table_stride) {
      const int pg = __ldg(p.table + static_cast<int64_t>(u.b) * p.table_stride + t);
      if (pg >= 0 && pg < p.pages) u.page = pg;
    }
  }
}

// Head of piece c (head_dim / 16 pieces a head): a product with floor(2^32 / (D / 16)) + 1, exact
// while c * D / 16 < 2^32.
__device__ __forceinline__ int head_of(const Kv4Params& p, int c) {
  return static_cast<int>(__umulhi(static_cast<uint32_t>(c), p.head_magic));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_min_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Step from the extremes (lo <= 0 <= hi): (hi - lo) / 15 rounded up to three significant bits; 0
// when it is tiny, NaN when the group is not finite.  15 * s has seven significant bits, so the
// comparison that settles the rounding is exact.
__device__ __forceinline__ float kv4_step(float lo, float hi) {
  const float d = hi - lo;
  const float t = d * (1.f / 15.f) * 0.99999904632568359375f;  // 1 - 2^-20: never above d / 15
  float s = __uint_as_float((__float_as_uint(t) + 0x1FFFFFu) & ~0x1FFFFFu);
  if (15.f * s < d) s = __uint_as_float(__float_as_uint(s) + 0x200000u);
  if (!(d >= 15.f * 7.7037197775489434e-34f)) s = 0.f;  // 2^-110
  if (!(s <= 5.316911983139663e36f)) s = __uint_as_float(kKv4NaNParam << 16);  // 2^122
  return d != d ? __uint_as_float(kKv4NaNParam << 16) : s;
}

__device__ __forceinline__ void load32(const char* p, uint32_t* w) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                 "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(char* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// kAligned: rows on 32-byte boundaries; otherwise values are read one by one.
template <int DT, bool kAligned, int ITEMS>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ Kv4Params p) {
  constexpr int NW = DT == DLLM_BF16 ? 8 : 16;  // words of a piece
  pdl_wait();
  pdl_trigger();
  Unit u = unit_of<ITEMS>(p);
  if (ITEMS > 1 && !u.valid) return;
  const int side = blockIdx.z;
  const int cpr = p.D / 16, pieces = p.heads * cpr;
  const char* x = p.x[side] + u.b * p.xb[side] + u.i * p.xt[side];
  const int64_t xh = p.xh[side];

  // the values are on their way while the entry and its page are looked up
  uint32_t raw[ITEMS][NW];
#pragma unroll
  for (int t = 0; t < ITEMS; ++t) {
    const int c = u.first + t * 32 + u.lane;
#pragma unroll
    for (int e = 0; e < NW; ++e) raw[t][e] = 0u;
    if (c >= pieces || (ITEMS == 1 && !u.valid)) continue;
    const int h = head_of(p, c);
    const char* src = x + h * xh + (c - h * cpr) * (NW * 4);
    if constexpr (kAligned) {
#pragma unroll
      for (int e = 0; e < NW; e += 8) load32(src + 4 * e, raw[t] + e);
    } else if constexpr (DT == DLLM_BF16) {
#pragma unroll
      for (int e = 0; e < NW; ++e)
        raw[t][e] = reinterpret_cast<const uint16_t*>(src)[2 * e] |
                    static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[2 * e + 1]) << 16;
    } else {
#pragma unroll
      for (int e = 0; e < NW; ++e) raw[t][e] = reinterpret_cast<const uint32_t*>(src)[e];
    }
  }
  find_page(p, u);
  if (ITEMS > 1 ? u.page < 0 : !__any_sync(kFull, u.page >= 0)) return;
  const int64_t row0 = static_cast<int64_t>(u.page) * p.heads * p.page_size + u.slot;
  uint8_t* codes = p.codes[side] + row0 * (p.D / 2);
  uint16_t* params = p.params[side] + row0 * (p.D / kKv4Group);
#pragma unroll
  for (int t = 0; t < ITEMS; ++t) {
    const int c = u.first + t * 32 + u.lane;
    float hi, lo;
    if constexpr (DT == DLLM_BF16) {
      // extremes in packed bf16; the maximum and the negated minimum share a word
      uint32_t mx = raw[t][0], mn = raw[t][0];
#pragma unroll
      for (int e = 1; e < NW; ++e) {
        mx = bf2_max_nan(mx, raw[t][e]);
        mn = bf2_min_nan(mn, raw[t][e]);
      }
      mn ^= 0x80008000u;
      uint32_t both = bf2_max_nan(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
      both = bf2_max_nan(both, __shfl_xor_sync(kFull, both, 1));
      both = bf2_max_nan(both, 0u);
      hi = bf16lo(both);
      lo = -bf16hi(both);
    } else {
      hi = 0.f, lo = 0.f;
#pragma unroll
      for (int e = 0; e < NW; ++e) {
        hi = max_nan(hi, __uint_as_float(raw[t][e]));
        lo = max_nan(lo, -__uint_as_float(raw[t][e]));
      }
      hi = max_nan(hi, __shfl_xor_sync(kFull, hi, 1));
      lo = -max_nan(lo, __shfl_xor_sync(kFull, lo, 1));
    }
    float s;
    uint32_t z, w[2] = {0u, 0u};
    if constexpr (DT == DLLM_BF16) {
      s = kv4_step(lo, hi);
      // x / s has at most eight and three significant bits: apart from exact ties it is no nearer
      // than 2^-9 to a tie, so a product with 1 / s enlarged by 2^-16 rounds ties away from zero
      // and everything else to the nearest.  Adding 1.5 * 2^23 rounds to an integer in the low
      // bits.
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      inv = s > 0.f ? inv * 1.0000152587890625f : 0.f;
      const float zf = fmaf(-lo, inv, 12582912.f);  // z in the low bits
      z = __float_as_uint(zf) & 15u;
#pragma unroll
      for (int e = 15; e >= 0; --e) {
        const float v = e & 1 ? bf16hi(raw[t][e >> 1]) : bf16lo(raw[t][e >> 1]);
        w[e >> 3] = w[e >> 3] * 16u + min(__float_as_uint(fmaf(v, inv, zf)), 0x4B40000Fu);
      }
      // what the eight words' upper bits have added up to
#pragma unroll
      for (int e = 0; e < 2; ++e) w[e] -= 0x4B400000u * 0x11111111u;
    } else {
      const float d = hi - lo;
      s = __fdiv_rn(d, 15.f);
      const bool finite = d < INFINITY;
      s = s < 7.7037197775489434e-34f ? 0.f
                                      : __uint_as_float((__float_as_uint(s) + 0x1FFFFFu) & ~0x1FFFFFu);
      if (!finite || s > 5.316911983139663e36f) s = __uint_as_float(kKv4NaNParam << 16);
      const float den = s > 0.f ? s : 1.f;
      z = static_cast<uint32_t>(fminf(floorf(__fadd_rn(__fdiv_rn(-lo, den), 0.5f)), 15.f));
#pragma unroll
      for (int e = 15; e >= 0; --e) {
        const float r = __fdiv_rn(__uint_as_float(raw[t][e]), den);
        const float k = s > 0.f ? copysignf(floorf(__fadd_rn(fabsf(r), 0.5f)), r) : 0.f;
        const float nf = fminf(fmaxf(k + static_cast<float>(z), 0.f), 15.f);
        w[e >> 3] = w[e >> 3] * 16u + static_cast<uint32_t>(nf);
      }
    }
    if (c >= pieces || (ITEMS == 1 && u.page < 0)) continue;
    if (s != s) z = 0u;
    const int h = head_of(p, c), cc = c - h * cpr;
    const int64_t row = static_cast<int64_t>(h) * p.page_size;
    *reinterpret_cast<uint2*>(codes + row * (p.D / 2) + cc * 8) = make_uint2(w[0], w[1]);
    if ((cc & 1) == 0)
      params[row * (p.D / kKv4Group) + (cc >> 1)] =
          static_cast<uint16_t>((__float_as_uint(s) >> 16) | z);
  }
}

template <int DT, bool kAligned, int ITEMS>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4Params p) {
  pdl_wait();
  pdl_trigger();
  Unit u = unit_of<ITEMS>(p);
  if (!u.valid) return;
  find_page(p, u);
  const int side = blockIdx.z;
  const int cpr = p.D / 16, pieces = p.heads * cpr;
  char* x = p.x[side] + u.b * p.xb[side] + u.i * p.xt[side];
  const int64_t xh = p.xh[side];
  const int64_t row0 = static_cast<int64_t>(max(u.page, 0)) * p.heads * p.page_size + u.slot;
  const uint8_t* codes = p.codes[side] + row0 * (p.D / 2);
  const uint16_t* params = p.params[side] + row0 * (p.D / kKv4Group);
  uint2 w[ITEMS];
  uint32_t pp[ITEMS];
#pragma unroll
  for (int t = 0; t < ITEMS; ++t) {
    const int c = u.first + t * 32 + u.lane;
    w[t] = make_uint2(0u, 0u);
    pp[t] = 0u;
    if (u.page < 0 || c >= pieces) continue;
    const int h = head_of(p, c), cc = c - h * cpr;
    const int64_t row = static_cast<int64_t>(h) * p.page_size;
    w[t] = __ldg(reinterpret_cast<const uint2*>(codes + row * (p.D / 2) + cc * 8));
    pp[t] = __ldg(params + row * (p.D / kKv4Group) + (cc >> 1));
  }
#pragma unroll
  for (int t = 0; t < ITEMS; ++t) {
    const int c = u.first + t * 32 + u.lane;
    if (c >= pieces) continue;
    const int h = head_of(p, c), cc = c - h * cpr;
    const Kv4Scale sc = kv4_scale(__byte_perm(pp[t], pp[t], 0x1010));
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // pairs of channels (j, j + 4), put back side by side
      const uint32_t word = k ? w[t].y : w[t].x;
      const uint32_t a = kv4_pair<0>(word, sc), b = kv4_pair<1>(word, sc),
                     d = kv4_pair<2>(word, sc), e = kv4_pair<3>(word, sc);
      v[4 * k] = __byte_perm(a, b, 0x5410);
      v[4 * k + 1] = __byte_perm(d, e, 0x5410);
      v[4 * k + 2] = __byte_perm(a, b, 0x7632);
      v[4 * k + 3] = __byte_perm(d, e, 0x7632);
    }
    char* dst = x + h * xh + cc * (DT == DLLM_BF16 ? 32 : 64);
    if constexpr (DT == DLLM_BF16) {
      if constexpr (kAligned) {
        store32(dst, v);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          reinterpret_cast<uint16_t*>(dst)[k] = static_cast<uint16_t>(v[k >> 1] >> (16 * (k & 1)));
      }
    } else {
      uint32_t f[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[2 * k] = v[k] << 16;
        f[2 * k + 1] = v[k] & 0xffff0000u;
      }
      if constexpr (kAligned) {
        store32(dst, f);
        store32(dst + 32, f + 8);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) reinterpret_cast<uint32_t*>(dst)[k] = f[k];
      }
    }
  }
}

bool aligned32(const dllm_heads& h) {
  const int es = h.dtype == DLLM_BF16 ? 2 : 4;
  return (reinterpret_cast<uintptr_t>(h.data) | static_cast<uintptr_t>(h.batch_stride * es) |
          static_cast<uintptr_t>(h.token_stride * es) | static_cast<uintptr_t>(h.head_stride * es)) %
             32 == 0;
}

template <bool kWrite, int DT, bool kAligned>
cudaError_t launch_items(Kv4Params& p, int sm_count, cudaStream_t stream) {
  const int pieces = p.heads * (p.D / 16);
  // Tokens of up to 16 pieces share a warp (32768 entries of one head: 11.8 us written and read, 39.3
  // with a token a warp; of two 20.7, 39.7).
  p.lanes_log2 = 5;
  while (p.lanes_log2 > 1 && pieces <= 1 << (p.lanes_log2 - 1)) --p.lanes_log2;
  const unsigned per_block = kThreads >> p.lanes_log2;
  auto run = [&](auto kern, int items) {
    const dim3 grid((p.tokens + per_block - 1) / per_block,
                    static_cast<unsigned>((pieces + 32 * items - 1) / (32 * items)), 2);
    return launch_dependent(kern, grid, dim3(kThreads), 0, stream, p);
  };
  // Two pieces a lane hide more of the load latency and share the page lookup; one piece a lane
  // when the call has too few warps to fill the SMs (1152 entries of 4 heads: 4.7 us, 5.1 with two).
  const bool few = pieces <= 32 || static_cast<int64_t>(p.tokens) * 2 * ((pieces + 63) / 64) <
                   static_cast<int64_t>(sm_count) * 16;
  if constexpr (kWrite)
    return few ? run(kv4_write_kernel<DT, kAligned, 1>, 1)
               : run(kv4_write_kernel<DT, kAligned, kItems>, kItems);
  else
    return few ? run(kv4_read_kernel<DT, kAligned, 1>, 1)
               : run(kv4_read_kernel<DT, kAligned, kItems>, kItems);
}

template <bool kWrite>
cudaError_t launch(const dllm_kv4_cache& cache, const dllm_heads& k, const dllm_heads& v, int B,
                   int n, const int32_t* pos, int64_t pos_stride, int sm_count,
                   cudaStream_t stream) {
  Kv4Params p{};
  const dllm_heads* x[2] = {&k, &v};
  const int es = k.dtype == DLLM_BF16 ? 2 : 4;
  for (int j = 0; j < 2; ++j) {
    p.x[j] = static_cast<char*>(x[j]->data);
    p.xb[j] = x[j]->batch_stride * es;
    p.xt[j] = x[j]->token_stride * es;
    p.xh[j] = x[j]->head_stride * es;
  }
  p.codes[0] = cache.k_codes, p.codes[1] = cache.v_codes;
  p.params[0] = cache.k_params, p.params[1] = cache.v_params;
  p.table = cache.page_table;
  p.table_stride = cache.table_stride;
  p.pages = cache.pages;
  p.heads = cache.heads;
  p.page_size = cache.page_size;
  p.D = cache.head_dim;
  p.pos = pos;
  p.pos_stride = pos_stride;
  p.n = n;
  p.tokens = static_cast<unsigned>(B) * static_cast<unsigned>(n);
  p.head_magic = static_cast<uint32_t>((uint64_t{1} << 32) / (cache.head_dim / 16) + 1);
  const bool al = aligned32(k) && aligned32(v);
  if (k.dtype == DLLM_BF16)
    return al ? launch_items<kWrite, DLLM_BF16, true>(p, sm_count, stream)
              : launch_items<kWrite, DLLM_BF16, false>(p, sm_count, stream);
  return al ? launch_items<kWrite, DLLM_F32, true>(p, sm_count, stream)
            : launch_items<kWrite, DLLM_F32, false>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_kv4_write(const dllm_kv4_cache& cache, const dllm_heads& k, const dllm_heads& v,
                             int B, int n, const int32_t* pos, int64_t pos_stride, int sm_count,
                             cudaStream_t stream) {
  return launch<true>(cache, k, v, B, n, pos, pos_stride, sm_count, stream);
}

cudaError_t launch_kv4_read(const dllm_kv4_cache& cache, const dllm_heads& k, const dllm_heads& v,
                            int B, int n, const int32_t* pos, int64_t pos_stride, int sm_count,
                            cudaStream_t stream) {
  return launch<false>(cache, k, v, B, n, pos, pos_stride, sm_count, stream);
}

}  // namespace dllm

// How much attention each cache entry receives (attention_weights.cu), for many query rows per cache
// head, on the 5th-generation tensor cores.
//
// S^T [128 entries x 64 rows] = K Q^T with the entries as the rows of the product: an entry's scores
// then lie in one lane of tensor memory, and its sum over the queries needs no other thread.  A CTA
// takes 256 entries (two tiles) of one head and walks through the queries in chunks of 64.
//
// The log-sum-exps go through the product too: K has a block of 16 more channels that are 1 (four of them
// used), the queries' rows there hold -lse / scale as four bf16 terms (32 bits of it), so that a weight is
// exp2(scale log2(e) * s) and the threads that add the weights up need nothing but the scores.
//
// Warps 0-15: two threads an entry, each half of the rows of a chunk.  They turn the entry's codes to bf16
// (half of the channels each) and store them in tensor memory (left operands may lie there), then add up
// the weights of every chunk; the next entries' K is stored, into a second place where head_dim <= 128
// leaves room, before the last chunk's scores are read, so that the products do not stop between entries.
// Warp 16 issues the products, warp 17 has the chunks copied in (bulk copies of tiles that
// weights_queries_kernel has laid out: 64 rows in the 128-byte swizzled layout, channels in the order in
// which codes come out).  Sums of an entry over heads and halves are partial results that
// weights_join_kernel adds in order.
//
// What it loses: products and exponentials hardly overlap.  256 entries x 64 rows of 128 channels take 1080
// cycles, the products 52 % of them and the exponentials (32 a cycle and SM) 47 %; neither pipe is full.  2
// sequences of up to 16384 entries, 8 heads, 4096 rows, causal: 271 us, 0.93 PFLOP/s; 16 of 4160, 2 heads,
// 512 rows: 31 us.  Eight sum warps, one thread an entry, took 420 for the first; log-sum-exps added by the
// threads 371; exponentials computed by polynomials in part, or scores loaded ahead, no less.
//
// TMEM, 512 columns: K 2 tiles x 1 or 2 x D/2, scores 2 tiles x 2 buffers x 64.
#include <math.h>

#include <algorithm>

#include "attention.h"
#include "attention_weights.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "mbarrier.cuh"
#include "vec_math.cuh"

namespace dllm {
namespace {

constexpr int kTile = 128;                // entries of a tile
constexpr int kPair = 2 * kTile;          // entries of a CTA at a time
constexpr int kChunk = 64;                // query rows of a product
constexpr int kSumWarps = 16;
constexpr int kThreads = 32 * (kSumWarps + 2);
constexpr int kTmemCols = 512;

struct WeightsPlan {
  Divisor by_pairs, by_heads, by_page;
  int rows, chunks, pairs;  // query rows of a head, chunks of them, pairs of entry tiles (of max_len)
  uint32_t items;           // pairs * heads * B, below 2^31
  uint8_t* queries;         // [B][heads][chunks] records
  float* sums;              // [B][heads * 2][pairs * kPair]
  int32_t* status;
};

// A record: D / 64 slabs of 64 rows x 128 bytes, and the block of -lse / scale (64 rows x 16 channels).
constexpr uint32_t kTermBytes = kChunk * 32, kOnesBytes = kTile * 32;
__host__ __device__ constexpr uint32_t record_bytes(int D) { return D * 128 + kTermBytes; }
__host__ __device__ constexpr int stages(int D) { return D <= 64 ? 8 : D <= 128 ? 6 : 4; }

// ---- tcgen05, one CTA

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// (whole warps issue with uniform operands, one elected lane executes: see attention_tc.cu)
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(kFull, x); }
__device__ __forceinline__ int uniform(int x) { return static_cast<int>(uniform(static_cast<uint32_t>(x))); }
// D [128 x 64] (+)= A [128 x 16] B [16 x 64], A in TMEM, B in shared memory
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// the same with A in shared memory
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor, 128-byte swizzle, K-major (attention_tc.cu).
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint64_t desc_of(uint32_t saddr) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(((saddr & 0x3FFFFu) >> 4) | (1u << 16)), "r"(kDescHigh));
  return d;
}
// The same without a swizzle, 16 channels: 8 rows x 16 bytes contiguous, the other 8 channels 128 bytes on,
// the next 8 rows 256 bytes on.
__device__ __forceinline__ uint64_t desc_block(uint32_t saddr) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};"
      : "=l"(d)
      : "r"(((saddr & 0x3FFFFu) >> 4) | ((128u >> 4) << 16)), "r"((256u >> 4) | 1u << 14));
  return d;
}
__host__ __device__ constexpr uint32_t block_at(int row, int channel) {
  return (row >> 3) * 256 + (channel >> 3) * 128 + (row & 7) * 16 + (channel & 7) * 2;
}
// D fp32, A and B bf16, M = 128, N = 64, both K-major
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kChunk >> 3) << 17) |
                            (static_cast<uint32_t>(kTile >> 4) << 24);

// A whole warp's wait (attention_tc.cu).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  return __all_sync(kFull, wait_bar(bar, parity, abort_flag, status)) != 0;
}

__device__ __forceinline__ int length_of(const AttnParams& p, int b) {
  return p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
}

// ---- the queries, once per call

// A thread: eight channels of a row, or a row's -lse and token.
__global__ void __launch_bounds__(256)
    weights_queries_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWeights x,
                           const __grid_constant__ WeightsPlan f, int D) {
  pdl_wait();
  pdl_trigger();
  const int64_t rec = blockIdx.x;  // (b, head, chunk)
  const int chunk = static_cast<int>(rec % f.chunks);
  const int64_t bh = rec / f.chunks;
  const int h = static_cast<int>(bh % p.heads), b = static_cast<int>(bh / p.heads);
  uint8_t* out = f.queries + rec * record_bytes(D);
  const int words = D / 8;
  for (int k = threadIdx.x; k < kChunk * words; k += blockDim.x) {
    const int row = k / words, w = k - row * words, r = chunk * kChunk + row, i = r / p.G;
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (r < f.rows) {
      const uint16_t* s8 =
          p.q + b * p.qb + i * p.qt + (static_cast<int64_t>(h) * p.G + r - i * p.G) * p.qh + 8 * w;
      if (x.q_aligned) {
        const uint4 y = *reinterpret_cast<const uint4*>(s8);
        v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) v[m] = s8[2 * m] | static_cast<uint32_t>(s8[2 * m + 1]) << 16;
      }
    }
    // channels of a code word come out in pairs (m, m + 4)
    *reinterpret_cast<uint4*>(out + (w >> 3) * (kChunk * 128) + row * 128 + (((w & 7) ^ (row & 7)) << 4)) =
        make_uint4(__byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632),
                   __byte_perm(v[1], v[3], 0x5410), __byte_perm(v[1], v[3], 0x7632));
  }
  for (int row = threadIdx.x; row < kChunk; row += blockDim.x) {
    const int r = chunk * kChunk + row, i = r / p.G;
    float l = -INFINITY;  // adds nothing
    if (r < f.rows) l = x.lse[(static_cast<int64_t>(b) * p.heads * p.G + h * p.G + r - i * p.G) * p.n + i];
    uint32_t w[8] = {};
    if (!(fabsf(l) < INFINITY)) {
      // infinite: the score becomes so small that the weight is 0
      w[0] = l != l ? 0x7FFFu : x.scale > 0.f ? 0xFF80u : 0x7F80u;
    } else {
      double rest = -static_cast<double>(l) / static_cast<double>(x.scale);
      const float whole = static_cast<float>(rest);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t term = __float_as_uint(static_cast<float>(rest)) & 0xFFFF0000u;  // (cut: the rest follows)
        rest -= static_cast<double>(__uint_as_float(term));
        w[k >> 1] |= term >> (k & 1 ? 0 : 16);
      }
      // (beyond the largest float the next terms would cancel it to NaN)
      if (fabsf(whole) == INFINITY) w[0] = __float_as_uint(whole) >> 16, w[1] = 0u;
    }
    *reinterpret_cast<uint4*>(out + D * 128 + block_at(row, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(out + D * 128 + block_at(row, 8)) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ---- what a CTA does at a time

struct Item {
  int b, h, j0, len, tiles;  // first entry; tiles with entries (0: none)
  int c0, c1;                // chunks (none where no query sees an entry)
  // (all roles count the same chunks)
  __device__ __forceinline__ Item(const AttnParams& p, const WeightsPlan& f, uint32_t at) {
    const uint32_t rest = f.by_pairs(at);
    j0 = static_cast<int>(at - rest * f.pairs) * kPair;
    b = static_cast<int>(f.by_heads(rest));
    h = static_cast<int>(rest) - b * p.heads;
    len = length_of(p, b);
    tiles = j0 >= len ? 0 : j0 + kTile >= len ? 1 : 2;
    c0 = 0;
    c1 = tiles > 0 ? f.chunks : 0;
    // row r sees the entries below len - n + r / G + 1: chunks whose last row sees none of these are passed over
    if (p.causal && tiles > 0) c0 = min(first_row(p, f, j0) / kChunk, c1);
  }
  // The first row that sees entry j (one beyond all rows: none does).
  __device__ __forceinline__ int first_row(const AttnParams& p, const WeightsPlan& f, int j) const {
    const int64_t token = static_cast<int64_t>(j) - (len - p.n);
    return token <= 0 ? 0 : static_cast<int>(min(token * p.G, static_cast<int64_t>(f.chunks) * kChunk));
  }
};

// Where the K of use n of a tile lies, from the tile's first column.
template <int D>
__device__ __forceinline__ constexpr uint32_t k_place(int tile, uint32_t n) {
  return D <= 128 ? tile * D + (n & 1) * (D / 2) : tile * (D / 2);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attention_weights_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ WeightsPlan f) {
  constexpr int S = stages(D);
  constexpr bool kTwoK = D <= 128;                      // two places for K
  constexpr uint32_t kScores = kTwoK ? 2 * D : D;       // first column of the scores
  static_assert(kScores + 4 * kChunk <= kTmemCols, "");
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * S + 4 + 8 + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t ones = sbase + S * record_bytes(D);  // K's block of 16 channels
  const uint32_t q_full = smem_u32(&bars[0]), q_empty = q_full + 8 * S;
  const uint32_t k_full = q_empty + 8 * S;  // of a tile and place (tile + 2 * place): K is there
  const uint32_t s_full = k_full + 32;      // of a buffer (tile + 2 * parity): scores are there, have been read
  const uint32_t s_empty = s_full + 32, done = s_empty + 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(q_full + 8 * s, 1);
      mbar_init(q_empty + 8 * s, 1);
    }
    for (int a = 0; a < 4; ++a) {
      mbar_init(k_full + 8 * a, kSumWarps / 2);
      mbar_init(s_full + 8 * a, 1);
      mbar_init(s_empty + 8 * a, kSumWarps / 2);
    }
    mbar_init(done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  for (int k = threadIdx.x; k < kTile * 2; k += kThreads) {
    const uint32_t one2 = k & 1 ? 0u : 0x3F803F80u;  // channels 0 to 3 are 1
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(ones + block_at(k >> 1, 8 * (k & 1))), "r"(one2),
                 "r"(one2), "r"(0u), "r"(0u)
                 : "memory");
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // Only the copies read what weights_queries_kernel writes.  That kernel's CTAs have all waited for the
  // kernels before it when this one may start: the cache, lengths and sums of those are complete, and
  // none of them holds tensor memory.
  pdl_trigger();
  if (warp == kSumWarps) tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort_v = &abort_flag;

  if (warp < kSumWarps) {
    // ---------------------------------------------------------------- two threads an entry
    const int tile = warp >> 2 & 1, half = warp >> 3;
    const int in_pair = tile * kTile + 32 * (warp & 3) + lane;  // entry
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    constexpr int kWords = D / 16, kParams = D / 64;  // of half an entry
    uint32_t mine = 0, k_use = 0;  // of chunks with this tile: buffer and phase; uses of its K
    bool ok = true;
    uint32_t code[kWords], par[kParams];
    auto sums_of = [&](const Item& it) {
      return f.sums + ((static_cast<int64_t>(it.b) * p.heads + it.h) * 2 + half) * f.pairs * kPair + it.j0 + in_pair;
    };
    // The next item from `at` on whose entries some query sees; the sums of others are 0.
    auto advance = [&](uint32_t& at) {
      for (;; at += gridDim.x) {
        const Item it(p, f, min(at, f.items - 1));
        if (at >= f.items || it.c1 > it.c0) return it;
        if (it.j0 + in_pair < it.len) *sums_of(it) = 0.f;
      }
    };
    // The codes of this thread's half; whether the entry counts.
    auto load = [&](uint32_t at, const Item& it) {
      bool there = false;
      const int j = it.j0 + in_pair;
      if (at < f.items && j < it.len) {
        const int t = static_cast<int>(f.by_page(static_cast<uint32_t>(j)));
        const int page = __ldg(p.table + static_cast<int64_t>(it.b) * p.table_stride + t);
        there = static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
        if (there && p.key_mask) there = __ldg(p.key_mask + it.b * p.mask_stride + j) != 0;
        if (there) {
          const int64_t row = (static_cast<int64_t>(page) * p.heads + it.h) * p.page_size + j - t * p.page_size;
          const uint4* src = reinterpret_cast<const uint4*>(p.k_codes + row * (D / 2) + half * (D / 4));
#pragma unroll
          for (int w = 0; w < kWords / 4; ++w) {
            const uint4 v = __ldg(src + w);
            code[4 * w] = v.x, code[4 * w + 1] = v.y, code[4 * w + 2] = v.z, code[4 * w + 3] = v.w;
          }
#pragma unroll
          for (int w = 0; w < kWords / 4; ++w) par[w] = __ldg(p.k_params + row * (D / 32) + half * (D / 64) + w);
        }
      }
      if (!there) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) code[w] = 0u;
#pragma unroll
        for (int w = 0; w < kParams; ++w) par[w] = 0u;
      }
      return there;
    };
    // Store K of the codes held, where its place is free.
    auto store = [&]() {
      const uint32_t t_k = tmem + lanes + k_place<D>(tile, k_use) + half * (D / 4);
#pragma unroll
      for (int c = 0; c < kWords / 4; ++c) {
        uint32_t v[16];
        const Kv4Scale sc = kv4_scale(__byte_perm(par[c], par[c], 0x1010));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          v[4 * w] = kv4_pair<0>(code[4 * c + w], sc);
          v[4 * w + 1] = kv4_pair<1>(code[4 * c + w], sc);
          v[4 * w + 2] = kv4_pair<2>(code[4 * c + w], sc);
          v[4 * w + 3] = kv4_pair<3>(code[4 * c + w], sc);
        }
        tmem_st16(t_k + 16 * c, v);
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + 8 * (tile + (kTwoK ? 2 * (k_use & 1) : 0)));
      ++k_use;
    };
    uint32_t at = blockIdx.x;
    Item it = advance(at);
    bool shown = load(at, it);
    if (at < f.items && tile < it.tiles) store();
    while (at < f.items && ok) {
      const bool here = tile < it.tiles;
      const int j = it.j0 + in_pair;
      uint32_t at_next = at + gridDim.x;
      const Item next = advance(at_next);
      const bool next_shown = load(at_next, next), next_here = at_next < f.items && tile < next.tiles;
      // the first chunk all of whose rows see all of the tile's entries; the first row that sees this one
      const int c_all = p.causal ? (it.first_row(p, f, min(it.len, it.j0 + (tile + 1) * kTile) - 1) + kChunk - 1) / kChunk
                                 : 0;
      const int own_row = p.causal ? it.first_row(p, f, j) - 32 * half : 0;
      float sum = 0.f;
      for (int c = it.c0; c < it.c1; ++c) {
        // (the products that read the other place's K are complete: their scores have been read)
        if (kTwoK && c == it.c1 - 1 && next_here) store();
        if (!here) continue;
        const int a = tile + 2 * (mine & 1);
        ok = wait_warp(s_full + 8 * a, mine >> 1 & 1, abort_v, f.status);
        if (!ok) break;
        tc_after();
        float s[32];
        tmem_ld32(tmem + lanes + kScores + a * kChunk + half * 32, s);
        tmem_wait_ld();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty + 8 * a);
        ++mine;
        if (c >= c_all) {
          const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
          uint64_t l2[4] = {pack2(0.f, 0.f), pack2(0.f, 0.f), pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a0, a1;
            unpack2(mul2(pack2(s[e], s[e + 1]), scale2), a0, a1);
            l2[e >> 1 & 3] = add2(l2[e >> 1 & 3], pack2(ex2(a0), ex2(a1)));
          }
          float a0, a1;
          unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), a0, a1);
          sum += a0 + a1;
        } else {
          float part = 0.f;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float w = ex2(s[e] * p.scale_log2);
            part += c * kChunk + e >= own_row ? w : 0.f;
          }
          sum += part;
        }
      }
      if (!ok) break;
      if (j < it.len && here) *sums_of(it) = shown ? sum : 0.f;
      if (!kTwoK && next_here) store();
      at = at_next;
      it = next;
      shown = next_shown;
    }
  } else if (warp == kSumWarps) {
    // ---------------------------------------------------------------- products
    const uint32_t lead = elect_lane(), ones_u = uniform(ones);
    int stage = 0;
    uint32_t phase = 0, mine[2] = {0u, 0u}, k_use[2] = {0u, 0u};
    bool ok = true;
    for (uint32_t at = blockIdx.x; at < f.items && ok; at += gridDim.x) {
      const Item it(p, f, at);
      if (it.c1 <= it.c0) continue;
      for (int t = 0; t < it.tiles && ok; ++t)
        ok = wait_warp(k_full + 8 * (t + (kTwoK ? 2 * (k_use[t] & 1) : 0)), (kTwoK ? k_use[t] >> 1 : k_use[t]) & 1,
                       abort_v, f.status);
      if (!ok) break;
      tc_after();
      for (int c = it.c0; c < it.c1; ++c) {
        const int st = uniform(stage);
        ok = wait_warp(q_full + 8 * st, phase, abort_v, f.status);
        if (!ok) break;
        const uint32_t q = uniform(sbase + st * record_bytes(D));
        for (int t = 0; t < it.tiles; ++t) {
          const uint32_t a = uniform(t + 2 * (mine[t] & 1));
          ok = wait_warp(s_empty + 8 * a, (mine[t] >> 1 & 1) ^ 1, abort_v, f.status);
          if (!ok) break;
          tc_after();
          const uint32_t d = uniform(tmem + kScores + a * kChunk), k = uniform(tmem + k_place<D>(t, k_use[t]));
          mma_ss(lead, d, desc_block(ones_u), desc_block(q + D * 128), kIdesc, 0u);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ts(lead, d, k + 8 * ks, desc_of(q + (ks >> 2) * (kChunk * 128) + (ks & 3) * 32), kIdesc, 1u);
          mma_commit(lead, s_full + 8 * a);
          ++mine[t];
        }
        if (!ok) break;
        mma_commit(lead, q_empty + 8 * st);
        if (++stage == S) stage = 0, phase ^= 1;
      }
      for (int t = 0; t < it.tiles; ++t) ++k_use[t];
    }
    mma_commit(lead, done);
  } else {
    // ---------------------------------------------------------------- copies
    uint32_t chunk = 0;
    bool ok = true;
    pdl_wait();
    for (uint32_t at = blockIdx.x; at < f.items && ok; at += gridDim.x) {
      const Item it(p, f, at);
      const uint8_t* src =
          f.queries + ((static_cast<int64_t>(it.b) * p.heads + it.h) * f.chunks + it.c0) * record_bytes(D);
      for (int c = it.c0; c < it.c1; ++c, ++chunk, src += record_bytes(D)) {
        const int st = chunk % S;
        ok = wait_warp(q_empty + 8 * st, (chunk / S & 1) ^ 1, abort_v, f.status);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(q_full + 8 * st, record_bytes(D));
          bulk_g2s(sbase + st * record_bytes(D), src, record_bytes(D), q_full + 8 * st);
        }
        __syncwarp();
      }
    }
    // after an abort: copies in flight land before shared memory goes
    if (!ok && lane < S && static_cast<int>(chunk) > lane) {
      const uint32_t uses = (chunk - lane + S - 1) / S;  // of this stage
      drain_bar(q_full + 8 * lane, (uses - 1) & 1);
    }
  }
  __syncthreads();
  if (warp == kSumWarps) {
    if (lane == 0) drain_bar(done, 0);
    __syncwarp();
    tc_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Partial sums in order, and what was there before.
__global__ void __launch_bounds__(256)
    weights_join_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWeights x,
                        const __grid_constant__ WeightsPlan f) {
  pdl_wait();
  pdl_trigger();
  const int64_t stride = static_cast<int64_t>(f.pairs) * kPair;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int b = static_cast<int>(at / stride), j = static_cast<int>(at - b * stride);
  if (j >= length_of(p, b)) return;
  const int parts = p.heads * 2;
  const float* src = f.sums + static_cast<int64_t>(b) * parts * stride + j;
  float v = 0.f;
#pragma unroll 8
  for (int k = 0; k < parts; ++k) v += src[k * stride];
  put_weight(x, b, j, v);
}

WeightsPlan make_plan(int B, int n, int G, int heads, int max_len, int page_size) {
  WeightsPlan f{};
  f.rows = n * G;
  f.chunks = (f.rows + kChunk - 1) / kChunk;
  f.pairs = (max_len + kPair - 1) / kPair;
  f.items = static_cast<uint32_t>(static_cast<int64_t>(B) * heads * f.pairs);
  f.by_pairs = divisor(f.pairs), f.by_heads = divisor(heads);
  f.by_page = divisor(page_size);
  return f;
}

size_t sums_at(const WeightsPlan& f, int B, int heads, int D) {
  return align_up(kWsHeader + static_cast<size_t>(B) * heads * f.chunks * record_bytes(D), 256);
}

template <int D>
cudaError_t launch(const AttnParams& p, const AttnWeights& x, const WeightsPlan& f, int sm_count,
                   cudaStream_t stream) {
  constexpr size_t smem = stages(D) * record_bytes(D) + kOnesBytes + 1024;
  cudaError_t e = allow_smem<attention_weights_tc_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t records = static_cast<int64_t>(p.B) * p.heads * f.chunks;
  e = launch_dependent(weights_queries_kernel, dim3(static_cast<unsigned>(records)), dim3(256), 0, stream, p, x, f, D);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attention_weights_tc_kernel<D>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(f.items, sm_count))), dim3(kThreads), smem, stream,
                       p, f);
  if (e != cudaSuccess) return e;
  return launch_dependent(weights_join_kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * f.pairs)),
                          dim3(256), 0, stream, p, x, f);
}

}  // namespace

bool weights_tc_scale(float scale) { return fabsf(scale) >= 0x1p-20f && fabsf(scale) <= 0x1p20f; }

// From 9 rows of 192 and 256 channels on, 17 of 128, 33 of 64 (us here and in attention_weights.cu; heads
// x entries, sequences in brackets: 12 rows of 256 channels, 8 x 2000 (8) 16 and 26; 9 of 192 14 and 24;
// 8 of 256, 8 x 4096 (32) 79 and 66; 16 of 128, 8 x 2000 (8) 13 and 9; 17 of 128, 8 x 4000 (8) 19.3 and 18.8, 48 of
// 128 19.5 and 33; 17 of 128, 8 x 777 (1) 7.8 and 11; 20 of 64, 8 x 2000 (32) 27 and 16; 33 of 64, 6 x 777 (3)
// 8.1 and 10).  The times are of a captured graph: three launches take the host longer than one, so that the
// smallest calls made one by one are slower here (the last of these 16.5 and 12.3).
bool weights_tc_takes(int B, int n, int G, int heads, int D, int max_len) {
  const int64_t rows = static_cast<int64_t>(n) * G;
  return rows > (D == 64 ? 32 : D == 128 ? 16 : 8) &&
         static_cast<int64_t>(B) * heads * (static_cast<int64_t>(max_len) + kPair) <= (int64_t{1} << 34);
}

size_t weights_tc_ws_bytes(int B, int n, int G, int heads, int D, int max_len) {
  const WeightsPlan f = make_plan(B, n, G, heads, max_len, 1);
  return sums_at(f, B, heads, D) +
         static_cast<size_t>(B) * heads * 2 * static_cast<size_t>(f.pairs) * kPair * 4;
}

cudaError_t launch_weights_tc(const AttnParams& p, const AttnWeights& x, int D, void* ws, int sm_count,
                              cudaStream_t stream) {
  WeightsPlan f = make_plan(p.B, p.n, p.G, p.heads, p.max_len, p.page_size);
  f.status = static_cast<int32_t*>(ws);
  f.queries = static_cast<uint8_t*>(ws) + kWsHeader;
  f.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sums_at(f, p.B, p.heads, D));
  switch (D) {
    case 64: return launch<64>(p, x, f, sm_count, stream);
    case 128: return launch<128>(p, x, f, sm_count, stream);
    case 192: return launch<192>(p, x, f, sm_count, stream);
    default: return launch<256>(p, x, f, sm_count, stream);
  }
}

}  // namespace dllm

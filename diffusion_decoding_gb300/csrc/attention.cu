// Attention over the 4-bit cache for few query rows per cache head (single tokens, small blocks),
// and the kernel that joins the parts of a split (dInfer explainer, KV-cache manager: the block's
// positions attend over the cached prefix and the block).
//
// Rows are the n * G queries that share a cache head, row r = i * G + g; a row tile is 8 * NT of
// them.  A warp takes 16 cache entries at a time and computes the transposed products
//   S^T [16 entries x rows] = K Q^T,   O^T [channels x rows] += V^T P^T
// with mma.sync m16n8k16, so that the cache is the left operand in both and nothing is padded
// beyond eight rows.  K and V are turned from codes into exact bf16 values in the registers of the
// lanes that the fragments want them in, straight from global loads: no shared memory, no
// transposition (P^T comes out of S^T by movmatrix).  The order of channels inside a product is
// free, so the lane's words are contiguous; the 16 entries of a tile go to the rows of the
// fragments so that each load instruction covers one contiguous run of memory.
//
// HBM-bound: an entry of one head costs 9/8 * head_dim bytes and, at head_dim 128 and eight rows,
// ~18 warp instructions, 3/4 of what an SM issues in the time HBM brings the entry.  The next
// tile's codes are loaded while this one is computed, and page ids one tile further ahead.
#include "attention.h"

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

struct FewPlan {
  int chunk;      // entries per split, a multiple of 16 * kWarps
  int splits;
  int row_tiles;
  int q_aligned;  // query rows on 16-byte boundaries
  float* part_o;  // [(b, head, row), split, D], or null: one split, the output is written directly
  float2* part_ml;  // [(b, head, row), split]: maximum (base 2) and sum
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// N words at p with the widest loads their alignment (N * 4 bytes) allows.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = ld_stream_v4(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    static_assert(N == 1, "");
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

// How the channels of an entry are spread over the lanes.  K: lane c of the four of an entry holds
// D / 32 words, V: lane g of eight holds D / 64.  The words of a lane are contiguous, except at
// head_dim 192, where contiguous words would straddle groups: there word i of lane l is i * lanes
// + l.  A param word per group that the lane touches.
template <int D>
struct Raw {
  static constexpr int KW = D / 32, VW = D / 64;
  static constexpr bool kSpread = D == 192;
  static constexpr int KP = kSpread ? 3 : 1, VP = kSpread ? 3 : 1;
  uint32_t k[2][KW], kp[2][KP], v[4][VW], vp[4][VP];

  // entries t0, t0 + 8 of the tile for K, c + 4 * {0..3} for V
  __device__ __forceinline__ void load(const uint8_t* kc, const uint16_t* kpar, const uint8_t* vc,
                                       const uint16_t* vpar, int t0, int c, int g) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = t0 + 8 * e;
      const uint8_t* src = kc + t * (D / 2);
      const uint16_t* par = kpar + t * (D / 32);
      if constexpr (kSpread) {
#pragma unroll
        for (int i = 0; i < KW; ++i) k[e][i] = __ldg(reinterpret_cast<const uint32_t*>(src) + 4 * i + c);
#pragma unroll
        for (int i = 0; i < KP; ++i) kp[e][i] = __ldg(reinterpret_cast<const uint32_t*>(par) + i);
      } else {
        load_words<KW>(src + c * KW * 4, k[e]);
        if constexpr (D == 256)
          kp[e][0] = __ldg(reinterpret_cast<const uint32_t*>(par) + c);
        else
          kp[e][0] = __ldg(par + (D == 64 ? c / 2 : c));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = c + 4 * e;
      const uint8_t* src = vc + t * (D / 2);
      const uint16_t* par = vpar + t * (D / 32);
      if constexpr (kSpread) {
#pragma unroll
        for (int i = 0; i < VW; ++i) v[e][i] = __ldg(reinterpret_cast<const uint32_t*>(src) + 8 * i + g);
#pragma unroll
        for (int i = 0; i < VP; ++i) vp[e][i] = __ldg(par + 2 * i + g / 4);
      } else {
        load_words<VW>(src + g * VW * 4, v[e]);
        vp[e][0] = __ldg(par + g * VW / 4);
      }
    }
  }

  // both halves: the param of K word i of entry e
  __device__ __forceinline__ uint32_t k_param(int e, int i) const {
    if constexpr (kSpread)
      return i & 1 ? __byte_perm(kp[e][i / 2], 0, 0x3232) : __byte_perm(kp[e][i / 2], 0, 0x1010);
    else
      return i < 4 ? __byte_perm(kp[e][0], 0, 0x1010) : __byte_perm(kp[e][0], 0, 0x3232);
  }
  __device__ __forceinline__ uint32_t v_param(int e, int i) const { return vp[e][kSpread ? i : 0]; }
  static __device__ __forceinline__ int k_word(int i, int c) { return kSpread ? 4 * i + c : c * KW + i; }
  static __device__ __forceinline__ int v_word(int i, int g) { return kSpread ? 8 * i + g : g * VW + i; }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads)
    attention_few_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FewPlan f) {
  using R = Raw<D>;
  constexpr int KW = R::KW, VW = R::VW, MT = D / 16, ROWS = 8 * NT;
  extern __shared__ float4 smem_raw[];
  float* so = reinterpret_cast<float*>(smem_raw);  // [kWarps][ROWS][D]
  __shared__ float sm[kWarps][ROWS], sl[kWarps][ROWS];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  int id = blockIdx.x;
  const int rt = id % f.row_tiles;
  id /= f.row_tiles;
  const int split = id % f.splits;
  id /= f.splits;
  const int h = id % p.heads, b = id / p.heads;
  const int rows = p.n * p.G, r0 = rt * ROWS;
  pdl_wait();
  pdl_trigger();
  const int len = p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
  // causal: row r sees the entries below len - n + i + 1, i = r / G; the last row of the tile most
  const int i_last = min(r0 + ROWS, rows) - 1;
  const int seen_last = p.causal ? min(len, len - p.n + i_last / p.G + 1) : len;
  const int seen_first = p.causal ? min(len, len - p.n + r0 / p.G + 1) : len;
  const int begin = split * f.chunk, end = min(seen_last, begin + f.chunk);
  if (f.part_o && begin >= len && begin > 0) return;  // the join does not look at this split

  // queries: channel pairs (j, j + 4) of the lane's words, as the K fragments hold them
  uint32_t q[NT][2 * KW][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = r0 + t * 8 + g;
    const int i = r / p.G;
    const uint16_t* src = p.q + b * p.qb + i * p.qt + (static_cast<int64_t>(h) * p.G + r - i * p.G) * p.qh;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint32_t x[4] = {0u, 0u, 0u, 0u};
      if (r < rows) {
        const uint16_t* s8 = src + R::k_word(w, c) * 8;
        if (f.q_aligned) {
          const uint4 v = *reinterpret_cast<const uint4*>(s8);
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = s8[2 * k] | static_cast<uint32_t>(s8[2 * k + 1]) << 16;
        }
      }
      q[t][2 * w][0] = __byte_perm(x[0], x[2], 0x5410);
      q[t][2 * w][1] = __byte_perm(x[0], x[2], 0x7632);
      q[t][2 * w + 1][0] = __byte_perm(x[1], x[3], 0x5410);
      q[t][2 * w + 1][1] = __byte_perm(x[1], x[3], 0x7632);
    }
  }

  // entries of the tile in fragment rows g and g + 8; V fragments then want entries c + 4 * {0..3}
  const int t0 = (g >> 1) + (g & 1) * 4;
  float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int k = 0; k < MT; ++k) o[t][k][0] = o[t][k][1] = o[t][k][2] = o[t][k][3] = 0.f;
  }

  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  const uint8_t* mask = p.key_mask ? p.key_mask + b * p.mask_stride : nullptr;
  auto page_at = [&](int j) {
    return j < end ? kv4_page(table, p.table_stride, p.pages, p.page_size, j) : -1;
  };
  R raw;
  int j = begin + warp * 16;
  int page = page_at(j), page_next = page_at(j + 16 * kWarps);
  auto load = [&](R& dst, int at, int pg) {
    if (pg < 0) return;
    const int64_t row = (static_cast<int64_t>(pg) * p.heads + h) * p.page_size + at % p.page_size;
    dst.load(p.k_codes + row * (D / 2), p.k_params + row * (D / 32), p.v_codes + row * (D / 2),
             p.v_params + row * (D / 32), t0, c, g);
  };
  load(raw, j, page);
  for (; j < end; j += 16 * kWarps) {
    R cur = raw;
    const int pg = page;
    page = page_next;
    load(raw, j + 16 * kWarps, page);
    page_next = page_at(j + 32 * kWarps);
    if (pg < 0) continue;
    // entries that no row may use: beyond the length or hidden by the mask
    uint32_t vis = 0xffffu;
    const bool whole = j + 16 <= seen_first;
    if (mask || !whole) {
      const int at = j + (lane & 15);
      const bool v = at < end && (!mask || __ldg(mask + at) != 0);
      vis = __ballot_sync(kFull, v) & 0xffffu;
      if (vis == 0u) continue;
    }

    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const Kv4Scale s0 = kv4_scale(cur.k_param(0, w)), s1 = kv4_scale(cur.k_param(1, w));
      uint32_t a0 = kv4_pair<0>(cur.k[0][w], s0), a1 = kv4_pair<0>(cur.k[1][w], s1);
      uint32_t a2 = kv4_pair<1>(cur.k[0][w], s0), a3 = kv4_pair<1>(cur.k[1][w], s1);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_bf16(s[t], a0, a1, a2, a3, q[t][2 * w][0], q[t][2 * w][1]);
      a0 = kv4_pair<2>(cur.k[0][w], s0), a1 = kv4_pair<2>(cur.k[1][w], s1);
      a2 = kv4_pair<3>(cur.k[0][w], s0), a3 = kv4_pair<3>(cur.k[1][w], s1);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma_bf16(s[t], a0, a1, a2, a3, q[t][2 * w + 1][0], q[t][2 * w + 1][1]);
    }
    // scores in base 2; hidden ones -inf, and hidden entries' values read as 0 (whatever they hold)
    bool above = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] *= p.scale_log2;
    }
    if (mask || !whole) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int entry = t0 + (e >> 1) * 8;
          const int r = r0 + t * 8 + 2 * c + (e & 1);
          const int bound = p.causal ? len - p.n + r / p.G + 1 : len;
          if (!(vis >> entry & 1u) || j + entry >= bound) s[t][e] = -INFINITY;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(vis >> (c + 4 * e) & 1u)) {
#pragma unroll
          for (int k = 0; k < R::VP; ++k) cur.vp[e][k] = 0u;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int x = 0; x < 2; ++x) above |= fmaxf(s[t][x], s[t][x + 2]) > m[t][x];
    }
    // the running maximum moves rarely after the first tiles: only then is it reduced over the
    // lanes and what was summed so far rescaled
    if (__any_sync(kFull, above)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = fmaxf(s[t][x], s[t][x + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
          const float mn = fmaxf(m[t][x], mx);
          const float keep = mn == -INFINITY ? 1.f : ex2(m[t][x] - mn);
          m[t][x] = mn;
          l[t][x] *= keep;
#pragma unroll
          for (int k = 0; k < MT; ++k) {
            o[t][k][x] *= keep;
            o[t][k][x + 2] *= keep;
          }
        }
      }
    }
    uint32_t pt[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0];
      const float m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
      const float p0 = ex2(s[t][0] - m0), p1 = ex2(s[t][1] - m1);
      const float p2 = ex2(s[t][2] - m0), p3 = ex2(s[t][3] - m1);
      l[t][0] += p0 + p2;
      l[t][1] += p1 + p3;
      pt[t][0] = transpose8x8(bf2_pack(p0, p1));
      pt[t][1] = transpose8x8(bf2_pack(p2, p3));
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      // entries (c, c + 4) and (c + 8, c + 12) side by side: fragment columns 2c, 2c + 1, + 8
      const Kv4Scale sa = kv4_scale(__byte_perm(cur.v_param(0, w), cur.v_param(1, w), 0x5410));
      const Kv4Scale sb = kv4_scale(__byte_perm(cur.v_param(2, w), cur.v_param(3, w), 0x5410));
      const uint32_t al = __byte_perm(cur.v[0][w], cur.v[1][w], 0x5410);
      const uint32_t ah = __byte_perm(cur.v[0][w], cur.v[1][w], 0x7632);
      const uint32_t bl = __byte_perm(cur.v[2][w], cur.v[3][w], 0x5410);
      const uint32_t bh = __byte_perm(cur.v[2][w], cur.v[3][w], 0x7632);
      const uint32_t fa[8] = {kv4_pair<0>(al, sa), kv4_pair<1>(al, sa), kv4_pair<2>(al, sa),
                              kv4_pair<3>(al, sa), kv4_pair<0>(ah, sa), kv4_pair<1>(ah, sa),
                              kv4_pair<2>(ah, sa), kv4_pair<3>(ah, sa)};
      const uint32_t fb[8] = {kv4_pair<0>(bl, sb), kv4_pair<1>(bl, sb), kv4_pair<2>(bl, sb),
                              kv4_pair<3>(bl, sb), kv4_pair<0>(bh, sb), kv4_pair<1>(bh, sb),
                              kv4_pair<2>(bh, sb), kv4_pair<3>(bh, sb)};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_bf16(o[t][w * 4 + k], fa[2 * k], fa[2 * k + 1], fb[2 * k], fb[2 * k + 1], pt[t][0],
                   pt[t][1]);
      }
    }
  }

  // join the warps: common maximum, rescaled sums
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float v = l[t][x];
      v += __shfl_xor_sync(kFull, v, 4);
      v += __shfl_xor_sync(kFull, v, 8);
      v += __shfl_xor_sync(kFull, v, 16);
      if (g == 0) {
        sm[warp][t * 8 + 2 * c + x] = m[t][x];
        sl[warp][t * 8 + 2 * c + x] = v;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = t * 8 + 2 * c + x;
      float mx = sm[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm[w][r]);
      const float keep = m[t][x] == -INFINITY ? 0.f : ex2(m[t][x] - mx);
      float* dst = so + (warp * ROWS + r) * D;
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        // the lane's word holds channels 0..7; tile k of the word has channels 2k and 2k + 1
        float* d8 = dst + R::v_word(w, g) * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float2*>(d8 + 2 * k) =
              make_float2(o[t][w * 4 + k][x] * keep, o[t][w * 4 + k][x + 2] * keep);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < ROWS * (D / 2); e += kThreads) {
    const int r = e / (D / 2), ch = e - r * (D / 2);
    if (r0 + r >= rows) break;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = *reinterpret_cast<const float2*>(so + (w * ROWS + r) * D + 2 * ch);
      acc.x += v.x;
      acc.y += v.y;
    }
    float mx = sm[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm[w][r]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      sum += sm[w][r] == -INFINITY ? 0.f : sl[w][r] * ex2(sm[w][r] - mx);
    const int64_t head_row = (static_cast<int64_t>(b) * p.heads + h) * rows + r0 + r;
    if (f.part_o) {
      const int64_t at = head_row * f.splits + split;
      *reinterpret_cast<float2*>(f.part_o + at * D + 2 * ch) = acc;
      if (ch == 0) f.part_ml[at] = make_float2(mx, sum);
    } else {
      const int i = (r0 + r) / p.G, hq = h * p.G + (r0 + r) - i * p.G;
      uint16_t* dst = p.out + b * p.ob + i * p.ot + hq * p.oh + 2 * ch;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const uint32_t w = bf2_pack(acc.x * inv, acc.y * inv);
      dst[0] = static_cast<uint16_t>(w);
      dst[1] = static_cast<uint16_t>(w >> 16);
      if (ch == 0 && p.lse)
        p.lse[(static_cast<int64_t>(b) * p.heads * p.G + hq) * p.n + i] =
            sum > 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
    }
  }
}

// Join the splits of each row in order: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.  One
// warp per row.
template <int D>
__global__ void __launch_bounds__(kThreads)
    attention_join_kernel(const __grid_constant__ AttnParams p, const float* part_o,
                          const float2* part_ml, int splits, int chunk) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  pdl_wait();
  pdl_trigger();
  const int rows = p.n * p.G;
  if (row >= static_cast<int64_t>(p.B) * p.heads * rows) return;
  const int r = static_cast<int>(row % rows);
  const int h = static_cast<int>(row / rows % p.heads), b = static_cast<int>(row / rows / p.heads);
  const int len = p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
  const int used = max(1, (len + chunk - 1) / chunk);
  const float2* ml = part_ml + row * splits;
  float mx = -INFINITY;
  for (int s = lane; s < used; s += 32) mx = fmaxf(mx, ml[s].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  float acc[D / 32] = {}, sum = 0.f;
  const float* src = part_o + row * splits * D;
  for (int s = 0; s < used; ++s) {
    const float2 v = ml[s];
    if (v.x == -INFINITY) continue;
    const float keep = ex2(v.x - mx);
    sum = fmaf(v.y, keep, sum);
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      const float2 x = *reinterpret_cast<const float2*>(src + static_cast<int64_t>(s) * D + 64 * k + 2 * lane);
      acc[2 * k] = fmaf(x.x, keep, acc[2 * k]);
      acc[2 * k + 1] = fmaf(x.y, keep, acc[2 * k + 1]);
    }
  }
  const int i = r / p.G, hq = h * p.G + r - i * p.G;
  uint16_t* dst = p.out + b * p.ob + i * p.ot + hq * p.oh;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const uint32_t w = bf2_pack(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    dst[64 * k + 2 * lane] = static_cast<uint16_t>(w);
    dst[64 * k + 2 * lane + 1] = static_cast<uint16_t>(w >> 16);
  }
  if (p.lse && lane == 0)
    p.lse[(static_cast<int64_t>(b) * p.heads * p.G + hq) * p.n + i] =
        sum > 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

struct Split {
  int nt, row_tiles, splits, chunk;
  size_t off_ml, bytes;
};

Split plan_few(int B, int n, int q_heads, int heads, int D, int max_len, int sm_count) {
  Split s{};
  const int64_t rows = static_cast<int64_t>(n) * (q_heads / heads);
  s.nt = rows > 8 && D <= 128 ? 2 : 1;
  s.row_tiles = static_cast<int>((rows + 8 * s.nt - 1) / (8 * s.nt));
  const int64_t base = static_cast<int64_t>(B) * heads * s.row_tiles;
  const int unit = 16 * kWarps;
  const int64_t units = std::max<int64_t>(1, (static_cast<int64_t>(max_len) + unit - 1) / unit);
  const int64_t want = std::max<int64_t>(1, (static_cast<int64_t>(sm_count) * 6 + base - 1) / base);
  const int64_t most = std::max<int64_t>(1, units / 4);
  const int64_t splits = std::min(want, most);
  s.chunk = static_cast<int>((units + splits - 1) / splits) * unit;
  s.splits = static_cast<int>((units * unit + s.chunk - 1) / s.chunk);
  s.bytes = kWsHeader;
  if (s.splits > 1) {
    const size_t parts = static_cast<size_t>(B) * heads * rows * s.splits;
    s.off_ml = kWsHeader + align_up(parts * D * 4, 256);
    s.bytes = s.off_ml + parts * 8;
  }
  return s;
}

template <int D, int NT>
cudaError_t launch_few(const AttnParams& p, FewPlan f, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(kWarps) * 8 * NT * D * 4;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(attention_few_kernel<D, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks = static_cast<int64_t>(p.B) * p.heads * f.row_tiles * f.splits;
  cudaError_t e = launch_dependent(attention_few_kernel<D, NT>, dim3(static_cast<unsigned>(blocks)),
                                   dim3(kThreads), smem, stream, p, f);
  if (e != cudaSuccess || !f.part_o) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.heads * p.n * p.G;
  return launch_dependent(attention_join_kernel<D>,
                          dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)), dim3(kThreads),
                          0, stream, p, static_cast<const float*>(f.part_o),
                          static_cast<const float2*>(f.part_ml), f.splits, f.chunk);
}

}  // namespace

size_t attention_ws_bytes(int B, int n, int q_heads, int heads, int D, int max_len, int sm_count) {
  return plan_few(B, n, q_heads, heads, D, max_len, sm_count).bytes;
}

cudaError_t launch_attention(AttnParams p, int D, void* ws, int sm_count, cudaStream_t stream) {
  const Split s = plan_few(p.B, p.n, p.heads * p.G, p.heads, D, p.max_len, sm_count);
  FewPlan f{};
  f.chunk = s.chunk;
  f.splits = s.splits;
  f.row_tiles = s.row_tiles;
  f.q_aligned = (reinterpret_cast<uintptr_t>(p.q) | static_cast<uintptr_t>(p.qb * 2) |
                 static_cast<uintptr_t>(p.qt * 2) | static_cast<uintptr_t>(p.qh * 2)) % 16 == 0;
  if (s.splits > 1) {
    f.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
    f.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + s.off_ml);
  }
  switch (D * 10 + s.nt) {
    case 641: return launch_few<64, 1>(p, f, stream);
    case 642: return launch_few<64, 2>(p, f, stream);
    case 1281: return launch_few<128, 1>(p, f, stream);
    case 1282: return launch_few<128, 2>(p, f, stream);
    case 1921: return launch_few<192, 1>(p, f, stream);
    default: return launch_few<256, 1>(p, f, stream);
  }
}

}  // namespace dllm

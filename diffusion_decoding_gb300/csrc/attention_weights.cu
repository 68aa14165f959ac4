// How much attention each cache entry receives: the column sums of the softmax weights that
// dllm_attention_kv4 computed, recomputed from its log-sum-exps,
//   got[j] = sum over queries and heads that see j of exp(scale * q.K_j - lse).
// Nothing but K is read of the cache, and no running maximum is needed: lse is final.
//
// Here, for few query rows per cache head (attention_weights_tc.cu: many): a warp takes 32 entries and
// computes S^T [32 entries x 8 rows] = K Q^T with mma.sync m16n8k16, the cache as the left operand
// (kv4.cuh turns codes into exact bf16 values in the fragments' lanes), head by head with the next
// head's codes on their way; the queries of a sequence are laid out in shared memory as the fragments
// want them.  The sums over rows and heads stay in the lanes, so nothing is joined.  Where there are few
// entries the warps of a CTA share out the heads and add up at the end.
#include <algorithm>

#include "attention.h"
#include "attention_weights.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// K of one entry row as a lane of four holds it: words (of eight channels) c * KW ... of the row, or,
// at head_dim 192, where those would straddle groups, words 4 i + c.
template <int D>
struct KRow {
  static constexpr int KW = D / 32;
  static constexpr bool kSpread = D == 192;
  static constexpr int PARAMS = kSpread ? 6 : D == 256 ? 2 : 1;
  uint32_t w[KW], par[PARAMS];

  static __device__ __forceinline__ int word(int i, int c) { return kSpread ? 4 * i + c : c * KW + i; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < KW; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < PARAMS; ++i) par[i] = 0u;
  }
  __device__ __forceinline__ void load(const AttnParams& p, int64_t row, int c) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.k_codes + row * (D / 2));
    const uint16_t* ps = p.k_params + row * (D / 32);
    if constexpr (kSpread) {
#pragma unroll
      for (int i = 0; i < KW; ++i) w[i] = __ldg(src + 4 * i + c), par[i] = __ldg(ps + i);
    } else if constexpr (D == 64) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + c);
      w[0] = v.x, w[1] = v.y;
      par[0] = __ldg(ps + (c >> 1));
    } else {
#pragma unroll
      for (int i = 0; i < KW / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + c * (KW / 4) + i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        par[i] = __ldg(ps + c * (KW / 4) + i);
      }
    }
  }
  __device__ __forceinline__ Kv4Scale scale(int i) const {
    const uint32_t x = par[kSpread ? i : i / 4];
    return kv4_scale(__byte_perm(x, x, 0x1010));
  }
};

// Rows of a row tile: 8 * NT.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps)
    attention_weights_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWeights x) {
  using R = KRow<D>;
  constexpr int KW = R::KW, ROWS = 8 * NT;
  constexpr bool kAhead = D <= 128;  // registers for the next head's codes
  extern __shared__ __align__(16) uint8_t dyn[];
  uint4* q_s = reinterpret_cast<uint4*>(dyn);  // [heads of a turn][NT][KW][32 lanes]
  float* l_s = reinterpret_cast<float*>(q_s + x.heads_at_once * NT * KW * 32);  // [heads of a turn][ROWS]
  __shared__ float sums[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int b = blockIdx.x / x.ctas_per_seq;
  const int len = p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
  const int per_cta = 32 * (kWarps >> x.split_log2);
  const int first = (blockIdx.x - b * x.ctas_per_seq) * per_cta;
  if (first >= len) return;
  const int part = warp & ((1 << x.split_log2) - 1), split = 1 << x.split_log2;
  const int j = first + 32 * (warp >> x.split_log2);
  const int rows = p.n * p.G;
  const uint8_t* mask = p.key_mask ? p.key_mask + b * p.mask_stride : nullptr;
  // of two tiles of 16 entries, each in one page: where head 0 of the lane's rows g and g + 8 starts
  int64_t at[2];
  bool shown[2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int jt = j + 16 * e, t = jt / p.page_size;
    const int page = jt < len ? __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + t) : -1;
    const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
    at[e] = (static_cast<int64_t>(there ? page : 0) * p.heads) * p.page_size + jt - t * p.page_size + g;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int jj = jt + g + 8 * y;
      shown[e][y] = there && jj < len && (!mask || __ldg(mask + jj) != 0);
    }
  }
  const bool some0 = __any_sync(kFull, shown[0][0] || shown[0][1]);
  const bool some1 = __any_sync(kFull, shown[1][0] || shown[1][1]);
  float acc[2][2] = {};
  R cur[2][2], next[2][2];
  auto load = [&](R (&k)[2][2], int h) {
    const int64_t up = static_cast<int64_t>(h) * p.page_size;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (e ? some1 : some0)
          k[e][y].load(p, at[e] + up + 8 * y, c);
        else
          k[e][y].clear();
      }
    }
  };
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    int see[NT][2];  // entries that the lane's query rows (columns of S^T) see
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = r0 + 8 * t + 2 * c + y;
        see[t][y] = r >= rows ? 0 : p.causal ? min(len, len - p.n + r / p.G + 1) : len;
      }
    }
    const bool diagonal = p.causal && j + 32 > len - p.n + r0 / p.G + 1;
    for (int h0 = 0; h0 < p.heads; h0 += x.heads_at_once) {
      const int h1 = min(h0 + x.heads_at_once, p.heads);
      if (kAhead && h0 + part < h1) load(next, h0 + part);
      if (r0 + h0 > 0) __syncthreads();
      for (int k = threadIdx.x; k < (h1 - h0) * NT * KW * 32; k += 32 * kWarps) {
        // lane l of word w: channels of word(w, l % 4) of row l / 4, in pairs (m, m + 4) as the codes give
        const int l = k & 31, w = k / 32 % KW, t = k / (32 * KW) % NT, h = h0 + k / (32 * KW * NT);
        const int r = r0 + 8 * t + (l >> 2), i = r / p.G;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (r < rows) {
          const uint16_t* s8 = p.q + b * p.qb + i * p.qt +
                               (static_cast<int64_t>(h) * p.G + r - i * p.G) * p.qh + R::word(w, l & 3) * 8;
          if (x.q_aligned) {
            const uint4 y = *reinterpret_cast<const uint4*>(s8);
            v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
          } else {
#pragma unroll
            for (int m = 0; m < 4; ++m) v[m] = s8[2 * m] | static_cast<uint32_t>(s8[2 * m + 1]) << 16;
          }
        }
        q_s[k] = make_uint4(__byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632),
                            __byte_perm(v[1], v[3], 0x5410), __byte_perm(v[1], v[3], 0x7632));
      }
      for (int k = threadIdx.x; k < (h1 - h0) * ROWS; k += 32 * kWarps) {
        const int r = r0 + k % ROWS, h = h0 + k / ROWS, i = r / p.G;
        float l = -INFINITY;  // adds nothing
        if (r < rows)
          l = x.lse[(static_cast<int64_t>(b) * p.heads * p.G + h * p.G + r - i * p.G) * p.n + i];
        l_s[k] = l == -INFINITY ? l : minus_l(x, l);
      }
      __syncthreads();
      if (!some0 && !some1) continue;
      for (int h = h0 + part; h < h1; h += split) {
        if constexpr (kAhead) {
#pragma unroll
          for (int e = 0; e < 4; ++e) cur[e >> 1][e & 1] = next[e >> 1][e & 1];
          if (h + split < h1) load(next, h + split);
        } else {
          load(cur, h);
        }
        const uint4* q_h = q_s + (h - h0) * NT * KW * 32 + lane;
        float s[2][NT][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int t = 0; t < NT; ++t) s[e][t][0] = s[e][t][1] = s[e][t][2] = s[e][t][3] = 0.f;
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t a[2][2][4];  // channel pairs of the lane's two rows
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const Kv4Scale sc = cur[e][y].scale(w);
              const uint32_t k = cur[e][y].w[w];
              a[e][y][0] = kv4_pair<0>(k, sc), a[e][y][1] = kv4_pair<1>(k, sc);
              a[e][y][2] = kv4_pair<2>(k, sc), a[e][y][3] = kv4_pair<3>(k, sc);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 q = q_h[(t * KW + w) * 32];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mma_bf16(s[e][t], a[e][0][0], a[e][1][0], a[e][0][1], a[e][1][1], q.x, q.y);
              mma_bf16(s[e][t], a[e][0][2], a[e][1][2], a[e][0][3], a[e][1][3], q.z, q.w);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 l = *reinterpret_cast<const float2*>(l_s + (h - h0) * ROWS + 8 * t + 2 * c);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float w = ex2(fmaf(s[e][t][y], p.scale_log2, y & 1 ? l.y : l.x));
              if (diagonal && j + 16 * e + g + 8 * (y >> 1) >= see[t][y & 1]) w = 0.f;
              acc[e][y >> 1] += w;
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float v = acc[e][y];
      v += __shfl_xor_sync(kFull, v, 1);
      v += __shfl_xor_sync(kFull, v, 2);
      if (c == 0) sums[warp][16 * e + 8 * y + g] = shown[e][y] ? v : 0.f;
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < per_cta; k += 32 * kWarps) {
    const int jj = first + k;
    if (jj >= len) break;
    float v = 0.f;
    for (int w = 0; w < split; ++w) v += sums[(k >> 5 << x.split_log2) + w][k & 31];
    put_weight(x, b, jj, v);
  }
}

template <int D, int NT>
cudaError_t launch_nt(const AttnParams& p, AttnWeights x, int sm_count, cudaStream_t stream) {
  // The warps of a CTA share out the heads while that does not leave fewer of them than the GPU holds
  // (the codes of a head are a warp's unit of work, one after the other).
  const int64_t tiles = static_cast<int64_t>(p.B) * ((p.max_len + 31) / 32);
  while ((2 << x.split_log2) <= kWarps && (1 << x.split_log2) < p.heads &&
         (tiles << x.split_log2) < 8 * static_cast<int64_t>(sm_count))
    ++x.split_log2;
  const int per_cta = 32 * (kWarps >> x.split_log2);
  x.ctas_per_seq = (p.max_len + per_cta - 1) / per_cta;
  constexpr int kHead = NT * (D / 32) * 512 + 8 * NT * 4;  // bytes of shared memory
  x.heads_at_once = std::min(p.heads, 64 * 1024 / kHead);
  const size_t smem = static_cast<size_t>(x.heads_at_once) * kHead;
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem<attention_weights_kernel<D, NT>>(64 * 1024);
    if (e != cudaSuccess) return e;
  }
  attention_weights_kernel<D, NT>
      <<<static_cast<unsigned>(static_cast<int64_t>(p.B) * x.ctas_per_seq), 32 * kWarps, smem, stream>>>(p, x);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const AttnParams& p, const AttnWeights& x, int sm_count, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.n) * p.G;
  if (rows <= 8) return launch_nt<D, 1>(p, x, sm_count, stream);
  if (rows <= 16) return launch_nt<D, 2>(p, x, sm_count, stream);
  return launch_nt<D, 4>(p, x, sm_count, stream);
}

}  // namespace

size_t attention_weights_ws_bytes(int B, int n, int G, int heads, int D, int max_len, int sm_count) {
  return weights_tc_takes(B, n, G, heads, max_len)
             ? weights_tc_ws_bytes(B, n, G, heads, D, max_len, sm_count)
             : kWsHeader;
}

cudaError_t launch_attention_weights(const AttnParams& p, AttnWeights x, int D, void* ws, int sm_count,
                                     cudaStream_t stream) {
  if (p.max_len == 0) return cudaSuccess;
  x.q_aligned = attention_rows_aligned(p.q, p.qb, p.qt, p.qh);
  // The scores are multiplied by scale_log2 = scale * log2(e) as it is rounded, so the log-sum-exps by the
  // same number over scale: the exponent's error is then relative to the exponent itself.
  const double ratio = x.scale != 0.f ? static_cast<double>(p.scale_log2) / x.scale : 1.4426950408889634074;
  x.l_hi = static_cast<float>(ratio);
  x.l_lo = static_cast<float>(ratio - static_cast<double>(x.l_hi));
  if (weights_tc_takes(p.B, p.n, p.G, p.heads, p.max_len) && weights_tc_scale(x.scale))
    return launch_weights_tc(p, x, D, ws, sm_count, stream);
  switch (D) {
    case 64: return launch<64>(p, x, sm_count, stream);
    case 128: return launch<128>(p, x, sm_count, stream);
    case 192: return launch<192>(p, x, sm_count, stream);
    default: return launch<256>(p, x, sm_count, stream);
  }
}

}  // namespace dllm

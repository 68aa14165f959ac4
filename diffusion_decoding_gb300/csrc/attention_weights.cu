// How much attention each cache entry receives: the column sums of the softmax weights that
// dllm_attention_kv4 computed, recomputed from its log-sum-exps,
//   got[j] = sum over queries and heads that see j of exp(scale * q.K_j - lse).
// Nothing but K is read of the cache, and no running maximum is needed: lse is final.
//
// A warp takes 16 entries and computes S^T [16 entries x 8 rows] = K Q^T with mma.sync m16n8k16, the
// cache as the left operand (kv4.cuh turns codes into exact bf16 values in the fragments' lanes);
// the sums over rows and heads stay in the lanes.
#include <algorithm>

#include "attention.h"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kWarps = 4;

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

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
    attention_weights_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWeights x) {
  constexpr int KW = KRow<D>::KW;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int b = blockIdx.x / x.ctas_per_seq;
  const int len = p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
  const int j = ((blockIdx.x - b * x.ctas_per_seq) * kWarps + warp) * 16;
  if (j >= len) return;
  const int rows = p.n * p.G;
  // the tile lies in one page (page sizes are multiples of 16)
  const int t = j / p.page_size;
  const int page = t < p.table_stride ? __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + t) : -1;
  const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
  const uint8_t* mask = p.key_mask ? p.key_mask + b * p.mask_stride : nullptr;
  bool shown[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int jj = j + g + 8 * e;
    shown[e] = there && jj < len && (!mask || __ldg(mask + jj) != 0);
  }
  float acc[2] = {0.f, 0.f};
  if (__any_sync(kFull, shown[0] || shown[1])) {
    for (int h = 0; h < p.heads; ++h) {
      const int64_t row = (static_cast<int64_t>(page) * p.heads + h) * p.page_size + j - t * p.page_size;
      KRow<D> k[2];
      k[0].load(p, row + g, c);
      k[1].load(p, row + g + 8, c);
      for (int r0 = 0; r0 < rows; r0 += 8) {
        const int r = r0 + g, i = r / p.G;
        const uint16_t* src = p.q + b * p.qb + i * p.qt + (static_cast<int64_t>(h) * p.G + r - i * p.G) * p.qh;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t v[4] = {0u, 0u, 0u, 0u};
          if (r < rows) {
            const uint16_t* s8 = src + KRow<D>::word(w, c) * 8;
            if (x.q_aligned) {
              const uint4 y = *reinterpret_cast<const uint4*>(s8);
              v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
            } else {
#pragma unroll
              for (int m = 0; m < 4; ++m) v[m] = s8[2 * m] | static_cast<uint32_t>(s8[2 * m + 1]) << 16;
            }
          }
          // channels come out of the codes in pairs (m, m + 4)
          const Kv4Scale s0 = k[0].scale(w), s1 = k[1].scale(w);
          mma_bf16(s, kv4_pair<0>(k[0].w[w], s0), kv4_pair<0>(k[1].w[w], s1), kv4_pair<1>(k[0].w[w], s0),
                   kv4_pair<1>(k[1].w[w], s1), __byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632));
          mma_bf16(s, kv4_pair<2>(k[0].w[w], s0), kv4_pair<2>(k[1].w[w], s1), kv4_pair<3>(k[0].w[w], s0),
                   kv4_pair<3>(k[1].w[w], s1), __byte_perm(v[1], v[3], 0x5410), __byte_perm(v[1], v[3], 0x7632));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int rr = r0 + 2 * c + y;
          if (rr >= rows) continue;
          const int ii = rr / p.G;
          const int see = p.causal ? min(len, len - p.n + ii + 1) : len;
          const float l = x.lse[(static_cast<int64_t>(b) * p.heads * p.G + h * p.G + rr - ii * p.G) * p.n + ii];
          if (l == -INFINITY) continue;  // it saw nothing
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (shown[e] && j + g + 8 * e < see)
              acc[e] += ex2(fmaf(s[y + 2 * e], p.scale_log2, -l * kLog2e));
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    acc[e] += __shfl_xor_sync(kFull, acc[e], 1);
    acc[e] += __shfl_xor_sync(kFull, acc[e], 2);
    const int jj = j + g + 8 * e;
    if (c == 0 && jj < len)
      x.out[b * x.out_stride + jj] = x.prior ? fmaf(x.keep, x.prior[b * x.prior_stride + jj], acc[e]) : acc[e];
  }
}

template <int D>
cudaError_t launch(const AttnParams& p, const AttnWeights& x, cudaStream_t stream) {
  attention_weights_kernel<D><<<static_cast<unsigned>(p.B * x.ctas_per_seq), 32 * kWarps, 0, stream>>>(p, x);
  return cudaGetLastError();
}

}  // namespace

size_t attention_weights_ws_bytes(int B, int n, int G, int heads, int D, int max_len, int sm_count) {
  return kWsHeader;
}

cudaError_t launch_attention_weights(const AttnParams& p, AttnWeights x, int D, void* ws, int sm_count,
                                     cudaStream_t stream) {
  if (p.max_len == 0) return cudaSuccess;
  x.ctas_per_seq = (p.max_len + 16 * kWarps - 1) / (16 * kWarps);
  x.q_aligned = attention_rows_aligned(p.q, p.qb, p.qt, p.qh);
  switch (D) {
    case 64: return launch<64>(p, x, stream);
    case 128: return launch<128>(p, x, stream);
    case 192: return launch<192>(p, x, stream);
    default: return launch<256>(p, x, stream);
  }
}

}  // namespace dllm

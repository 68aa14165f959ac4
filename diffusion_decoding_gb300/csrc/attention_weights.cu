// How much attention each cache entry receives: the column sums of the softmax weights that
// dllm_attention_kv4 computed, recomputed from its log-sum-exps,
//   got[j] = sum over queries and heads that see j of exp(scale * q.K_j - lse).
// Nothing but K is read of the cache, and no running maximum is needed: lse is final.
//
// Here, for few query rows per cache head (attention_weights_tc.cu: many): a warp takes 32 entries and
// computes S^T [32 entries x 8 rows] = K Q^T with mma.sync m16n8k16, the cache as the left operand
// (kv4.cuh turns codes into exact bf16 values in the fragments' lanes), head by head.  Codes and params
// come through a ring of the warp's own in shared memory (16-byte asynchronous copies); the queries of a
// sequence are laid out in shared memory as the fragments want them.  The sums over rows and heads stay
// in the lanes, so nothing is joined.  Where there are few entries the warps of a CTA share out the heads
// and add up at the end.
//
// Nothing is full: 0.42 of the copy rate, and 490 instructions for 32 entries of a head of 128 channels
// (codes to bf16 more than a third), which are half of the issue slots, the integer pipe 53 % busy.  The 24
// warps an SM that the registers leave room for do not fill the other half.  32 sequences of up to 8192
// entries, 8 heads of 128, 4 rows each: 41 us (with codes loaded to registers ahead instead of through the
// ring 43; a warp a head with its queries in registers 54; CTAs of four warps 47).
#include <algorithm>

#include "attention.h"
#include "attention_weights.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "mbarrier.cuh"

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

constexpr int kStages = 3;

// A stage: codes of 32 entries of one head, then their params.  A lane of four reads words (of eight
// channels) c * KW ... of a row, or, at head_dim 192, where those would straddle groups, words 4 i + c.
template <int D>
struct Stage {
  static constexpr int KW = D / 32, ROW = D / 2, PAR = D / 16;
  static constexpr bool kSpread = D == 192;
  static constexpr int kParams = 32 * ROW, kBytes = kParams + 32 * PAR;
  static constexpr int kPieces = 16 * ROW / 16;     // 16-byte pieces of codes of half a stage (one page)
  static constexpr int kParPieces = 16 * PAR / 16;  // and of params
  // 128-byte rows are read by eight lanes at a time in two rows: their pieces are permuted
  static __device__ __forceinline__ int place(int row, int piece) {
    return row * ROW + 16 * (D == 256 ? piece ^ (row & 1) : piece);
  }
  static __device__ __forceinline__ int word(int i, int c) { return kSpread ? 4 * i + c : c * KW + i; }
  uint32_t w[KW], par[kSpread ? 6 : D == 256 ? 2 : 1];

  // Row `row` of the stage at `at`.
  __device__ __forceinline__ void read(uint32_t at, int row, int c) {
    const uint32_t ps = at + kParams + row * PAR;
    if constexpr (kSpread) {
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(at + row * ROW + 16 * i + 4 * c));
        par[i] = ld_shared_u16(ps + 2 * i);
      }
    } else if constexpr (D == 64) {
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at + row * ROW + 8 * c));
      par[0] = ld_shared_u16(ps + 2 * (c >> 1));
    } else {
#pragma unroll
      for (int i = 0; i < KW / 4; ++i) {
        const uint4 v = ld_shared_v4(at + place(row, c * (KW / 4) + i));
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        par[i] = ld_shared_u16(ps + 2 * (c * (KW / 4) + i));
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
__global__ void __launch_bounds__(32 * kWarps, D <= 128 && NT == 1 ? 3 : 2)
    attention_weights_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWeights x) {
  using R = Stage<D>;
  constexpr int KW = R::KW, ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t dyn[];
  const uint32_t ring = smem_u32(dyn) + (threadIdx.x >> 5) * kStages * R::kBytes;
  uint4* q_s = reinterpret_cast<uint4*>(dyn + kWarps * kStages * R::kBytes);  // [heads of a turn][NT][KW][32 lanes]
  float* l_s = reinterpret_cast<float*>(q_s + x.heads_at_once * NT * KW * 32);  // [heads of a turn][ROWS]
  __shared__ float sums[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int b = blockIdx.x / x.ctas_per_seq;
  const int len = p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
  const int split = 1 << x.split_log2, part = warp & (split - 1), step = 32 * (kWarps >> x.split_log2);
  const int first = (blockIdx.x - b * x.ctas_per_seq) * step * x.tiles_per_warp;
  if (first >= len) return;
  const int j0 = first + 32 * (warp >> x.split_log2);  // this warp's tiles: every step entries
  const int tiles = max(0, min(x.tiles_per_warp, (len - j0 + step - 1) / step));
  const int rows = p.n * p.G;
  const uint8_t* mask = p.key_mask ? p.key_mask + b * p.mask_stride : nullptr;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  const uint32_t page_rows = static_cast<uint32_t>(p.heads) * p.page_size;

  // ---- the walk through the stages, ahead of the computation: heads h0 + part, + split ... of each tile
  int j_ahead, h_ahead, tiles_ahead, h0, h1;
  int page_next[2];
  // of the lane's pieces of both halves (half a tile lies in one page), null where its page is absent
  const uint8_t *codes[2], *params[2];
  auto look = [&](int j) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int jt = j + 16 * e;
      page_next[e] = jt < len ? __ldg(table + x.by_page(static_cast<uint32_t>(jt))) : -1;
    }
  };
  auto point = [&](int j) {  // at head h0 + part of the tile at j, whose pages are in page_next
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int jt = j + 16 * e, slot = jt - static_cast<int>(x.by_page(static_cast<uint32_t>(jt))) * p.page_size;
      const int64_t row =
          static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(page_next[e])) * page_rows) +
          (static_cast<int64_t>(h0 + part) * p.page_size + slot);
      const bool there = static_cast<unsigned>(page_next[e]) < static_cast<unsigned>(p.pages);
      codes[e] = there ? p.k_codes + row * R::ROW + lane * 16 : nullptr;
      params[e] = reinterpret_cast<const uint8_t*>(p.k_params) + row * R::PAR + lane * 16;
    }
  };
  auto begin = [&]() {
    j_ahead = j0;
    h_ahead = h0 + part;
    tiles_ahead = h_ahead < h1 ? tiles : 0;
    if (tiles_ahead > 0) {
      look(j0);
      point(j0);
      look(j0 + step);
    }
  };
  const uint32_t dst_codes = ring + R::place(lane / (R::ROW / 16), lane % (R::ROW / 16));
  const uint32_t head_codes = static_cast<uint32_t>(split * p.page_size) * R::ROW,
                 head_params = static_cast<uint32_t>(split * p.page_size) * R::PAR;
  auto copy = [&](uint32_t at) {
    if (tiles_ahead > 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (codes[e] == nullptr) continue;
#pragma unroll
        for (int i = 0; i < (R::kPieces + 31) / 32; ++i) {
          // (32 pieces on: whole rows, an even number of them, except at head_dim 192)
          const int k = lane + 32 * i;
          const uint32_t to = R::kSpread ? ring + R::place(16 * e + k / (R::ROW / 16), k % (R::ROW / 16))
                                         : dst_codes + 16 * e * R::ROW + 512 * i;
          if (R::kPieces % 32 == 0 || k < R::kPieces) cp_async16(to + at, codes[e] + 512 * i);
        }
        if (lane < R::kParPieces) cp_async16(ring + R::kParams + 16 * e * R::PAR + lane * 16 + at, params[e]);
        codes[e] += head_codes;
        params[e] += head_params;
      }
      h_ahead += split;
      if (h_ahead >= h1) {
        h_ahead = h0 + part;
        --tiles_ahead;
        j_ahead += step;
        if (tiles_ahead > 0) point(j_ahead);
        if (tiles_ahead > 1) look(j_ahead + step);
      }
    }
    cp_async_commit();
  };

  float acc[2][2] = {};
  // the sums of the tile at j, entries 16 e + 8 y + g in the lanes c = 0
  auto finish = [&](int j) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int jt = j + 16 * e, t = static_cast<int>(x.by_page(static_cast<uint32_t>(jt)));
      const int pg = jt < len ? __ldg(table + t) : -1;
      const bool there = static_cast<unsigned>(pg) < static_cast<unsigned>(p.pages);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int jj = jt + 8 * y + g;
        float v = acc[e][y];
        v += __shfl_xor_sync(kFull, v, 1);
        v += __shfl_xor_sync(kFull, v, 2);
        if (c == 0) {
          // (an entry that does not count may have met anything)
          v = there && jj < len && (!mask || __ldg(mask + jj) != 0) ? v : 0.f;
          if (split > 1)
            sums[warp][16 * e + 8 * y + g] = v;
          else if (jj < len)
            put_weight(x, b, jj, v);
        }
        acc[e][y] = 0.f;
      }
    }
  };

  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    int see[NT][2];  // entries that the lane's query rows (columns of S^T) see
    if (p.causal) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = r0 + 8 * t + 2 * c + y;
          see[t][y] = r >= rows ? 0 : min(len, len - p.n + r / p.G + 1);
        }
      }
    }
    const int all_see = p.causal ? len - p.n + r0 / p.G + 1 : len;  // what every row sees
    for (h0 = 0; h0 < p.heads; h0 += x.heads_at_once) {
      h1 = min(h0 + x.heads_at_once, p.heads);
      const bool last_turn = r0 + ROWS >= rows && h1 == p.heads;
      begin();
#pragma unroll
      for (int k = 0; k < kStages - 1; ++k) copy(k * R::kBytes);
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
      uint32_t at = 0u, into = (kStages - 1) * R::kBytes;
      for (int i = 0, j = j0; i < tiles; ++i, j += step) {
        const bool diagonal = j + 32 > all_see && p.causal;
        for (int h = h0 + part; h < h1; h += split) {
          cp_async_wait_group<kStages - 2>();
          __syncwarp();  // every lane's pieces have landed, and all are done with the stage before
          copy(into);
          into = at;
          const uint32_t from = ring + at;
          at = at == (kStages - 1) * R::kBytes ? 0u : at + R::kBytes;
          const uint4* q_h = q_s + (h - h0) * NT * KW * 32 + lane;
          float s[2][NT][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int t = 0; t < NT; ++t) s[e][t][0] = s[e][t][1] = s[e][t][2] = s[e][t][3] = 0.f;
          }
          R k[2][2];
#pragma unroll
          for (int e = 0; e < 4; ++e) k[e >> 1][e & 1].read(from, 16 * (e >> 1) + 8 * (e & 1) + g, c);
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            uint32_t a[2][2][4];  // channel pairs of the lane's two rows
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const Kv4Scale sc = k[e][y].scale(w);
                const uint32_t v = k[e][y].w[w];
                a[e][y][0] = kv4_pair<0>(v, sc), a[e][y][1] = kv4_pair<1>(v, sc);
                a[e][y][2] = kv4_pair<2>(v, sc), a[e][y][3] = kv4_pair<3>(v, sc);
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
              for (int y = 0; y < 4; ++y)
                s[e][t][y] = ex2(fmaf(s[e][t][y], p.scale_log2, y & 1 ? l.y : l.x));
            }
          }
          if (diagonal) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (j + 16 * e + g + 8 * (y >> 1) >= see[t][y & 1]) s[e][t][y] = 0.f;
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              acc[e][0] += s[e][t][0] + s[e][t][1];
              acc[e][1] += s[e][t][2] + s[e][t][3];
            }
          }
        }
        if (last_turn) finish(j);
      }
      cp_async_wait_all();
      __syncwarp();
    }
  }
  if (split == 1) return;
  __syncthreads();
  for (int k = threadIdx.x; k < step; k += 32 * kWarps) {
    const int jj = first + k;
    if (jj >= len) break;
    float v = 0.f;
    for (int w = 0; w < split; ++w) v += sums[(k >> 5 << x.split_log2) + w][k & 31];
    put_weight(x, b, jj, v);
  }
}

template <int D, int NT>
cudaError_t launch_nt(const AttnParams& p, AttnWeights x, int sm_count, cudaStream_t stream) {
  constexpr int kHead = NT * (D / 32) * 512 + 8 * NT * 4;  // bytes of shared memory of a head's queries
  constexpr size_t kRing = static_cast<size_t>(kWarps) * kStages * Stage<D>::kBytes;
  x.heads_at_once = std::min(p.heads, 48 * 1024 / kHead);
  // The warps of a CTA share out the heads while that does not leave fewer of them than the GPU holds (the
  // codes of a head are a warp's unit of work, one after the other).
  const int64_t tiles = static_cast<int64_t>(p.B) * ((p.max_len + 31) / 32);
  while ((2 << x.split_log2) <= kWarps && (2 << x.split_log2) <= p.heads &&
         (tiles << x.split_log2) < 8 * static_cast<int64_t>(sm_count))
    ++x.split_log2;
  // Several tiles a warp, one after the other, while three CTAs an SM are left: what a CTA sets up first is
  // then a small part of its time.
  x.tiles_per_warp = 1;
  if (x.split_log2 == 0 && p.n * p.G <= 8 * NT && x.heads_at_once == p.heads)
    x.tiles_per_warp =
        static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, tiles / (kWarps * int64_t{3} * sm_count))));
  const int per_cta = 32 * (kWarps >> x.split_log2) * x.tiles_per_warp;
  x.ctas_per_seq = (p.max_len + per_cta - 1) / per_cta;
  const size_t smem = kRing + static_cast<size_t>(x.heads_at_once) * kHead;
  const cudaError_t e = allow_smem<attention_weights_kernel<D, NT>>(kRing + 48 * 1024);
  if (e != cudaSuccess) return e;
  attention_weights_kernel<D, NT>
      <<<static_cast<unsigned>(static_cast<int64_t>(p.B) * x.ctas_per_seq), 32 * kWarps, smem, stream>>>(p, x);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const AttnParams& p, const AttnWeights& x, int sm_count, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.n) * p.G;
  if (rows <= 8) return launch_nt<D, 1>(p, x, sm_count, stream);
  // (more rows come here with 64 channels, or with a scale that the other kernel cannot have)
  if (rows <= 16 || D > 64) return launch_nt<D, 2>(p, x, sm_count, stream);
  return launch_nt<D, D == 64 ? 4 : 2>(p, x, sm_count, stream);
}

}  // namespace

size_t attention_weights_ws_bytes(int B, int n, int G, int heads, int D, int max_len) {
  return weights_tc_takes(B, n, G, heads, D, max_len) ? weights_tc_ws_bytes(B, n, G, heads, D, max_len)
                                                      : kWsHeader;
}

cudaError_t launch_attention_weights(const AttnParams& p, AttnWeights x, int D, void* ws, int sm_count,
                                     cudaStream_t stream) {
  if (p.max_len == 0) return cudaSuccess;
  x.q_aligned = attention_rows_aligned(p.q, p.qb, p.qt, p.qh);
  x.by_page = divisor(static_cast<uint32_t>(p.page_size));
  // The scores are multiplied by scale_log2 = scale * log2(e) as it is rounded, so the log-sum-exps by the
  // same number over scale: the exponent's error is then relative to the exponent itself.
  const double ratio = x.scale != 0.f ? static_cast<double>(p.scale_log2) / x.scale : 1.4426950408889634074;
  x.l_hi = static_cast<float>(ratio);
  x.l_lo = static_cast<float>(ratio - static_cast<double>(x.l_hi));
  if (weights_tc_takes(p.B, p.n, p.G, p.heads, D, p.max_len) && weights_tc_scale(x.scale))
    return launch_weights_tc(p, x, D, ws, sm_count, stream);
  switch (D) {
    case 64: return launch<64>(p, x, sm_count, stream);
    case 128: return launch<128>(p, x, sm_count, stream);
    case 192: return launch<192>(p, x, sm_count, stream);
    default: return launch<256>(p, x, sm_count, stream);
  }
}

}  // namespace dllm

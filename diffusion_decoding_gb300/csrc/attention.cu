// Attention over the 4-bit cache for few query rows per cache head (single tokens, small blocks),
// and the kernel that joins the parts of a split (dInfer explainer, KV-cache manager: the block's
// positions attend over the cached prefix and the block).
//
// Rows are the n * G queries that share a cache head, row r = i * G + g; a row tile is 8 * NT of
// them.  A warp takes 16 cache entries at a time and computes the transposed products
//   S^T [16 entries x rows] = K Q^T,   O^T [channels x rows] += V^T P^T
// with mma.sync m16n8k16, so that the cache is the left operand in both and nothing is padded
// beyond eight rows.  K and V are turned from codes into exact bf16 values in the registers of the
// lanes that the fragments want them in; nothing is transposed (P^T comes out of S^T by
// movmatrix).  The order of channels inside a product is free, so the lane's words are contiguous.
//
// The grid is one wave of resident CTAs that share the work evenly (attention_line.cuh).
//
// An entry of one head costs 9/8 * head_dim bytes of HBM traffic.  Each warp keeps kStages - 1 tiles on
// their way into a ring of its own in shared memory (16-byte asynchronous copies, no block
// barrier), and page ids one tile further ahead.
//
// Measured: one token of each of 32 sequences of up to 8192 entries, 4 query heads to each of 8 cache
// heads of 128 channels: 65.5 us, 3.5 TB/s of cache, 0.51 of the copy rate.  No unit is full: 66 % of the
// issue slots and 63 % of the integer pipe are busy, and warps that could issue wait for one another
// or for that pipe.  A warp issues 452 instructions for a tile of 16 entries.  Turning its codes takes
// 192 of them (64 pairs a lane at a shift, a mask and a packed fma); the rest is the walk through the
// pages, copies, loads from the ring, votes, scores and products, and is paid for every 16 entries.
// Registers (121) allow four warps a scheduler; five CTAs an SM spill (72.7 us).  One sequence of
// 65536 entries: 21 us, of which the join takes a third.
#include "attention.h"

#include <algorithm>

#include "attention_line.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "mbarrier.cuh"

namespace dllm {
namespace {

// Warps of a CTA: four, so that many CTAs share an SM's registers; eight where segments are few and
// short, so that each is done in half the steps.
constexpr int kWarps = 4, kWideWarps = 8;

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

// N words of shared memory at p with the widest loads their alignment (N * 4 bytes) allows.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t p, uint32_t* w) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(p));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p));
}
// A tile of 16 entries in shared memory: K codes, V codes (rows in the order of the fragments'
// rows), K params, V params (in entry order).
//
// Fragment row g (0..7) holds entry (g >> 1) + 4 * (g & 1), row g + 8 the entry 8 further; the V
// fragments of lane c then want entries c, c + 4, c + 8, c + 12, rows 2c, 2c + 1, 2c + 8, 2c + 9.
// How the channels of an entry are spread over the lanes: K: lane c of four holds D / 32 words, V:
// lane g of eight holds D / 64.  The words of a lane are contiguous, except at head_dim 192, where
// contiguous words would straddle groups: there word i of lane l is i * lanes + l.  The 16-byte
// pieces of a row are permuted within their 128-byte line so that neither the K nor the V loads
// meet in a bank (head_dim 192: two lanes a bank).
template <int D>
struct Tile {
  static constexpr int KW = D / 32, VW = D / 64, ROW = D / 2;
  static constexpr bool kSpread = D == 192;
  static constexpr int kV = 16 * ROW, kKp = 32 * ROW, kVp = kKp + D, kBytes = kKp + 2 * D;
  static constexpr int PIECES = D / 64;  // 16-byte pieces of K (and of V) a lane copies

  static __device__ __forceinline__ int row_of(int entry) {
    return (entry & 8) + 2 * (entry & 3) + (entry >> 2 & 1);
  }
  // byte of piece q of row r
  static __device__ __forceinline__ int place(int r, int q) {
    if constexpr (D == 64) return (r * 32 + q * 16) ^ ((r >> 2 & 1) * 32);
    if constexpr (D == 128) return (r * 64 + q * 16) ^ ((r >> 1 & 3) * 32);
    if constexpr (D == 256) return r * 128 + ((q ^ 2 * (r >> 1 & 3) ^ (r & 1)) * 16);
    return r * 96 + q * 16;
  }
  static __device__ __forceinline__ int k_word(int i, int c) { return kSpread ? 4 * i + c : c * KW + i; }
  static __device__ __forceinline__ int v_word(int i, int g) { return kSpread ? 8 * i + g : g * VW + i; }

  uint32_t k[2][KW], v[4][VW];
  uint32_t kp[2][kSpread ? 6 : D == 256 ? 2 : 1], vp[4][kSpread ? 3 : 1];

  // What a lane reads, as bytes from the tile's start: K words of row g (row g + 8 is 8 rows
  // further; head_dim 256: also the next piece), V words of rows 2c and 2c + 1, and their params.
  struct Lane {
    uint32_t k, k2, kp, v0, v1, vp;
    __device__ __forceinline__ Lane(uint32_t ring, int c, int g) {
      const int entry = (g >> 1) + 4 * (g & 1);
      constexpr int LANES = kSpread ? 4 : 4 / VW;  // lanes of a V piece
      k2 = 0u;
      if constexpr (kSpread) {
        k = place(g, 0) + 4 * c;
        kp = entry * (D / 16);
      } else if constexpr (D == 256) {
        k = place(g, 2 * c);
        k2 = ring + place(g, 2 * c + 1);
        kp = entry * (D / 16) + 4 * c;
      } else if constexpr (D == 128) {
        k = place(g, c);
        kp = entry * (D / 16) + 2 * c;
      } else {
        k = place(g, c >> 1) + 8 * (c & 1);
        kp = entry * (D / 16) + 2 * (c >> 1);
      }
      const int in = kSpread ? 4 * (g & 3) : (g % LANES) * VW * 4;
      v0 = ring + kV + place(2 * c, g / LANES) + in;
      v1 = ring + kV + place(2 * c + 1, g / LANES) + in;
      vp = ring + kVp + c * (D / 16) + 2 * (kSpread ? g >> 2 : g * VW / 4);
      k += ring;
      kp += ring + kKp;
    }
  };

  // `at`: bytes of the stage from the ring's start
  __device__ __forceinline__ void read_k(const Lane& l, uint32_t at) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t row = at + 8 * ROW * e, par = l.kp + at + 8 * (D / 16) * e;
      if constexpr (kSpread) {
#pragma unroll
        for (int i = 0; i < KW; ++i) lds_words<1>(l.k + row + 16 * i, &k[e][i]);
#pragma unroll
        for (int i = 0; i < 6; ++i) kp[e][i] = ld_shared_u16(par + 2 * i);
      } else if constexpr (D == 256) {
        lds_words<4>(l.k + row, &k[e][0]);
        lds_words<4>(l.k2 + row, &k[e][4]);
        kp[e][0] = ld_shared_u16(par);
        kp[e][1] = ld_shared_u16(par + 2);
      } else {
        lds_words<KW>(l.k + row, &k[e][0]);
        kp[e][0] = ld_shared_u16(par);
      }
    }
  }
  __device__ __forceinline__ void read_v(const Lane& l, uint32_t at) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t row = (e & 1 ? l.v1 : l.v0) + at + 8 * ROW * (e >> 1);
      const uint32_t par = l.vp + at + 4 * (D / 16) * e;
      if constexpr (kSpread) {
#pragma unroll
        for (int i = 0; i < VW; ++i) lds_words<1>(row + 32 * i, &v[e][i]);
#pragma unroll
        for (int i = 0; i < 3; ++i) vp[e][i] = ld_shared_u16(par + 4 * i);
      } else {
        lds_words<VW>(row, &v[e][0]);
        vp[e][0] = ld_shared_u16(par);
      }
    }
  }
  // param of K word i of entry e, in both halves
  __device__ __forceinline__ uint32_t k_param(int e, int i) const {
    const uint32_t w = kp[e][kSpread ? i : i / 4];
    return __byte_perm(w, w, 0x1010);
  }
  __device__ __forceinline__ uint32_t v_param(int e, int i) const { return vp[e][kSpread ? i : 0]; }
};

// A weight may reach 2^kSlack before the reference moves: sums of 2^30 of them stay far inside fp32,
// and bf16 keeps the same relative precision at every magnitude.
constexpr float kSlack = 8.f;
constexpr uint32_t kDiagonal = 1u << 16;  // beside a tile's 16 entries: not all rows see the same of them

// CTAs of the one resident wave per SM: what the registers allow (checked with -Xptxas -v).
constexpr int few_ctas_per_sm(int D, int NT) {
  return D == 64 ? (NT == 1 ? 5 : 4) : D == 128 ? (NT == 1 ? 4 : 3) : 2;
}
constexpr int kStages = 4;
template <int D, int NT, int WARPS>
constexpr size_t few_smem() {
  const size_t ring = static_cast<size_t>(WARPS) * kStages * Tile<D>::kBytes;
  const size_t join = static_cast<size_t>(WARPS) * 8 * NT * D * 4;
  return ring > join ? ring : join;
}

// A function of its own: inlined it costs single tokens over a masked cache 2 %.
template <int D, int ROWS>
__device__ __noinline__ void put_nans_few(const AttnParams& p, const AttnPlan& f, Segment<ROWS> sg, int u0,
                                          int u1) {
  put_nans<D, ROWS, 16, false>(p, f, sg, u0, u1);
}

template <int D, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, few_ctas_per_sm(D, NT) * kWarps / WARPS)
    attention_few_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPlan f) {
  using R = Tile<D>;
  constexpr int KW = R::KW, VW = R::VW, MT = D / 16, ROWS = 8 * NT, kThreads = 32 * WARPS;
  constexpr int kStep = 16 * WARPS;  // entries that the warps take together
  extern __shared__ __align__(128) float4 smem_raw[];  // (the rings' bank pattern counts on it)
  float* so = reinterpret_cast<float*>(smem_raw);  // [WARPS][ROWS][D]
  __shared__ float sm[WARPS][ROWS], sl[WARPS][ROWS];
  __shared__ uint32_t nan_s[WARPS];  // the warp met a NaN of V on the diagonal

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int rows = p.n * p.G;
  pdl_wait();
  pdl_trigger();
  Line<ROWS> line;
  line.build(p, f);
  const int u0 = line.start(blockIdx.x), u1 = line.start(blockIdx.x + 1);
  if (u0 >= u1) return;
  Segment<ROWS> sg;
  sg.find(p, f, line, u0);

  const int t0 = (g >> 1) + (g & 1) * 4;  // entry of fragment row g
  const int step_pages = kStep / p.page_size, step_slots = kStep % p.page_size;
  // this warp's ring, and where the lane's pieces of a tile go
  const uint32_t ring = smem_u32(smem_raw) + warp * kStages * R::kBytes;
  uint32_t dst[R::PIECES];
#pragma unroll
  for (int i = 0; i < R::PIECES; ++i) {
    const int piece = lane + 32 * i;
    dst[i] = ring + R::place(R::row_of(piece / (D / 32)), piece % (D / 32));
  }
  const uint32_t dst_par = ring + (lane < 16 ? R::kKp : R::kVp) + (lane & 15) * 16;
  const uint16_t* par_of_lane = (lane < 16 ? p.k_params : p.v_params) + (lane & 15) * 8;
  const uint8_t* k_of_lane = p.k_codes + lane * 16;
  const uint8_t* v_of_lane = p.v_codes + lane * 16;
  const typename R::Lane at_lane(ring, c, g);

  if (lane == 0) nan_s[warp] = 0u;
  for (int u = u0; u < u1;) {
    const int piece = min(sg.units - sg.k0, u1 - u);
    const int b = sg.b, h = sg.h, len = sg.len, r0 = sg.rt * ROWS, k0 = sg.k0;
    const int seen_first = rows_see(p, len, r0);  // what the tile's first row sees
    const int end = min(sg.seen, (k0 + piece) << f.unit_log2);

    // queries: channel pairs (j, j + 4) of the lane's words, as the K fragments hold them
    uint32_t q[NT][2 * KW][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = r0 + t * 8 + g;
      const int i = token_of(p, r);
      const uint16_t* src =
          p.q + b * p.qb + i * p.qt + (static_cast<int64_t>(h) * p.G + r - i * p.G) * p.qh;
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
            for (int k = 0; k < 4; ++k)
              x[k] = s8[2 * k] | static_cast<uint32_t>(s8[2 * k + 1]) << 16;
          }
        }
        q[t][2 * w][0] = __byte_perm(x[0], x[2], 0x5410);
        q[t][2 * w][1] = __byte_perm(x[0], x[2], 0x7632);
        q[t][2 * w + 1][0] = __byte_perm(x[1], x[3], 0x5410);
        q[t][2 * w + 1][1] = __byte_perm(x[1], x[3], 0x7632);
      }
    }
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
    // the walk through the pages, ahead of the computation: word of the table and slot of the
    // next tile to copy
    const int j0 = (k0 << f.unit_log2) + warp * 16;
    int j_ahead = j0;
    int t_ahead = j_ahead / p.page_size, slot_ahead = j_ahead - t_ahead * p.page_size;
    // (the word is looked at only when its tile is copied: a test here would wait for the load)
    auto page_ahead = [&]() {
      return j_ahead < end && t_ahead < p.table_stride ? __ldg(table + t_ahead) : -1;
    };
    int page = page_ahead();
    // copy the next tile into the stage at byte `at` of the ring and look the page after it up;
    // whether the tile was there
    auto copy = [&](uint32_t at) {
      const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
      if (there) {
        const int64_t row = (static_cast<int64_t>(page) * p.heads + h) * p.page_size + slot_ahead;
        const uint8_t* ks = k_of_lane + row * (D / 2);
        const uint8_t* vs = v_of_lane + row * (D / 2);
#pragma unroll
        for (int i = 0; i < R::PIECES; ++i) {
          cp_async16(dst[i] + at, ks + 512 * i);
          cp_async16(dst[i] + at + R::kV, vs + 512 * i);
        }
        if ((lane & 15) < D / 16) cp_async16(dst_par + at, par_of_lane + row * (D / 32));
      }
      cp_async_commit();
      j_ahead += kStep;
      t_ahead += step_pages;
      slot_ahead += step_slots;
      if (slot_ahead >= p.page_size) {
        slot_ahead -= p.page_size;
        ++t_ahead;
      }
      page = page_ahead();
      return there;
    };

    auto compute = [&](uint32_t at, int j) {
      R cur;
      // entries that no row may use: beyond the length or hidden by the mask
      uint32_t vis = 0xffffu;
      const bool whole = j + 16 <= seen_first;
      if (mask || !whole) {
        const int e = j + (lane & 15);
        vis = __ballot_sync(kFull, e < end && (!mask || __ldg(mask + e) != 0)) & 0xffffu;
        if (vis == 0u) return;
        if (p.causal && !whole) vis |= kDiagonal;
      }
      cur.read_k(at_lane, at);
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const Kv4Scale s0 = kv4_scale(cur.k_param(0, w)), s1 = kv4_scale(cur.k_param(1, w));
        uint32_t a0 = kv4_pair<0>(cur.k[0][w], s0), a1 = kv4_pair<0>(cur.k[1][w], s1);
        uint32_t a2 = kv4_pair<1>(cur.k[0][w], s0), a3 = kv4_pair<1>(cur.k[1][w], s1);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_bf16(s[t], a0, a1, a2, a3, q[t][2 * w][0], q[t][2 * w][1]);
        a0 = kv4_pair<2>(cur.k[0][w], s0), a1 = kv4_pair<2>(cur.k[1][w], s1);
        a2 = kv4_pair<3>(cur.k[0][w], s0), a3 = kv4_pair<3>(cur.k[1][w], s1);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_bf16(s[t], a0, a1, a2, a3, q[t][2 * w + 1][0], q[t][2 * w + 1][1]);
      }
      // scores in base 2; hidden ones -inf, and hidden entries' values read as 0 (whatever they
      // hold)
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
            const int bound = rows_see(p, len, r);
            if (!(vis >> entry & 1u) || j + entry >= bound) s[t][e] = -INFINITY;
          }
        }
      }
      bool above = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) above |= fmaxf(s[t][x], s[t][x + 2]) > m[t][x] + kSlack;
      }
      // m is a reference that no score exceeds by more than kSlack, not the maximum itself: it
      // moves rarely after the first tile, and only then are the scores reduced over the lanes and
      // what was summed so far rescaled
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
      cur.read_v(at_lane, at);
      if (vis != 0xffffu) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(vis >> (c + 4 * e) & 1u)) {
#pragma unroll
            for (int k = 0; k < (R::kSpread ? 3 : 1); ++k) cur.vp[e][k] = 0u;
          }
        }
        if (vis & kDiagonal) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int k = 0; k < (R::kSpread ? 3 : 1); ++k)
              if (kv4_nan(cur.vp[e][k])) cur.vp[e][k] = 0u, nan_s[warp] = 1u;
          }
        }
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
    };

    uint32_t there = 0;  // bit k: the tile k steps ahead is there
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) there |= copy(k * R::kBytes) ? 1u << k : 0u;
    uint32_t at = 0, into = (kStages - 1) * R::kBytes;
    for (int j = j0; j < end; j += kStep) {
      cp_async_wait_group<kStages - 2>();
      __syncwarp();  // every lane's pieces have landed, and all are done with the stage before
      there |= copy(into) ? 1u << (kStages - 1) : 0u;
      if (there & 1u) compute(at, j);
      there >>= 1;
      into = at;
      at = at == (kStages - 1) * R::kBytes ? 0u : at + R::kBytes;
    }
    cp_async_wait_all();
    __syncthreads();  // the rings become the buffers of the join

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
        for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, sm[w][r]);
        const float keep = m[t][x] == -INFINITY ? 0.f : ex2(m[t][x] - mx);
        float* dst = so + (warp * ROWS + r) * D;
        if (r0 + r >= rows) continue;
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
    const bool direct = piece == sg.units;
    const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (u == u0 ? 0 : 1);
    if (threadIdx.x == 0) note_segment(f, p, line, sg, u, u0, direct);
    for (int e = threadIdx.x; e < ROWS * (D / 2); e += kThreads) {
      const int r = e / (D / 2), ch = e - r * (D / 2);
      if (r0 + r >= rows) break;
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(so + (w * ROWS + r) * D + 2 * ch);
        acc.x += v.x;
        acc.y += v.y;
      }
      float mx = sm[0][r];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, sm[w][r]);
      // A warp whose reference is -inf saw nothing (a sum of 0) or scores that are NaN (a sum of NaN).
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
        sum += sm[w][r] == -INFINITY ? sl[w][r] : sl[w][r] * ex2(sm[w][r] - mx);
      if (!direct) {
        *reinterpret_cast<float2*>(f.part_o + (part * ROWS + r) * D + 2 * ch) = acc;
        if (ch == 0) f.part_ml[part * ROWS + r] = make_float2(mx, sum);
      } else {
        const int i = token_of(p, r0 + r), hq = h * p.G + (r0 + r) - i * p.G;
        uint16_t* dst = p.out + b * p.ob + i * p.ot + hq * p.oh + 2 * ch;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const uint32_t w = bf2_pack(acc.x * inv, acc.y * inv);
        dst[0] = static_cast<uint16_t>(w);
        dst[1] = static_cast<uint16_t>(w >> 16);
        if (ch == 0 && p.lse)
          p.lse[(static_cast<int64_t>(b) * p.heads * p.G + hq) * p.n + i] =
              sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
      }
    }
    u += piece;
    if (u < u1) {
      __syncthreads();  // the buffers are reused
      sg.next(p, f);
    }
  }
  if (!p.causal) return;
  __syncthreads();
  uint32_t nan_met = nan_s[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) nan_met |= nan_s[w];
  if (nan_met) {
    sg.find(p, f, line, u0);
    put_nans_few<D, ROWS>(p, f, sg, u0, u1);
  }
}

struct FewSizes {
  int nt, row_tiles, ctas, unit_log2;
  bool wide;   // eight warps a CTA
  bool split;  // some segment can have more than one unit
  size_t off_ml, off_parts, bytes;
};

FewSizes few_sizes(int B, int n, int G, int heads, int D, int max_len, int sm_count) {
  FewSizes s{};
  const int64_t rows = static_cast<int64_t>(n) * G, per_tile = static_cast<int64_t>(B) * heads;
  constexpr int kShort = 9;
  const bool brief = max_len <= 1 << kShort;
  // Sixteen rows a tile read the cache half as often (16 rows over 32 x 8192 entries: 94 us, 141 with
  // eight); eight where short segments leave SMs free anyway (1 x 331 entries: 7.3 us, 8.9 with 16).
  s.nt = rows > 8 && D <= 128 && !(brief && per_tile * ((rows + 7) / 8) <= sm_count) ? 2 : 1;
  s.row_tiles = static_cast<int>((rows + 8 * s.nt - 1) / (8 * s.nt));
  const int64_t segments = per_tile * s.row_tiles;
  // Up to 2^kShort entries a segment is one unit: its warps take it in a few tiles each, sooner than a
  // second kernel could join its parts; in eight warps' steps where that leaves no SM without a CTA.
  // Four segments of 512 entries take 7.5 us whole with eight warps, 8.6 with four, 7.4 to 7.6 split;
  // 64 segments 7.9, 9.0 and 9 to 10; four of 1024 entries 10.8 whole and 7.5 split.  (Sixteen warps
  // lose more in adding up their rows than they gain: 331 entries 7.7 us, 6.5 with eight.)
  s.wide = brief && segments <= sm_count;
  s.ctas = s.wide ? sm_count : sm_count * few_ctas_per_sm(D, s.nt);
  s.unit_log2 = brief ? kShort : unit_log2_of(segments, max_len, 6);
  s.split = max_len > 1 << s.unit_log2;
  const size_t parts = static_cast<size_t>(2) * s.ctas * 8 * s.nt;
  s.off_ml = kWsHeader + parts * D * 4;
  s.off_parts = s.off_ml + parts * 8;
  s.bytes = s.off_parts + static_cast<size_t>(B) * s.row_tiles * heads * 8;
  return s;
}

template <int D, int NT, int WARPS>
cudaError_t launch_few_warps(const AttnParams& p, const AttnPlan& f, cudaStream_t stream) {
  constexpr size_t smem = few_smem<D, NT, WARPS>();
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = allow_smem<attention_few_kernel<D, NT, WARPS>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(attention_few_kernel<D, NT, WARPS>, dim3(f.ctas), dim3(32 * WARPS), smem,
                          stream, p, f);
}

template <int D, int NT>
cudaError_t launch_few(const AttnParams& p, const AttnPlan& f, const FewSizes& s,
                       cudaStream_t stream) {
  if (s.wide) return launch_few_warps<D, NT, kWideWarps>(p, f, stream);
  const cudaError_t e = launch_few_warps<D, NT, kWarps>(p, f, stream);
  if (e != cudaSuccess || !s.split) return e;
  return launch_join<D, 8 * NT>(p, f, stream);
}

}  // namespace

bool attention_rows_aligned(const void* x, int64_t sb, int64_t st, int64_t sh) {
  return (reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(sb * 2) |
          static_cast<uintptr_t>(st * 2) | static_cast<uintptr_t>(sh * 2)) % 16 == 0;
}

size_t attention_ws_bytes(int B, int n, int G, int heads, int D, int max_len, int sm_count) {
  // which kernel runs depends on the lengths too: enough for both
  const size_t few = few_sizes(B, n, G, heads, D, max_len, sm_count).bytes;
  return attention_tc_can(n, G, D)
             ? std::max(few, attention_tc_ws_bytes(B, n, G, heads, D, sm_count))
             : few;
}

cudaError_t launch_attention(const AttnParams& p, int D, void* ws, int sm_count, cudaStream_t stream) {
  if (attention_tc_takes(p, D, sm_count)) return launch_attention_tc(p, D, ws, sm_count, stream);
  const FewSizes s = few_sizes(p.B, p.n, p.G, p.heads, D, p.max_len, sm_count);
  AttnPlan f{};
  f.row_tiles = s.row_tiles;
  f.ctas = s.ctas;
  f.unit_log2 = s.unit_log2;
  f.whole = !s.split;
  f.q_aligned = attention_rows_aligned(p.q, p.qb, p.qt, p.qh);
  f.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  f.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + s.off_ml);
  f.parts = reinterpret_cast<int2*>(static_cast<char*>(ws) + s.off_parts);
  switch (D * 10 + s.nt) {
    case 641: return launch_few<64, 1>(p, f, s, stream);
    case 642: return launch_few<64, 2>(p, f, s, stream);
    case 1281: return launch_few<128, 1>(p, f, s, stream);
    case 1282: return launch_few<128, 2>(p, f, s, stream);
    case 1921: return launch_few<192, 1>(p, f, s, stream);
    default: return launch_few<256, 1>(p, f, s, stream);
  }
}

}  // namespace dllm

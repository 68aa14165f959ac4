// How the attention's work is shared out, and the kernel that joins what was split.
//
// Rows are the n * G queries of a sequence that share a cache head, row r = i * G + g; a row tile
// is ROWS of them.  A segment is one (sequence, row tile, head); the entries it has to look at are
// cut into units.  All segments form one line of units, and CTA k of a single resident wave takes
// the k-th equal stretch of it, whatever the lengths.  A segment inside one stretch is written
// straight to the output; of the others each CTA leaves a partial result (at most two a CTA: the
// segments its stretch begins and ends in), which attention_join_kernel adds in order; the CTA that
// starts a segment notes where they are.
#pragma once

#include "attention.h"
#include "common.cuh"
#include "kv4.cuh"

namespace dllm {

struct AttnPlan {
  int unit_log2;    // entries of a unit, a power of two; the line has fewer than 2^31 units
  int whole;        // a segment is one unit whatever its length: the line needs no lengths
  int row_tiles;
  int q_aligned;    // query rows on 16-byte boundaries
  int out_aligned;  // output rows too
  int copy_span;    // entries that surely lie in one page: 16, 32 or 64
  float* part_o;    // [2 * CTAs, rows of a tile, D]
  float2* part_ml;  // [2 * CTAs, rows of a tile]: reference (base 2) and sum of weights
  int2* parts;      // [segments]: see note_segment
  int ctas;
  int32_t* status;
};

// log2 of the entries of a unit: at least `least`, and so many that no line reaches 2^31 units (2^30 at
// most, for up to 2^30 segments of up to 2^30 entries).
inline int unit_log2_of(int64_t segments, int max_len, int least) {
  int lg = least;
  auto units = [&] {
    const int64_t n = (static_cast<int64_t>(max_len) + (int64_t{1} << lg) - 1) >> lg;
    return segments * (n > 1 ? n : 1);
  };
  while (units() >= (int64_t{1} << 31)) ++lg;
  return lg;
}

namespace {

__device__ __forceinline__ int length_of(const AttnParams& p, int b) {
  return p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
}
__device__ __forceinline__ int units_of(int entries, const AttnPlan& f) {
  return max(1, (entries + (1 << f.unit_log2) - 1) >> f.unit_log2);
}
// Token of row r.
__device__ __forceinline__ int token_of(const AttnParams& p, int r) {
  return p.g_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(r), p.g_magic))
                   : p.G == 1 ? r : r / p.G;
}
// Row r sees the entries below this (if its mask and the pages let it).
__device__ __forceinline__ int rows_see(const AttnParams& p, int len, int r) {
  return p.causal ? min(len, len - p.n + token_of(p, r) + 1) : len;
}
// The last row of a tile sees the most.
template <int ROWS>
__device__ __forceinline__ int tile_sees(const AttnParams& p, int len, int rt) {
  return rows_see(p, len, min((rt + 1) * ROWS, p.n * p.G) - 1);
}

// The line of units: items (sequence, row tile) in order, each with the same units for every head,
// cut into f.ctas stretches that differ by one unit at most.  Built and asked by whole warps.
template <int ROWS>
struct Line {
  int total, each, longer;  // units; units of a stretch; stretches with one unit more
  int own, upto;            // this lane's item (of the first 32): its units, and all up to it
  int items;
  bool equal;

  __device__ __forceinline__ int weight(const AttnParams& p, const AttnPlan& f, int item) const {
    if (item >= items) return 0;
    if (f.whole) return p.heads;
    const int b = f.row_tiles == 1 ? item : item / f.row_tiles, rt = item - b * f.row_tiles;
    return p.heads * units_of(tile_sees<ROWS>(p, length_of(p, b), rt), f);
  }
  static __device__ __forceinline__ int scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += x;
    }
    return v;
  }
  __device__ __forceinline__ void build(const AttnParams& p, const AttnPlan& f) {
    items = p.B * f.row_tiles;
    equal = f.whole || (!p.lens && !p.causal);
    if (equal) {
      total = weight(p, f, 0) * items;
    } else {
      own = weight(p, f, threadIdx.x & 31);
      upto = scan(own);
      total = __shfl_sync(kFull, upto, 31);
      int sum = 0;
      for (int k = 32 + (threadIdx.x & 31); k < items; k += 32) sum += weight(p, f, k);
      if (items > 32) total += static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(sum)));
    }
    each = static_cast<int>(static_cast<unsigned>(total) / static_cast<unsigned>(f.ctas));
    longer = total - each * f.ctas;
  }
  // first unit of CTA c's stretch
  __device__ __forceinline__ int start(int c) const { return each * c + min(c, longer); }
  // CTA whose stretch holds unit u
  __device__ __forceinline__ int holder(int u) const {
    const int head = longer * (each + 1);
    return u < head ? static_cast<int>(static_cast<unsigned>(u) / static_cast<unsigned>(each + 1))
                    : longer + static_cast<int>(static_cast<unsigned>(u - head) /
                                                static_cast<unsigned>(each));
  }
  // item that holds unit `at` (< total), and the units before that item
  __device__ __forceinline__ int find(const AttnParams& p, const AttnPlan& f, int at,
                                      int* before) const {
    const int lane = threadIdx.x & 31;
    if (equal) {
      const int per = weight(p, f, 0), item = at / per;
      *before = item * per;
      return item;
    }
    int base = 0, mine = own, incl = upto;
    for (int i0 = 0;;) {
      const unsigned hit = __ballot_sync(kFull, base + incl > at);
      if (hit != 0u || i0 + 32 >= items) {
        const int l = hit ? __ffs(hit) - 1 : 31;
        *before = base + __shfl_sync(kFull, incl - mine, l);
        return min(i0 + l, items - 1);
      }
      base += __shfl_sync(kFull, incl, 31);
      i0 += 32;
      mine = weight(p, f, i0 + lane);
      incl = scan(mine);
    }
  }
};

// Where a CTA is on the line: a segment and the unit in it.
template <int ROWS>
struct Segment {
  int item, b, rt, h;
  int len;    // of the sequence
  int seen;   // entries the tile's last row sees
  int units;  // of the segment
  int k0;     // first unit to do

  __device__ __forceinline__ void at_item(const AttnParams& p, const AttnPlan& f) {
    b = f.row_tiles == 1 ? item : item / f.row_tiles;
    rt = item - b * f.row_tiles;
    len = length_of(p, b);
    seen = tile_sees<ROWS>(p, len, rt);
    units = units_of(seen, f);
  }
  __device__ __forceinline__ void find(const AttnParams& p, const AttnPlan& f, const Line<ROWS>& line,
                                       int u) {
    int before;
    item = line.find(p, f, u, &before);
    at_item(p, f);
    const int in = u - before;
    h = static_cast<int>(static_cast<unsigned>(in) / static_cast<unsigned>(units));
    k0 = in - h * units;
  }
  __device__ __forceinline__ void next(const AttnParams& p, const AttnPlan& f) {
    k0 = 0;
    if (++h == p.heads) {
      h = 0;
      ++item;
      at_item(p, f);
    }
  }
};

// What the CTA that starts a segment leaves for the join: its part, and the last CTA that has one
// (the CTAs between have theirs first in their stretches); {-1, 0} for a segment that is whole.
template <int ROWS>
__device__ __forceinline__ void note_segment(const AttnPlan& f, const AttnParams& p,
                                             const Line<ROWS>& line, const Segment<ROWS>& sg,
                                             int u, int u0, bool whole) {
  if (sg.k0 != 0) return;
  f.parts[static_cast<int64_t>(sg.item) * p.heads + sg.h] =
      whole ? make_int2(-1, 0)
            : make_int2(2 * static_cast<int>(blockIdx.x) + (u == u0 ? 0 : 1),
                        line.holder(u + sg.units - 1));
}

// On the diagonal of a causal call a weight of 0 must not meet a NaN of V that only later rows of the tile
// see.  Entries in tiles of `TILE` that not all rows see alike therefore count as 0 in the products where
// their group of V is NaN; a CTA that met one runs this when it is done (all its threads, its stores made
// visible to each other): the rows that do see such an entry get their NaN.  It stands at the end,
// out of the way: the same look-up at the end of each segment cost every call 1 to 9 %.  Here causal
// pieces of 256 channels take 44.4 us (43.8 without), of 192 41.4 (40.9), blocks of 32 tokens 18.5 (18.3),
// other calls the same.
template <int D, int ROWS, int TILE, bool kRowsTogether>
__device__ __forceinline__ void put_nans(const AttnParams& p, const AttnPlan& f, Segment<ROWS> sg, int u0,
                                         int u1) {
  constexpr int GROUPS = D / 32;
#pragma unroll 1
  for (int u = u0; u < u1;) {
    const int piece = min(sg.units - sg.k0, u1 - u), r0 = sg.rt * ROWS;
    const int from = max(sg.k0 << f.unit_log2, max(rows_see(p, sg.len, r0), 0) & ~(TILE - 1));
    const int end = min(sg.seen, (sg.k0 + piece) << f.unit_log2);
    const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (u == u0 ? 0 : 1);
#pragma unroll 1
    for (int x = threadIdx.x; x < ROWS * GROUPS; x += blockDim.x) {
      const int row = x / GROUPS, g = x - row * GROUPS, r = r0 + row;
      if (r >= p.n * p.G) break;
      const int to = min(end, rows_see(p, sg.len, r));
      bool nan = false;
#pragma unroll 1
      for (int e = from; e < to && !nan; ++e) {
        if (p.key_mask && __ldg(p.key_mask + sg.b * p.mask_stride + e) == 0) continue;
        const int word = e / p.page_size;
        const int page = __ldg(p.table + static_cast<int64_t>(sg.b) * p.table_stride + word);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) continue;
        const int64_t at = (static_cast<int64_t>(page) * p.heads + sg.h) * p.page_size + e - word * p.page_size;
        nan = kv4_nan(__ldg(p.v_params + at * GROUPS + g));
      }
      if (!nan) continue;
      const int i = token_of(p, r), hq = sg.h * p.G + r - i * p.G;
      uint16_t* out = p.out + sg.b * p.ob + i * p.ot + hq * p.oh + g * 32;
#pragma unroll 1
      for (int c = g * 32; c < g * 32 + 32; ++c) {
        if (piece == sg.units)
          *out++ = 0x7FFFu;
        else if (kRowsTogether)  // the layout of attention_tc.cu
          f.part_o[((part * (D / 4) + c / 4) * ROWS + row) * 4 + c % 4] = NAN;
        else
          f.part_o[(part * ROWS + row) * D + c] = NAN;
      }
    }
    u += piece;
    if (u < u1) sg.next(p, f);
  }
}

__device__ __forceinline__ void store_joined(const AttnParams& p, int b, int h, int r, int ch, float2 a,
                                             float inv) {
  const int i = token_of(p, r), hq = h * p.G + r - i * p.G;
  const uint32_t w = bf2_pack(a.x * inv, a.y * inv);
  uint16_t* dst = p.out + b * p.ob + i * p.ot + hq * p.oh + ch;
  dst[0] = static_cast<uint16_t>(w);
  dst[1] = static_cast<uint16_t>(w >> 16);
}
__device__ __forceinline__ void store_lse(const AttnParams& p, int b, int h, int r, float m, float sum) {
  const int i = token_of(p, r), hq = h * p.G + r - i * p.G;
  if (p.lse)
    p.lse[(static_cast<int64_t>(b) * p.heads * p.G + hq) * p.n + i] =
        sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// Join the parts of the segments that several CTAs share, in order of their entries:
//   out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.
// A CTA per row; each of its WARPS warps takes every WARPS-th part.
template <int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
    attention_join_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPlan f) {
  constexpr int V = D / 64, kThreadsJ = 32 * WARPS;
  __shared__ float2 acc_s[WARPS][D / 2];
  __shared__ float sum_s[WARPS], max_s[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int64_t seg = blockIdx.x;
  const int r = blockIdx.y;
  const int2 info = f.parts[seg];
  if (info.x < 0) return;
  const int h = static_cast<int>(seg % p.heads), item = static_cast<int>(seg / p.heads);
  const int b = item / f.row_tiles, rt = item - b * f.row_tiles;
  const int c0 = info.x >> 1, count = info.y - c0 + 1;
  auto part_of = [&](int k) { return static_cast<int64_t>(k == 0 ? info.x : 2 * (c0 + k)) * ROWS; };
  if (rt * ROWS + r >= p.n * p.G) return;
  float mx = -INFINITY;
  for (int k = threadIdx.x; k < count; k += kThreadsJ) mx = fmaxf(mx, f.part_ml[part_of(k) + r].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  if (lane == 0) max_s[warp] = mx;
  __syncthreads();
  mx = max_s[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, max_s[w]);
  float2 acc[V] = {};
  float sum = 0.f;
  // kAhead parts of the warp at a time, all their loads before the first use
  constexpr int kAhead = 4;
  for (int k0 = warp; k0 < count; k0 += kAhead * WARPS) {
    float2 v[kAhead], o[kAhead][V];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int k = k0 + y * WARPS;
      const int64_t part = part_of(k < count ? k : 0) + r;
      v[y] = k < count ? f.part_ml[part] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int x = 0; x < V; ++x)
        o[y][x] = k < count ? *reinterpret_cast<const float2*>(f.part_o + part * D + 64 * x + 2 * lane)
                            : make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const float keep = v[y].x == -INFINITY ? 0.f : ex2(v[y].x - mx);
      sum = fmaf(v[y].y, keep, sum);
#pragma unroll
      for (int x = 0; x < V; ++x) {
        acc[x].x = fmaf(o[y][x].x, keep, acc[x].x);
        acc[x].y = fmaf(o[y][x].y, keep, acc[x].y);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < V; ++x) acc_s[warp][32 * x + lane] = acc[x];
  if (lane == 0) sum_s[warp] = sum;
  __syncthreads();
  sum = sum_s[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) sum += sum_s[w];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int e = threadIdx.x; e < D / 2; e += kThreadsJ) {
    float2 a = acc_s[0][e];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      a.x += acc_s[w][e].x;
      a.y += acc_s[w][e].y;
    }
    store_joined(p, b, h, rt * ROWS + r, 2 * e, a, inv);
  }
  if (threadIdx.x == 0) store_lse(p, b, h, rt * ROWS + r, mx, sum);
}

// Sixteen warps where a segment is cut into more than 16 parts (152 parts a row: attention and join
// 21 us, 29 with four warps), else four (fewer than 16 parts would leave warps idle).
template <int D, int ROWS>
cudaError_t launch_join(const AttnParams& p, const AttnPlan& f, cudaStream_t stream) {
  const int64_t segments = static_cast<int64_t>(p.B) * f.row_tiles * p.heads;
  const dim3 blocks(static_cast<unsigned>(segments), ROWS);  // up to 2^30 segments
  if (f.ctas > 16 * segments)
    return launch_dependent(attention_join_kernel<D, ROWS, 16>, blocks, dim3(512), 0, stream, p, f);
  return launch_dependent(attention_join_kernel<D, ROWS, 4>, blocks, dim3(128), 0, stream, p, f);
}

}  // namespace
}  // namespace dllm

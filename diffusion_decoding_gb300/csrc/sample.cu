// One token per open row of a block, drawn from the row's filtered softmax (temperature, top-k,
// top-p, min-p) with a given uniform number, beside the row's statistics.
//
// Candidates are ordered by falling logit, lower ids first among equals; every filter keeps a prefix
// of that order (a "cut": the last candidate kept), so the tightest cut holds.  The draw walks the
// kept candidates by rising id.  All comparisons of masses are of exact integer sums
// (exp_fixed.cuh), so a row's token does not depend on how its work was split.
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "exp_fixed.cuh"
#include "internal.h"
#include "vec_math.cuh"

namespace dllm {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLaneVecs = 4;                // 16-byte vectors a lane takes of a tile
constexpr int kTileVecs = 32 * kLaneVecs;   // a tile: 2 KB of a row, one warp's
constexpr int kCap = 1024;                  // candidates that are sorted
// Histogram of weights: 32 bins an octave, down to where a weight is a unit.
constexpr int kBinsPerOctave = 32;
constexpr int kBins = kWeightBits * kBinsPerOctave;
constexpr int kBinsPerThread = (kBins + kThreads - 1) / kThreads;

struct SampleParams {
  const char* logits;
  int64_t row_stride_bytes;
  int V;
  const uint8_t* masked;   // null: every row
  const float* uniform;
  dllm_stats out;
  InvTemp t;
  double temperature;
  double log_min_p;        // -inf: no min-p
  double top_p;            // 1: no top-p
  int top_k;               // V: no top-k
};

// The last candidate kept: z above, or equal with an id up to this.
struct Cut {
  float z;
  int id;
};
__device__ __forceinline__ bool kept(const Cut& c, float z, int id) {
  return z > c.z || (z == c.z && id <= c.id);
}
__device__ __forceinline__ Cut tighter(const Cut& a, const Cut& b) {
  return a.z > b.z || (a.z == b.z && a.id < b.id) ? a : b;
}

// Rising order of the floats as integers (both zeros alike, as they compare).
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// What the first CTA of a row finds out and the others read.
struct Control {
  Cut cut;
  uint64_t mass;     // of the candidates up to the cut
  uint64_t before;   // mass of the bins before the one with the cut
  int count_before;
  int bin, bin_count;
  int listed;        // candidates in the list
  uint32_t lo, hi;   // bisection
  uint64_t above;    // mass (or count) from hi on
  int64_t ties;      // of the candidates equal to the cut's: how many are kept
  int found;         // token or id that locate() found
};

struct Shared {
  float2 pow2[32];
  Control ctl;
  float2 part[kWarps];      // (reference, sum) of a warp
  uint64_t warp_mass[kWarps];
  int warp_count[kWarps];
  float2 mine;              // (maximum, sum) of this CTA, read by the others
  uint64_t total[2];        // of this CTA: mass, count
  uint64_t bins_lo_hi[kBins];  // mass of a bin: low word, high word
  int bins[kBins];
  uint64_t keys[kCap];      // candidates: ~order(z) << 32 | id
};

// A row as whole vectors from the 16-byte boundary at or before its start.
template <int DT>
struct Row {
  static constexpr int VEC = DT == DLLM_BF16 ? 8 : 4, ES = DT == DLLM_BF16 ? 2 : 4;
  const char* base;  // on the boundary
  int skip;          // elements of the first vector before the row
  int V, vecs;

  __device__ __forceinline__ Row(const char* row, int v) {
    skip = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / ES;
    base = row - skip * ES;
    V = v;
    vecs = static_cast<int>((static_cast<int64_t>(V) + skip + VEC - 1) / VEC);
  }
  __device__ __forceinline__ int id(int vec) const { return vec * VEC - skip; }
  // Vector `vec`; elements outside the row (or vectors behind it) are -inf and not read.
  __device__ __forceinline__ uint4 load(int vec) const {
    const int e = id(vec);
    if (e >= 0 && e + VEC <= V) return ld_stream_v4(base + static_cast<int64_t>(vec) * 16);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == DLLM_BF16) {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(base) + static_cast<int64_t>(vec) * 8 + 2 * k;
        const uint32_t a = e + 2 * k >= 0 && e + 2 * k < V ? src[0] : 0xFF80u;
        const uint32_t b = e + 2 * k + 1 >= 0 && e + 2 * k + 1 < V ? src[1] : 0xFF80u;
        w[k] = a | b << 16;
      } else {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(base) + static_cast<int64_t>(vec) * 4 + k;
        w[k] = e + k >= 0 && e + k < V ? src[0] : 0xFF800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// One row, by the CTAs of a cluster (kCluster) or one CTA: each has a contiguous range of tiles.
template <int DT, bool kCluster>
struct Sampler {
  const SampleParams& p;
  Shared& s;
  Shared& first;    // of the cluster's first CTA
  uint64_t* sums;   // [tiles of a CTA]
  Row<DT> row;
  int rank, ranks;
  int tile0, tiles;
  float m;

  __device__ __forceinline__ Sampler(const SampleParams& p_, Shared& s_, Shared& f_, uint64_t* sums_,
                                     const char* r)
      : p(p_), s(s_), first(f_), sums(sums_), row(r, p_.V) {}

  __device__ __forceinline__ void sync() const {
    if constexpr (kCluster)
      cg::this_cluster().sync();
    else
      __syncthreads();
  }
  __device__ __forceinline__ Shared& of(int r) const {
    if constexpr (kCluster)
      return *cg::this_cluster().map_shared_rank(&s, r);
    else
      return s;
  }

  // f(z, id) of the elements of a tile, by one warp (every lane calls it as often; elements outside
  // the row come as -inf with an id outside [0, V)).
  template <typename F>
  __device__ __forceinline__ void each_of_tile(int tile, F f) const {
    uint4 q[kLaneVecs];
    const int v0 = tile * kTileVecs + (threadIdx.x & 31);
#pragma unroll
    for (int u = 0; u < kLaneVecs; ++u) q[u] = row.load(v0 + 32 * u);
#pragma unroll
    for (int u = 0; u < kLaneVecs; ++u) {
      float x[Row<DT>::VEC];
      unpack_vec<DT>(q[u], x);
#pragma unroll
      for (int j = 0; j < Row<DT>::VEC; ++j) f(x[j], row.id(v0 + 32 * u) + j);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int t = threadIdx.x >> 5; t < tiles; t += kWarps) each_of_tile(tile0 + t, f);
  }

  __device__ __forceinline__ uint64_t weight(float z) const { return weight_fixed(z, m, p.t, s.pow2); }
  // Bin of z, or one beyond kBins.
  __device__ __forceinline__ int bin_of(float z) const {
    const float y = octaves_below(z, m, p.t) * kBinsPerOctave;
    return y < kBins ? static_cast<int>(y) : INT_MAX;  // (NaN: INT_MAX)
  }

  // Maximum and log-sum-exp of the row (the same in every thread of the row).
  __device__ __forceinline__ float statistics() {
    const int warp = threadIdx.x >> 5;
    float ref = -INFINITY, sum = 0.f;
    for (int t = warp; t < tiles; t += kWarps) {
      uint4 q[kLaneVecs];
      const int v0 = (tile0 + t) * kTileVecs + (threadIdx.x & 31);
#pragma unroll
      for (int u = 0; u < kLaneVecs; ++u) q[u] = row.load(v0 + 32 * u);
      float top = vec_max<DT>(q[0]);
#pragma unroll
      for (int u = 1; u < kLaneVecs; ++u) top = fmaxf(top, vec_max<DT>(q[u]));
      top = warp_max(top);
      if (top > ref) {
        sum *= ex2((ref - top) * kLog2e);  // from nothing: 0 * 2^-inf
        ref = top;
      }
      if (ref == -INFINITY) continue;
#pragma unroll
      for (int u = 0; u < kLaneVecs; ++u) {
        float x[Row<DT>::VEC];
        unpack_vec<DT>(q[u], x);
#pragma unroll
        for (int j = 0; j < Row<DT>::VEC; ++j) sum += ex2((x[j] - ref) * kLog2e);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if ((threadIdx.x & 31) == 0) s.part[warp] = make_float2(ref, sum);
    __syncthreads();
    float2 all = joined(kWarps, [&](int w) { return s.part[w]; });
    if constexpr (kCluster) {
      if (threadIdx.x == 0) s.mine = all;
      sync();
      all = joined(ranks, [&](int r) { return of(r).mine; });
    }
    m = all.x;
    return m == -INFINITY ? -INFINITY : m + logf(all.y);
  }
  template <typename F>
  __device__ __forceinline__ float2 joined(int n, F get) const {
    float2 a = make_float2(-INFINITY, 0.f);
    for (int k = 0; k < n; ++k) a.x = fmaxf(a.x, get(k).x);
    if (a.x == -INFINITY) return a;
    for (int k = 0; k < n; ++k) {
      const float2 b = get(k);
      a.y += b.y * ex2((b.x - a.x) * kLog2e);
    }
    return a;
  }

  // The id at which the running sum of f(z, id) by rising id first exceeds target(total); -1 if it
  // never does.
  template <typename F, typename G>
  __device__ __forceinline__ int locate(F f, G target_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < tiles; t += kWarps) {
      uint64_t sum = 0;
      each_of_tile(tile0 + t, [&](float z, int id) { sum += f(z, id); });
      sum = warp_sum(sum);
      if (lane == 0) sums[t] = sum;
    }
    if (threadIdx.x == 0 && rank == 0) s.ctl.found = -1;
    __syncthreads();
    if (warp == 0) {
      uint64_t sum = 0;
      for (int t = lane; t < tiles; t += 32) sum += sums[t];
      sum = warp_sum(sum);
      if (lane == 0) s.total[0] = sum;
    }
    sync();
    uint64_t before = 0, all = 0;
    for (int r = 0; r < ranks; ++r) {
      const uint64_t x = of(r).total[0];
      if (r < rank) before += x;
      all += x;
    }
    const double target = target_of(all);
    if (warp == 0 && !(static_cast<double>(before) > target) &&
        static_cast<double>(before + s.total[0]) > target) {
      int tile = 0;
      for (int t0 = 0; t0 < tiles; t0 += 32) {
        const uint64_t x = t0 + lane < tiles ? sums[t0 + lane] : 0;
        const uint64_t upto = before + warp_scan(x);
        const unsigned hit = __ballot_sync(kFull, static_cast<double>(upto) > target);
        if (hit) {
          const int l = __ffs(hit) - 1;
          tile = t0 + l;
          before = __shfl_sync(kFull, upto - x, l);
          break;
        }
        before = __shfl_sync(kFull, upto, 31);
      }
      for (int u = 0; u < kLaneVecs; ++u) {
        const int vec = (tile0 + tile) * kTileVecs + 32 * u + lane;
        float x[Row<DT>::VEC];
        unpack_vec<DT>(row.load(vec), x);
        uint64_t sum = 0;
#pragma unroll
        for (int j = 0; j < Row<DT>::VEC; ++j) sum += f(x[j], row.id(vec) + j);
        uint64_t upto = before + warp_scan(sum);
        const unsigned hit = __ballot_sync(kFull, static_cast<double>(upto) > target);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            upto -= sum;
            int id = -1;
#pragma unroll
            for (int j = 0; j < Row<DT>::VEC; ++j) {
              upto += f(x[j], row.id(vec) + j);
              if (id < 0 && static_cast<double>(upto) > target) id = row.id(vec) + j;
            }
            first.ctl.found = id;
          }
          break;
        }
        before = __shfl_sync(kFull, upto, 31);
      }
    }
    sync();
    const int id = first.ctl.found;
    sync();
    return id;
  }

  // ---- the histogram of weights

  __device__ __forceinline__ uint32_t* bin_words(int b) {
    return reinterpret_cast<uint32_t*>(&s.bins_lo_hi[b]);
  }
  __device__ __forceinline__ void histogram() {
    for (int b = threadIdx.x; b < kBins; b += kThreads) s.bins_lo_hi[b] = 0, s.bins[b] = 0;
    __syncthreads();
    each([&](float z, int) {
      const int b = bin_of(z);
      if (b >= kBins) return;
      const uint64_t w = weight(z);
      uint32_t* words = bin_words(b);
      const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(words, lo);
      const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
      if (hi) atomicAdd(words + 1, hi);
      atomicAdd(&s.bins[b], 1);
    });
    sync();
    if (rank == 0 && ranks > 1) {
      for (int b = threadIdx.x; b < kBins; b += kThreads) {
        for (int r = 1; r < ranks; ++r) {
          const Shared& o = of(r);
          s.bins_lo_hi[b] += o.bins_lo_hi[b];
          s.bins[b] += o.bins[b];
        }
      }
    }
    __syncthreads();
  }
  // Exclusive sums over the block of one value a thread; ends synchronised.
  __device__ __forceinline__ void block_scan(uint64_t& mass, int& count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t mi = warp_scan(mass);
    const int ci = warp_scan(count);
    if (lane == 31) s.warp_mass[warp] = mi, s.warp_count[warp] = ci;
    __syncthreads();
    mass = mi - mass;
    count = ci - count;
    for (int w = 0; w < warp; ++w) mass += s.warp_mass[w], count += s.warp_count[w];
    __syncthreads();
  }
  // Does a prefix of this count and mass reach the goal (k candidates, or the mass x)?
  struct Goal {
    bool by_mass;
    int k;
    double x;
    __device__ __forceinline__ bool reached(int64_t count, uint64_t mass) const {
      return by_mass ? static_cast<double>(mass) >= x : count >= k;
    }
  };

  // The shortest prefix that reaches `goal`; its cut and mass are in first.ctl afterwards.  The whole
  // prefix of weights above 0 where that does not reach it.
  __device__ __forceinline__ void find_cut(const Goal& goal) {
    if (rank == 0) {
      uint64_t mass = 0;
      int count = 0;
      const int b0 = threadIdx.x * kBinsPerThread;
      for (int b = b0; b < min(b0 + kBinsPerThread, kBins); ++b) mass += s.bins_lo_hi[b], count += s.bins[b];
      if (threadIdx.x == 0) s.ctl.bin = -1, s.ctl.listed = 0;
      block_scan(mass, count);
      for (int b = b0; b < min(b0 + kBinsPerThread, kBins); ++b) {
        const uint64_t mass1 = mass + s.bins_lo_hi[b];
        const int count1 = count + s.bins[b];
        if (!goal.reached(count, mass) && goal.reached(count1, mass1)) {
          s.ctl.bin = b;
          s.ctl.bin_count = s.bins[b];
          s.ctl.before = mass;
          s.ctl.count_before = count;
        }
        mass = mass1;
        count = count1;
      }
      if (threadIdx.x == kThreads - 1) {
        s.total[1] = mass;
      }
      __syncthreads();
      if (threadIdx.x == 0 && s.ctl.bin < 0) {
        s.ctl.cut = Cut{-INFINITY, INT_MAX};
        s.ctl.mass = s.total[1];
      }
    }
    sync();
    const int bin = first.ctl.bin, in_bin = first.ctl.bin_count;
    if (bin < 0) {
      sync();
      return;
    }
    if (in_bin <= kCap) {
      each([&](float z, int id) {
        if (bin_of(z) == bin) append(z, id);
      });
      sync();
      if (rank == 0) cut_in_list(goal);
      sync();
    } else {
      cut_in_bin(goal, bin);
    }
  }
  __device__ __forceinline__ void append(float z, int id) {
    const int at = atomicAdd(&first.ctl.listed, 1);
    if (at < kCap) first.keys[at] = static_cast<uint64_t>(~order_of(z)) << 32 | static_cast<uint32_t>(id);
  }
  // Sort keys[0, n) rising (n <= kCap; the rest up to a power of two is filled up).
  __device__ __forceinline__ void sort_list(int n) {
    int size = 2;
    while (size < n) size *= 2;
    for (int k = n + threadIdx.x; k < size; k += kThreads) s.keys[k] = ~uint64_t{0};
    __syncthreads();
    for (int len = 2; len <= size; len *= 2) {
      for (int d = len / 2; d > 0; d /= 2) {
        for (int k = threadIdx.x; k < size / 2; k += kThreads) {
          const int i = 2 * d * (k / d) + k % d, j = i + d;
          const uint64_t a = s.keys[i], b = s.keys[j];
          if ((a > b) == ((i & len) == 0)) s.keys[i] = b, s.keys[j] = a;
        }
        __syncthreads();
      }
    }
  }
  __device__ __forceinline__ float listed_z(int k) const {
    return of_order(~static_cast<uint32_t>(s.keys[k] >> 32));
  }
  __device__ __forceinline__ int listed_id(int k) const { return static_cast<int>(s.keys[k] & 0xFFFFFFFFu); }

  // First CTA: the cut among the listed candidates, behind ctl.before and ctl.count_before.
  __device__ __forceinline__ void cut_in_list(const Goal& goal) {
    constexpr int kEach = kCap / kThreads;
    const int n = min(s.ctl.listed, kCap);
    sort_list(n);
    uint64_t w[kEach], mass = 0;
    int count = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int at = threadIdx.x * kEach + k;
      w[k] = at < n ? weight(listed_z(at)) : 0;
      mass += w[k];
      count += at < n ? 1 : 0;
    }
    block_scan(mass, count);
    mass += s.ctl.before;
    count += s.ctl.count_before;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int at = threadIdx.x * kEach + k;
      const bool was = goal.reached(count, mass);
      if (at < n) mass += w[k], ++count;
      if (at < n && !was && goal.reached(count, mass)) {
        s.ctl.cut = Cut{listed_z(at), listed_id(at)};
        s.ctl.mass = mass;
      }
    }
    __syncthreads();
  }

  // The cut inside a bin of more candidates than are sorted: the value by bisection, then how many of
  // the candidates with that value.
  __device__ __noinline__ void cut_in_bin(const Goal& goal, int bin) {
    // reached from lo on, not from hi on
    uint32_t lo = 0u, hi = 0xFFFFFFFFu;
    const uint64_t before = first.ctl.before;
    const int64_t count_before = first.ctl.count_before;
    uint64_t above = 0;
    int64_t count_above = 0;
    while (hi - lo > 1u) {
      const uint32_t mid = lo + (hi - lo) / 2;
      uint64_t mass = 0;
      uint64_t count = 0;
      each([&](float z, int) {
        if (bin_of(z) == bin && order_of(z) >= mid) mass += weight(z), ++count;
      });
      sum_of_row(mass, count);
      if (goal.reached(count_before + static_cast<int64_t>(count), before + mass)) {
        lo = mid;
      } else {
        hi = mid;
        above = mass;
        count_above = static_cast<int64_t>(count);
      }
    }
    const float z = of_order(lo);
    const uint64_t w = weight(z), base = before + above;
    int64_t ties = goal.k - (count_before + count_above);
    if (goal.by_mass) {
      ties = static_cast<int64_t>((goal.x - static_cast<double>(base)) / static_cast<double>(w));
      while (ties > 1 && goal.reached(0, base + (ties - 1) * w)) --ties;
      while (!goal.reached(0, base + ties * w)) ++ties;
    }
    const int id = locate([&](float x, int) { return x == z ? uint64_t{1} : uint64_t{0}; },
                          [&](uint64_t) { return static_cast<double>(ties - 1); });
    if (threadIdx.x == 0 && rank == 0) {
      s.ctl.cut = Cut{z, id};
      s.ctl.mass = base + ties * w;
    }
    sync();
  }
  // Sums over all threads of the row, in every thread.
  __device__ __forceinline__ void sum_of_row(uint64_t& a, uint64_t& b) {
    const int warp = threadIdx.x >> 5;
    int none = 0;
    a = warp_sum(a);
    b = warp_sum(b);
    (void)none;
    sync();  // the totals of the last call have been read
    if ((threadIdx.x & 31) == 0) s.warp_mass[warp] = a, s.warp_count[warp] = static_cast<int>(b);
    __syncthreads();
    if (threadIdx.x == 0) {
      uint64_t x = 0, y = 0;
      for (int w = 0; w < kWarps; ++w) x += s.warp_mass[w], y += s.warp_count[w];
      s.total[0] = x;
      s.total[1] = y;
    }
    sync();
    a = b = 0;
    for (int r = 0; r < ranks; ++r) a += of(r).total[0], b += of(r).total[1];
  }

  // The token: cuts by the filters, then the draw.
  __device__ __forceinline__ int draw(float u) {
    Cut cut{-INFINITY, INT_MAX};
    const bool by_k = p.top_k < p.V, by_p = p.top_p < 1.0;
    if (by_k || by_p) {
      histogram();
      if (by_k) {
        find_cut(Goal{false, p.top_k, 0.0});
        cut = first.ctl.cut;
      }
      if (by_p) {
        uint64_t all = first.ctl.mass;
        if (!by_k) {
          if (rank == 0) {
            uint64_t mass = 0;
            int none = 0;
            const int b0 = threadIdx.x * kBinsPerThread;
            for (int b = b0; b < min(b0 + kBinsPerThread, kBins); ++b) mass += s.bins_lo_hi[b];
            const uint64_t own = mass;
            block_scan(mass, none);
            if (threadIdx.x == kThreads - 1) s.ctl.mass = mass + own;
          }
          sync();
          all = first.ctl.mass;
        }
        sync();
        find_cut(Goal{true, 0, p.top_p * static_cast<double>(all)});
        cut = tighter(cut, first.ctl.cut);
        sync();
      }
    }
    if (p.log_min_p > -INFINITY) {
      const double least = static_cast<double>(m) + p.temperature * p.log_min_p;
      cut = tighter(cut, Cut{__double2float_ru(least), INT_MAX});
    }
    return locate([&](float z, int id) { return kept(cut, z, id) ? weight(z) : 0; },
                  [&](uint64_t all) { return static_cast<double>(u) * static_cast<double>(all); });
  }
};

template <int DT, bool kCluster>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  const int ranks = kCluster ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
  const int rank = kCluster ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int64_t r = blockIdx.x / ranks;
  if (p.masked && p.masked[r] == 0) {
    if (rank == 0 && threadIdx.x == 0) {
      p.out.row_max[r] = p.out.lse[r] = -INFINITY;
      p.out.conf[r] = 0.f;
      p.out.argmax[r] = -1;
    }
    return;
  }
  if (threadIdx.x < 32) s.pow2[threadIdx.x] = kPow2Table[threadIdx.x];
  Shared* first = &s;
  if constexpr (kCluster) first = cg::this_cluster().map_shared_rank(&s, 0);
  const char* logits = p.logits + r * p.row_stride_bytes;
  Sampler<DT, kCluster> x(p, s, *first, reinterpret_cast<uint64_t*>(dyn + sizeof(Shared)), logits);
  x.rank = rank;
  x.ranks = ranks;
  const int tiles = (x.row.vecs + kTileVecs - 1) / kTileVecs;
  x.tile0 = static_cast<int>(static_cast<int64_t>(tiles) * rank / ranks);
  x.tiles = static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / ranks) - x.tile0;
  const float lse = x.statistics();
  int token = -1;
  if (x.m > -INFINITY) {
    const float u = fminf(fmaxf(p.uniform[r], 0.f), 0x1.fffffep-1f);
    token = x.draw(u);
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.out.row_max[r] = x.m;
    p.out.lse[r] = lse;
    p.out.argmax[r] = token;
    p.out.conf[r] = token < 0 ? 0.f : ex2((load_logit(logits, DT, token) - lse) * kLog2e);
  }
  if constexpr (kCluster) x.sync();  // nobody leaves while its shared memory may be read
}

template <int DT, bool kCluster>
cudaError_t launch(const SampleParams& p, int64_t rows, int ranks, size_t smem, cudaStream_t stream) {
  cudaError_t e = allow_smem<sample_kernel<DT, kCluster>>(200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, sample_kernel<DT, kCluster>, p);
}

}  // namespace

cudaError_t launch_sample(const void* logits, const dllm_shape& sh, const uint8_t* masked,
                          const float* uniform, const dllm_sampling& how, const dllm_stats& out,
                          int sm_count, cudaStream_t stream) {
  const int es = sh.dtype == DLLM_BF16 ? 2 : 4;
  SampleParams p{};
  p.logits = static_cast<const char*>(logits);
  p.row_stride_bytes = sh.row_stride * es;
  p.V = sh.V;
  p.masked = masked;
  p.uniform = uniform;
  p.out = out;
  // temperature 0: the most probable token, as the only candidate
  const bool greedy = how.temperature == 0.f;
  p.temperature = greedy ? 1.0 : static_cast<double>(how.temperature);
  const double inv = 1.4426950408889634074 / p.temperature;
  p.t.hi = static_cast<float>(inv);
  p.t.lo = static_cast<float>(inv - static_cast<double>(p.t.hi));
  p.top_k = greedy ? 1 : how.top_k > 0 && how.top_k < sh.V ? how.top_k : sh.V;
  p.top_p = greedy ? 1.0 : static_cast<double>(how.top_p);
  p.log_min_p = !greedy && how.min_p > 0.f ? log(static_cast<double>(how.min_p)) : -INFINITY;
  const int64_t rows = static_cast<int64_t>(sh.B) * sh.L;
  const int64_t tiles = (static_cast<int64_t>(sh.V) * es + 2047) / 2048 + 1;
  int ranks = 1;
  while (ranks < 8 && rows * ranks * 2 <= 4 * static_cast<int64_t>(sm_count) &&
         tiles >= 2 * ranks * kWarps)
    ranks *= 2;
  const size_t smem = sizeof(Shared) + static_cast<size_t>((tiles + ranks - 1) / ranks + 1) * 8;
  if (sh.dtype == DLLM_BF16)
    return ranks > 1 ? launch<DLLM_BF16, true>(p, rows, ranks, smem, stream)
                     : launch<DLLM_BF16, false>(p, rows, ranks, smem, stream);
  return ranks > 1 ? launch<DLLM_F32, true>(p, rows, ranks, smem, stream)
                   : launch<DLLM_F32, false>(p, rows, ranks, smem, stream);
}

}  // namespace dllm

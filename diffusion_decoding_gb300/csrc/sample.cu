// One token per open row of a block, drawn from the row's filtered softmax (temperature, top-k,
// top-p, min-p) with a given uniform number, beside the row's statistics.
//
// Candidates are ordered by falling logit, lower ids first among equals; every filter keeps a prefix
// of that order (a "cut": the last candidate kept), so the tightest cut holds.  The draw walks the
// kept candidates by rising id.  All comparisons of masses are of exact integer sums
// (exp_fixed.cuh), so a row's token does not depend on how its work was split.
//
// sample_kernel reads a row once, a CTA a row or, where that leaves SMs idle, a cluster of up to eight:
// maximum, sum of exponentials, and the maximum and the sum of weights (32 bits) of every chunk (what a
// lane has of a 4 KB tile).  Those say from which logit on the filters keep something; the candidates from
// there on are listed, weighed exactly and ordered (the sum of all weights, which top_p needs, is known
// to 2^-18 of what its chunks hold, and the row is settled where that error changes nothing; chunks that
// weigh much are summed up exactly for a second try).  Without a filter the sums of chunks lead to the
// token in the same way, and the second try walks the tiles that hold it by exact weights.  What stays
// open, or has more candidates than the list holds, goes through exact passes over all weights:
// sample_rest_kernel, a cluster a row (or, in clusters and with top_k, at once: in_full).
//
// The one pass takes its time for special-function operations, one exponential an element at temperature 1 and
// two at another, and for loads in flight: 64 KB of them a CTA's turn at four CTAs an SM.  1024 rows of
// 126464 bf16 logits in a captured graph: 59 us with top_k 50, 57 drawn from the whole distribution at 0.7
// (77 to 84 with a few rows left open), 67 with top_p 0.9 there: 4.5 and 3.9 TB/s; fp32 119 to 122 us
// (4.4 TB/s).  Neither DRAM nor the special-function pipe is full (36 to 45 and 24 to 51 % of an ncu run).  A
// single row 8 to 13 us: launch, barriers and first fetches of code.  Clusters where the rows fill the GPU
// anyway cost more than they even out (640 rows: 2 CTAs a row 56 to 70 us, one 48 to 55).
#include <algorithm>
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
constexpr int kLaneVecs = 8, kLaneVecsLog2 = 3;  // 16-byte vectors a lane takes of a tile
constexpr int kTileVecs = 32 * kLaneVecs;   // a tile: 4 KB of a row, one warp's
constexpr int kCap = 2048;                  // candidates that are listed and ordered, at most
constexpr int kFew = 128;                   // candidates ordered by counting, more by sorting
constexpr int kMaxGroups = 256;             // chunks of a CTA / 32
constexpr int kMaxRanks = 8;                // CTAs of a row
// Histogram of chunk maxima: 8 bins an octave.
constexpr int kCoarse = 8, kCoarseBins = kWeightBits * kCoarse;
// Histogram of weights: 32 bins an octave, down to where a weight is a unit.
constexpr int kBinsPerOctave = 32;
constexpr int kBins = kWeightBits * kBinsPerOctave;
constexpr int kBinsPerThread = (kBins + kThreads - 1) / kThreads;

struct SampleParams {
  const char* logits;
  int64_t row_stride_bytes;
  int V;
  int span_log2;           // tiles of a group
  uint32_t sums_at, keys_at;  // in shared memory
  int cap;                 // candidates that are listed, a power of two
  bool at_once;            // no row is left to sample_rest_kernel
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

// What a CTA tells the others of its part of the row.
struct Summary {
  float m, sum;      // maximum, sum of exp(z - m)
  float some, all;   // logits that its share of top_k, and all of top_k, of its chunks reach
  uint64_t mass;     // weights
  uint64_t light;    // of that: by sums of chunks in 32 bits
};

struct Shared {
  float2 pow2[32];
  Control ctl;
  float2 part[kWarps];      // (reference, sum) of a warp
  uint64_t warp_mass[kWarps], warp_light[kWarps];
  int warp_count[kWarps];
  Summary mine;             // read by the others
  uint64_t total[2];        // of this CTA: mass, count; read by the others
  uint64_t group_before;    // find_group's
  int group;
  int coarse[kCoarseBins];  // of this CTA's part
  int row_coarse[kCoarseBins];
  ulonglong2 few[kFew];     // key, weight
  int queued;
  uint64_t goal, goal_error;  // what one thread worked out for all: a mass in units
  float least, from;
  bool sure;
};
// The histogram of all weights, where the chunks' maxima and sums were.
struct Fine {
  uint64_t bins_lo_hi[kBins];  // mass of a bin: low word, high word
  int bins[kBins];
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
  __device__ __forceinline__ float at(int i) const { return load_logit(base + skip * ES, DT, i); }
  __device__ __forceinline__ uint4 whole(int vec) const {  // neither the first nor the last
    return ld_stream_v4(base + static_cast<int64_t>(vec) * 16);
  }
  // Vector `vec`; elements outside the row (or vectors behind it) are -inf and not read.
  __device__ __forceinline__ uint4 load(int vec) const {
    const int e = id(vec);
    if (e >= 0 && e + VEC <= V) return ld_stream_v4(base + static_cast<int64_t>(vec) * 16);
    return e < V ? load_edge(base, vec, e, V) : none();
  }
  static __device__ __forceinline__ uint4 none() {
    constexpr uint32_t x = DT == DLLM_BF16 ? 0xFF80FF80u : 0xFF800000u;
    return make_uint4(x, x, x, x);
  }
  // (a function of its own: eight of it in a row take longer to fetch than to run)
  static __device__ __noinline__ uint4 load_edge(const char* base, int vec, int e, int V) {
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
  // The first two elements of q, which go from it.
  static __device__ __forceinline__ void take2(uint4& q, float& a, float& b) {
    if constexpr (DT == DLLM_BF16) {
      a = bf16lo(q.x), b = bf16hi(q.x);
      q.x = q.y, q.y = q.z, q.z = q.w;
    } else {
      a = __uint_as_float(q.x), b = __uint_as_float(q.y);
      q.x = q.z, q.y = q.w;
    }
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

// Bitonic sort of kThreads * E keys, E a thread, rising: neighbours in a thread's registers, then lanes of
// a warp by shuffles, then warps through `keys`.  (A row of 1500 with top_k 900, two sorts: 26 us; with
// every step through shared memory 63.)
template <int E>
__device__ __noinline__ void sort_block(uint64_t* keys, int n) {
  const int t = threadIdx.x;
  uint64_t k[E];
#pragma unroll
  for (int e = 0; e < E; ++e) k[e] = t * E + e < n ? keys[t * E + e] : ~uint64_t{0};
#pragma unroll 1
  for (int len = 2; len <= kThreads * E; len *= 2) {
#pragma unroll 1
    for (int d = len / 2; d >= E; d /= 2) {
      const int far = d / E;  // threads apart
      // the lower of a pair keeps the smaller key in a rising run (E <= d < len: a thread's run is one)
      const bool small = ((t & far) == 0) == ((t * E & len) == 0);
      if (far < 32) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint64_t o = __shfl_xor_sync(kFull, k[e], far);
          k[e] = (o < k[e]) == small ? o : k[e];
        }
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) keys[e * kThreads + t] = k[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint64_t o = keys[e * kThreads + (t ^ far)];
          k[e] = (o < k[e]) == small ? o : k[e];
        }
      }
    }
#pragma unroll
    for (int d = E / 2; d > 0; d /= 2) {
      if (d >= len) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e & d) continue;
        const uint64_t x = k[e], y = k[e | d];
        if ((x > y) == (((t * E + e) & len) == 0)) k[e] = y, k[e | d] = x;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) keys[t * E + e] = k[e];
  __syncthreads();
}
// Sort keys[0, n), n <= kCap; behind them come the largest ones.
__device__ __forceinline__ void sort_keys(uint64_t* keys, int n) {
  static_assert(kCap == 8 * kThreads, "");
  if (n <= kThreads)
    sort_block<1>(keys, n);
  else if (n <= 2 * kThreads)
    sort_block<2>(keys, n);
  else if (n <= 4 * kThreads)
    sort_block<4>(keys, n);
  else
    sort_block<8>(keys, n);
}

// One row, by the CTAs of a cluster (kCluster) or one CTA: each has a contiguous range of tiles.
template <int DT, bool kCluster>
struct Sampler {
  const SampleParams& p;
  Shared& s;
  Shared& first;    // of the cluster's first CTA
  Fine& fine;
  uint64_t* sums;   // of groups of tiles, or of strips; behind fine
  float* tops;      // [groups * 32] maximum of a chunk
  float* masses;    // [groups * 32] weights of a chunk, to the reference refs[group]
  float* refs;      // [groups]
  uint64_t* keys;   // [cap] candidates: ~order(z) << 32 | id
  uint64_t* first_keys;  // the first CTA's
  uint16_t* queue;  // [cap] chunks that are looked through again
  Row<DT> row;
  int rank, ranks;
  int tile0, tiles, groups;
  int strips_log2;  // strips that are summed up together
  float m, total;   // of the row: maximum, sum of exp(z - m)
  float highest;    // of this thread's elements

  __device__ __forceinline__ Sampler(const SampleParams& p_, Shared& s_, Shared& f_, Fine& fine_,
                                     const char* r)
      : p(p_), s(s_), first(f_), fine(fine_), row(r, p_.V) {}

  // Its part of the row, and of the shared memory.
  __device__ __forceinline__ void place(uint8_t* dyn, int rank_, int ranks_) {
    rank = rank_;
    ranks = ranks_;
    const int all = (row.vecs + kTileVecs - 1) / kTileVecs;
    tile0 = static_cast<int>(static_cast<int64_t>(all) * rank / ranks);
    tiles = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) / ranks) - tile0;
    groups = (tiles + (1 << p.span_log2) - 1) >> p.span_log2;
    // single strips where there are few (32 rows of 1500: 25 us, by whole tiles 34), else so many together
    // that every warp has four sums or more (200 rows of 120000: 100 us, by single strips 129)
    strips_log2 = 0;
    while ((2 << strips_log2) <= kLaneVecs && tiles * kLaneVecs >> strips_log2 >= 8 * kWarps) ++strips_log2;
    tops = reinterpret_cast<float*>(dyn + sizeof(Shared));
    masses = tops + groups * 32;
    refs = masses + groups * 32;
    sums = reinterpret_cast<uint64_t*>(dyn + p.sums_at);
    keys = reinterpret_cast<uint64_t*>(dyn + p.keys_at);
    queue = reinterpret_cast<uint16_t*>(keys + p.cap);
    first_keys = keys;
    if constexpr (kCluster) first_keys = cg::this_cluster().map_shared_rank(keys, 0);
  }
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

  // f(z, id) of the elements of this CTA's part, a strip (32 vectors) at a time, 2^strips_log2 in a row by
  // one warp; after(these strips' number) by every lane (elements outside the row come as -inf with an id
  // outside [0, V)).
  // (Two elements at a time: unrolled further, the code of an f of sixty instructions takes longer to
  // fetch than to run.)
  template <typename F, typename G>
  __device__ __forceinline__ void each(F f, G after) const {
    constexpr int kAhead = 3;  // vectors on their way
    const int warp = threadIdx.x >> 5, mask = (1 << strips_log2) - 1, strips = tiles * kLaneVecs;
    const int v0 = tile0 * kTileVecs + (threadIdx.x & 31);
    // the i-th strip of this warp
    auto strip_of = [&](int i) { return (warp + (i >> strips_log2) * kWarps) << strips_log2 | (i & mask); };
    auto fetch = [&](int strip, uint4& q) {
      const int vec = v0 + 32 * strip;
      if (strip >= strips) return;
      if (vec - (threadIdx.x & 31) > 0 && vec - (threadIdx.x & 31) + 32 < row.vecs)
        q = row.whole(vec);
      else
        q = row.load(vec);
    };
    uint4 next[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(strip_of(u), next[u]);
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int k = strip_of(i);
      if (k >= strips) break;
      uint4 q = next[0];
#pragma unroll
      for (int u = 0; u + 1 < kAhead; ++u) next[u] = next[u + 1];
      fetch(strip_of(i + kAhead), next[kAhead - 1]);
      int id = row.id(v0 + 32 * k);
#pragma unroll 1
      for (int j = 0; j < Row<DT>::VEC; j += 2, id += 2) {
        float a, b;
        Row<DT>::take2(q, a, b);
        f(a, id);
        f(b, id + 1);
      }
      if ((i & mask) == mask) after(k >> strips_log2);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each(f, [](int) {});
  }

  __device__ __forceinline__ uint64_t weight(float z) const { return weight_fixed(z, m, p.t, s.pow2); }
  // Bin of z, or one beyond kBins.
  __device__ __forceinline__ int bin_of(float z) const {
    const float y = octaves_below(z, m, p.t) * kBinsPerOctave;
    return y < kBins ? static_cast<int>(y) : INT_MAX;  // (NaN: INT_MAX)
  }

  // One pass over this CTA's part: the maximum and the sum of exp(z - m) of the row, the maximum of
  // every chunk (what a lane has of a group of tiles) and, with kMass, the sum of weights of every
  // chunk; with kOne the temperature is 1 and both sums are of the same terms.
  //
  // exp(z - ref) = 2^(z k - ref k): one fma and one special-function operation a term.  ref k is
  // rounded (hi), the rest goes into the factor 2^-rest that a chunk's sum is multiplied by once; a
  // term in 32 bits is then at most 2^-22 + |log2 of it| 2^-24 off.
  template <bool kMass, bool kOne>
  __device__ __forceinline__ void pass() {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float ref = -INFINITY, sum = 0.f;
    highest = -INFINITY;
    Scale one{kLog2e}, temp{p.t.hi};
    for (int g = warp; g < groups; g += kWarps) {
      float top = -INFINITY, mass = 0.f;
      const int t1 = min((g + 1) << p.span_log2, tiles);
      for (int t = g << p.span_log2; t < t1; ++t) {
        uint4 q[kLaneVecs];
        const int v0 = (tile0 + t) * kTileVecs + lane;
        if (v0 - lane > 0 && v0 - lane + kTileVecs < row.vecs) {
#pragma unroll
          for (int u = 0; u < kLaneVecs; ++u) q[u] = row.whole(v0 + 32 * u);
        } else {
#pragma unroll
          for (int u = 0; u < kLaneVecs; ++u) q[u] = row.load(v0 + 32 * u);
        }
        const float here = top_of(q);
        top = fmaxf(top, here);
        highest = fmaxf(highest, here);
        if (__any_sync(kFull, here > ref)) {
          const float up = fmaxf(ref, warp_max(here));
          sum *= ex2((ref - up) * kLog2e);  // from nothing: 0 * 2^-inf
          if (kMass) mass *= ex2((ref - up) * p.t.hi);
          ref = up;
          one.set(ref);
          if (kMass && !kOne) temp.set(ref);
        }
        if (ref == -INFINITY) continue;
        float a, b;
        if (one.far || (kMass && !kOne && temp.far))
          sums_far<kMass && !kOne>(q, ref, a, b);
        else
          sums_near<kMass && !kOne>(q, one, temp, a, b);
        sum += a;
        if (kMass) mass += kOne ? a : b;
      }
      tops[g * 32 + lane] = top;
      if (kMass) {
        masses[g * 32 + lane] = mass;
        if (lane == 0) refs[g] = ref;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) s.part[warp] = make_float2(ref, sum);
    __syncthreads();
    const float2 all = joined(kWarps, [&](int w) { return s.part[w]; });
    m = all.x;
    total = all.y;
  }
  // The largest of a lane's elements of a tile.
  static __device__ __forceinline__ float top_of(const uint4 (&q)[kLaneVecs]) {
    if constexpr (DT == DLLM_BF16) {
      uint32_t t = bf16x2_max(bf16x2_max(q[0].x, q[0].y), bf16x2_max(q[0].z, q[0].w));
#pragma unroll
      for (int u = 1; u < kLaneVecs; ++u)
        t = bf16x2_max(t, bf16x2_max(bf16x2_max(q[u].x, q[u].y), bf16x2_max(q[u].z, q[u].w)));
      return fmaxf(bf16lo(t), bf16hi(t));
    } else {
      float t = vec_max<DT>(q[0]);
#pragma unroll
      for (int u = 1; u < kLaneVecs; ++u) t = fmaxf(t, vec_max<DT>(q[u]));
      return t;
    }
  }
  // 2^(x k - ref k) is computed as 2^(x k - hi) * rest, which needs a ref k that hi misses by little: both
  // factors are within 2^(1/2) up to 2^24, and from 2^31 on one would be infinite and the other 0.
  struct Scale {
    float k, hi, rest;
    bool far;  // hi is no use
    __device__ __forceinline__ explicit Scale(float k_) : k(k_), hi(0.f), rest(1.f), far(false) {}
    __device__ __forceinline__ void set(float r) {
      hi = r * k;
      far = !(fabsf(hi) < 0x1p24f);
      rest = ex2(-fmaf(r, k, -hi));
    }
  };
  // The sums of a lane's elements of a tile, at temperature 1 and (kTwo) at the temperature.
  template <bool kTwo>
  static __device__ __forceinline__ void sums_near(const uint4 (&q)[kLaneVecs], const Scale& one, const Scale& temp,
                                                   float& a, float& b) {
    const uint64_t k1 = pack2(one.k, one.k), h1 = pack2(-one.hi, -one.hi);
    const uint64_t k2 = pack2(temp.k, temp.k), h2 = pack2(-temp.hi, -temp.hi);
    uint64_t s1[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)}, s2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
    for (int u = 0; u < kLaneVecs; ++u) {
      float x[Row<DT>::VEC];
      unpack_vec<DT>(q[u], x);
#pragma unroll
      for (int j = 0; j < Row<DT>::VEC; j += 2) {
        const uint64_t xx = pack2(x[j], x[j + 1]);
        float c, d;
        unpack2(fma2(xx, k1, h1), c, d);
        s1[(j >> 1) & 1] = add2(s1[(j >> 1) & 1], pack2(ex2(c), ex2(d)));
        if (kTwo) {
          unpack2(fma2(xx, k2, h2), c, d);
          s2[(j >> 1) & 1] = add2(s2[(j >> 1) & 1], pack2(ex2(c), ex2(d)));
        }
      }
    }
    float c, d;
    unpack2(add2(s1[0], s1[1]), c, d);
    a = (c + d) * one.rest;
    unpack2(add2(s2[0], s2[1]), c, d);
    b = (c + d) * temp.rest;
  }
  // (logits so large that ref * k is off by one or more)
  template <bool kTwo>
  __device__ __forceinline__ void sums_far(const uint4 (&q)[kLaneVecs], float ref, float& a, float& b) const {
    a = b = 0.f;
#pragma unroll
    for (int u = 0; u < kLaneVecs; ++u) {
      float x[Row<DT>::VEC];
      unpack_vec<DT>(q[u], x);
#pragma unroll
      for (int j = 0; j < Row<DT>::VEC; ++j) {
        a += ex2((x[j] - ref) * kLog2e);
        if (kTwo) b += ex2((x[j] - ref) * p.t.hi);
      }
    }
  }
  // A value of every CTA of the row, summed up, and of those before this one; every lane calls it.
  template <typename F>
  __device__ __forceinline__ uint64_t sum_of_ranks(F get, uint64_t& before) const {
    const int lane = threadIdx.x & 31;
    const uint64_t x = lane < ranks ? get(lane) : 0;
    before = warp_sum(lane < rank ? x : 0);
    return warp_sum(x);
  }
  // (reference, sum) pairs of up to 32 parts, joined; every warp calls it.
  template <typename F>
  __device__ __forceinline__ float2 joined(int n, F get) const {
    const int lane = threadIdx.x & 31;
    const float2 b = lane < n ? get(lane) : make_float2(-INFINITY, 0.f);
    float2 a = make_float2(warp_max(b.x), 0.f);
    if (a.x == -INFINITY) return a;
    a.y = b.y * ex2((b.x - a.x) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.y += __shfl_xor_sync(kFull, a.y, o);
    return a;
  }

  // ---- few candidates: a logit that enough chunk maxima reach, and all candidates from there on

  // Histogram of this CTA's chunk maxima, or (few) its threads' maxima, by octaves below `from`; the
  // bins are 0 before.  kMass: their weights in units of 2^-12 of a bin's upper border, rounded down.
  template <bool kMass>
  __device__ __forceinline__ void coarse_histogram(float from, bool few) {
    auto add = [&](float z) {
      const float y = octaves_below(z, from, p.t) * kCoarse;
      if (!(y < kCoarseBins)) return;
      const int b = static_cast<int>(y);
      atomicAdd(&s.coarse[b], kMass ? static_cast<int>(ex2((b - y) * (1.f / kCoarse) + 11.9995f)) : 1);
    };
    if (few) {
      add(highest);
    } else {
      for (int k = threadIdx.x; k < groups * 32; k += kThreads) add(tops[k]);
    }
    __syncthreads();
  }
  // A logit that everything in bins up to b below `from` reaches.
  __device__ __forceinline__ float logit_of(float from, int b) const {
    return from - (static_cast<float>(b) + 1.01f) / (kCoarse * p.t.hi);
  }
  // Warp 0: the first bin with which the sum of value(b) reaches each of the goals, or kCoarseBins.
  template <typename F>
  __device__ __forceinline__ void coarse_reach(F value, float goal0, float goal1, int& b0, int& b1) const {
    constexpr int kEach = (kCoarseBins + 31) / 32;
    const int lane = threadIdx.x & 31;
    float own[kEach], sum = 0.f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int b = lane * kEach + k;
      own[k] = b < kCoarseBins ? value(b) : 0.f;
      sum += own[k];
    }
    float upto = warp_scan(sum) - sum;
    b0 = b1 = kCoarseBins;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      upto += own[k];
      if (upto >= goal0) b0 = min(b0, lane * kEach + k);
      if (upto >= goal1) b1 = min(b1, lane * kEach + k);
    }
    b0 = static_cast<int>(__reduce_min_sync(kFull, static_cast<unsigned>(b0)));
    b1 = static_cast<int>(__reduce_min_sync(kFull, static_cast<unsigned>(b1)));
  }

  // The weights of this CTA's groups, from the sums of chunks; kRefine: those of chunks that weigh much
  // element by element.
  template <bool kRefine>
  __device__ __forceinline__ void weigh_chunks() {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr float kUnit = static_cast<float>(int64_t{1} << kWeightBits);
    float limit = INFINITY;
    if (kRefine) {
      float part = 0.f;
      for (int g = warp; g < groups; g += kWarps) part += masses[g * 32 + lane] * ex2((refs[g] - m) * p.t.hi);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kFull, part, o);
      if (lane == 0) s.part[warp].x = part;
      __syncthreads();
      part = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) part += s.part[w].x;
      limit = part * kHeavy;
    }
    uint64_t mass = 0, light = 0;
    for (int g = warp; g < groups; g += kWarps) {
      const float w = masses[g * 32 + lane] * ex2((refs[g] - m) * p.t.hi);  // nothing: 2^-inf
      unsigned todo = kRefine ? __ballot_sync(kFull, w > limit) : 0u;
      float rest = kRefine && w > limit ? 0.f : w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(kFull, rest, o);
      const uint64_t in_light = static_cast<uint64_t>(rest * kUnit);
      uint64_t in_heavy = 0;
      while (todo) {  // one chunk by the whole warp
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const int t1 = min((g + 1) << p.span_log2, tiles);
        for (int t = g << p.span_log2; t < t1; ++t) {
#pragma unroll 1
          for (int e = lane; e < kLaneVecs * Row<DT>::VEC; e += 32) {
            const int id = row.id((tile0 + t) * kTileVecs + 32 * (e / Row<DT>::VEC) + l) + e % Row<DT>::VEC;
            if (id >= 0 && id < p.V) in_heavy += weight(row.at(id));
          }
        }
      }
      if (kRefine && __any_sync(kFull, in_heavy != 0)) in_heavy = warp_sum(in_heavy);
      if (lane == 0) sums[g] = in_light + in_heavy;
      light += in_light;
      mass += in_light + in_heavy;
    }
    set_mass(mass, light);
  }
  static constexpr float kHeavy = 0x1p-8f;  // of this CTA's weights
  __device__ __forceinline__ void set_mass(uint64_t of_warp, uint64_t light) {
    if ((threadIdx.x & 31) == 0) s.warp_mass[threadIdx.x >> 5] = of_warp, s.warp_light[threadIdx.x >> 5] = light;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint64_t mass = 0;
      light = 0;
      for (int w = 0; w < kWarps; ++w) mass += s.warp_mass[w], light += s.warp_light[w];
      s.mine.mass = mass;
      s.mine.light = light;
    }
    __syncthreads();
  }
  // A sum over chunks is off by less than this share of the light ones among them (at most 2^20 terms
  // of at least 2^-20 each make up half of a sum that is at least 1): 20 * 2^-23 * ln 2 of the
  // exponents, 2^-22 of each term and of the factors, and the additions.
  static constexpr double kError = 0x1p-18;
  static constexpr uint64_t kRounding = 64 * (kMaxGroups + 1);  // of a CTA's sums to whole units, amply

  // All candidates from logit t on, to the first CTA's list: first the chunks that have some, then
  // their vectors, one a thread (a chunk at a time in the lane that found it would wait for memory once
  // for every chunk).
  __device__ __forceinline__ void list_from(float t) {
    if (highest >= t) {
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      for (int g = warp; g < groups; g += kWarps) {
        if (!(tops[g * 32 + lane] >= t)) continue;
        const int at = atomicAdd(&s.queued, 1);
        if (at < p.cap) queue[at] = static_cast<uint16_t>(g * 32 + lane);
      }
    }
    __syncthreads();
    // more chunks than the list holds: no need to look
    const int queued = s.queued;
    if (queued > p.cap) {
      if (threadIdx.x == 0) atomicAdd(&first.ctl.listed, p.cap + 1);
      return;
    }
    constexpr int kAhead = 4;  // vectors on their way
    const int each_log2 = kLaneVecsLog2 + p.span_log2, all = queued << each_log2;
    for (int k0 = threadIdx.x; k0 < all; k0 += kAhead * kThreads) {
      uint4 q[kAhead];
      int vec[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kThreads;
        q[u] = Row<DT>::none();
        vec[u] = 0;
        if (k >= all) continue;
        const int chunk = queue[k >> each_log2];
        const int tile = ((chunk >> 5) << p.span_log2) + (k >> kLaneVecsLog2 & ((1 << p.span_log2) - 1));
        vec[u] = (tile0 + tile) * kTileVecs + 32 * (k & (kLaneVecs - 1)) + (chunk & 31);
        if (tile < tiles) q[u] = row.load(vec[u]);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!(vec_max<DT>(q[u]) >= t)) continue;
        int id = row.id(vec[u]);
#pragma unroll 1
        for (int j = 0; j < Row<DT>::VEC; j += 2, id += 2) {
          float a, b;
          Row<DT>::take2(q[u], a, b);
          if (a >= t && a > -INFINITY) append(a, id);
          if (b >= t && b > -INFINITY) append(b, id + 1);
        }
      }
    }
  }

  // First CTA: drops listed candidates that come behind the k-th (by_k) or behind the mass `goal`, as far as
  // coarse bins tell; how many are left.  (The list began with what the largest of chunks alone reach.)
  __device__ __forceinline__ int drop_behind(int n, bool by_k, uint64_t goal) const {
    constexpr int kEach = kCap / kThreads;
    int* const low = s.coarse;   // of halved weights in a bin (or their number): the lower 21 bits' sum
    int* const high = s.row_coarse;
    for (int b = threadIdx.x; b < kCoarseBins; b += kThreads) low[b] = high[b] = 0;
    if (threadIdx.x == 0) s.queued = 0;
    __syncthreads();
    // (a weight is at most 2^42, that included; a unit that a half drops keeps a candidate more, at worst)
    static_assert(kCap <= 1 << 11 && kWeightBits - 22 + 11 < 32 && 21 + 11 <= 32, "sums of 2048 in 32 bits");
#pragma unroll 1
    for (int k = threadIdx.x; k < n; k += kThreads) {
      const float y = octaves_below(listed_z(k), m, p.t) * kCoarse;
      if (!(y < kCoarseBins)) continue;
      const int b = static_cast<int>(y);
      if (by_k) {
        atomicAdd(low + b, 1);
      } else {
        const uint64_t w = weight(listed_z(k));
        atomicAdd(reinterpret_cast<unsigned*>(low + b), static_cast<unsigned>(w >> 1 & ((1u << 21) - 1)));
        atomicAdd(reinterpret_cast<unsigned*>(high + b), static_cast<unsigned>(w >> 22));
      }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      int b0, b1;
      coarse_reach(
          [&](int b) {
            return static_cast<float>(static_cast<unsigned>(low[b])) +
                   static_cast<float>(static_cast<unsigned>(high[b])) * 0x1p21f;
          },
          by_k ? static_cast<float>(p.top_k) : static_cast<float>(goal) * 0.50005f, INFINITY, b0, b1);
      if (threadIdx.x == 0) s.from = b0 < kCoarseBins ? logit_of(m, b0) : -INFINITY;
    }
    uint64_t mine[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) mine[e] = e * kThreads + threadIdx.x < n ? keys[e * kThreads + threadIdx.x] : 0;
    __syncthreads();
    const float from = s.from;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (e * kThreads + threadIdx.x < n && of_order(~static_cast<uint32_t>(mine[e] >> 32)) >= from)
        keys[atomicAdd(&s.queued, 1)] = mine[e];
    }
    __syncthreads();
    return s.queued;
  }

  // x rounded up (down) to whole units, in every thread: the doubles cost one warp's time, not eight's
  // (this GPU has a 64th of the 32-bit rate for them).
  template <typename F>
  __device__ __forceinline__ void set_goal(F f) {
    if (threadIdx.x == 0) f();
    __syncthreads();
  }

  // First CTA: the token among n <= kFew listed candidates, which hold all that the filters keep
  // (reaches: all up to the mass goal_p, else all from `least` on).  goal_p: what top_p has to reach,
  // known to +- error (with top_k: found here, exact); -2 where that leaves the cut open.
  __device__ __forceinline__ int draw_few(int n, float u, uint64_t goal_p, uint64_t error, float least,
                                          bool reaches) {
    // 2, 4 or 8 threads a candidate compare it with all
    const int sh = n <= 32 ? 3 : n <= 64 ? 2 : 1, step = 1 << sh;
    const int i = threadIdx.x >> sh, part = threadIdx.x & (step - 1);
    if (threadIdx.x == 0) s.ctl.found = INT_MAX, s.ctl.bin = n - 1, s.ctl.mass = 0, s.ctl.lo = 0u;
    if (threadIdx.x < n) {
      const uint64_t key = keys[threadIdx.x];
      s.few[threadIdx.x] = make_ulonglong2(key, weight(listed_z(threadIdx.x)));
    }
    __syncthreads();
    const bool busy = __any_sync(kFull, i < n);
    const ulonglong2 mine = s.few[min(i, n - 1)];
    int place = 0;
    uint64_t before = 0;
    if (busy) {
      for (int j = part; j < n; j += step) {
        const ulonglong2 o = s.few[j];
        if (o.x < mine.x) ++place, before += o.y;
      }
      for (int o = 1; o < step; o *= 2) {
        place += __shfl_xor_sync(kFull, place, o);
        before += __shfl_xor_sync(kFull, before, o);
      }
    }
    const uint64_t upto = before + mine.y;
    const bool lead = i < n && part == 0;
    const int limit = min(n, p.top_k);
    if (p.top_p < 1.0) {
      if (p.top_k < p.V) {
        if (lead && place == limit - 1) s.goal = static_cast<uint64_t>(ceil(p.top_p * static_cast<double>(upto)));
        __syncthreads();
        goal_p = s.goal;
      }
      // the shortest prefix that reaches the goal; open if the goal's error could move it
      if (lead && before < goal_p && upto >= goal_p) s.ctl.bin = place;
      if (lead && error != 0 &&
          ((upto + error >= goal_p && upto <= goal_p + error) ||
           (reaches && place == limit - 1 && upto < goal_p + error)))
        s.ctl.lo = 1u;
      __syncthreads();
      if (s.ctl.lo != 0u) return -2;
    }
    const int last = min(s.ctl.bin, limit - 1);
    const float z = of_order(~static_cast<uint32_t>(mine.x >> 32));
    const bool keep = lead && place <= last && z >= least;
    // the same threads again, by id among the kept
    __syncthreads();
    if (lead) s.few[i] = make_ulonglong2(keep ? mine.x & 0xFFFFFFFFu : 0xFFFFFFFFu, keep ? mine.y : 0);
    __syncthreads();
    uint64_t by_id = 0, kept_mass = 0;
    const uint64_t id = s.few[min(i, n - 1)].x;
    if (busy) {
      for (int j = part; j < n; j += step) {
        const ulonglong2 o = s.few[j];
        kept_mass += o.y;
        if (o.x <= id) by_id += o.y;
      }
      for (int o = 1; o < step; o *= 2) {
        by_id += __shfl_xor_sync(kFull, by_id, o);
        kept_mass += __shfl_xor_sync(kFull, kept_mass, o);
      }
    }
    if (threadIdx.x == 0)
      s.goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(kept_mass));
    __syncthreads();
    if (keep && by_id > s.goal) atomicMin(&s.ctl.found, static_cast<int>(id));
    __syncthreads();
    return s.ctl.found == INT_MAX ? -1 : s.ctl.found;
  }

  // The same for up to kCap candidates, by sorting.  (Weights are computed again where they are needed
  // again: a thread has eight at most, and loops are short to fetch.)
  __device__ __forceinline__ int draw_listed(int n, float u, uint64_t goal_p, uint64_t error, float least,
                                             bool reaches) {
    sort_list(n);
    const int each = (n + kThreads - 1) / kThreads, at0 = threadIdx.x * each, at1 = min(at0 + each, n);
    uint64_t mass = 0;
    int count = 0;
    if (threadIdx.x == 0) s.ctl.bin = n - 1, s.ctl.lo = 0u, s.ctl.found = -1;
    const int limit = min(n, p.top_k);
    if (p.top_p < 1.0) {
#pragma unroll 1
      for (int at = at0; at < at1; ++at) mass += weight(listed_z(at));
      block_scan(mass, count);
      if (p.top_k < p.V) {
        if (at0 < limit && at1 >= limit) {
          uint64_t upto = mass;
#pragma unroll 1
          for (int at = at0; at < limit; ++at) upto += weight(listed_z(at));
          s.goal = static_cast<uint64_t>(ceil(p.top_p * static_cast<double>(upto)));
        }
        __syncthreads();
        goal_p = s.goal;
      }
      uint64_t upto = mass;
#pragma unroll 1
      for (int at = at0; at < at1; ++at) {
        const uint64_t before = upto;
        upto += weight(listed_z(at));
        if (before < goal_p && upto >= goal_p) s.ctl.bin = at;
        if (error != 0 && ((upto + error >= goal_p && upto <= goal_p + error) ||
                           (reaches && at == limit - 1 && upto < goal_p + error)))
          s.ctl.lo = 1u;
      }
      __syncthreads();
      if (s.ctl.lo != 0u) return -2;
    }
    __syncthreads();
    const int last = min(s.ctl.bin, limit - 1);
    // the kept by id: key id << 32 | order(z)
#pragma unroll 1
    for (int at = at0; at < min(at1, last + 1); ++at) {
      const float z = listed_z(at);
      keys[at] = z >= least ? static_cast<uint64_t>(listed_id(at)) << 32 | order_of(z) : ~uint64_t{0};
    }
    sort_list(last + 1);
    auto weight_at = [&](int at) {
      return keys[at] != ~uint64_t{0} ? weight(of_order(static_cast<uint32_t>(keys[at]))) : 0;
    };
    const int end = min(at1, last + 1);
    mass = 0;
#pragma unroll 1
    for (int at = at0; at < end; ++at) mass += weight_at(at);
    const uint64_t own = mass;
    block_scan(mass, count);
    if (threadIdx.x == kThreads - 1)
      s.goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(mass + own));
    __syncthreads();
    const uint64_t goal = s.goal;
    if (!(mass > goal) && mass + own > goal) {
#pragma unroll 1
      for (int at = at0; at < end; ++at) {
        mass += weight_at(at);
        if (mass > goal) {
          s.ctl.found = static_cast<int>(keys[at] >> 32);
          break;
        }
      }
    }
    __syncthreads();
    return s.ctl.found;
  }

  // The id in tiles [t, t1) at which the sum of weights relative to the largest exceeds `goal` (it does);
  // by the whole CTA, a tile at a time, a warp each 32 of its vectors.  Left as it is where that sum comes
  // within `error` of the goal before or behind the token.
  __device__ __forceinline__ void find_in_tiles(int t, int t1, float goal, float error) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float before = 0.f;
    for (; t < t1; ++t) {
      const int vec = (tile0 + t) * kTileVecs + 32 * warp + lane;
      float x[Row<DT>::VEC];
      unpack_vec<DT>(row.load(vec), x);
      float w[Row<DT>::VEC], sum = 0.f;
#pragma unroll
      for (int j = 0; j < Row<DT>::VEC; ++j) w[j] = ex2((x[j] - m) * p.t.hi), sum += w[j];
      float upto = warp_scan(sum);
      if (lane == 31) s.part[warp].x = upto;
      __syncthreads();
      float from = before;
      for (int k = 0; k < kWarps; ++k) {
        if (k == warp) from = before;
        before += s.part[k].x;
      }
      upto += from;
      if (upto > goal && !(upto - sum > goal)) {
        upto -= sum;
#pragma unroll
        for (int j = 0; j < Row<DT>::VEC; ++j) {
          const float low = upto;
          upto += w[j];
          if (!(low > goal) && w[j] > 0.f && upto > goal + error && low + error < goal)
            first.ctl.found = row.id(vec) + j;
        }
      }
      __syncthreads();
      if (before > goal) break;
    }
  }
  // The same by exact weights, in units: where the heavy chunks' sums are exact the guard is far below what
  // sums in 32 bits are off by.
  __device__ __forceinline__ void find_exactly(int t, int t1, uint64_t goal, uint64_t error) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t before = 0;
    for (; t < t1; ++t) {
      const int vec = (tile0 + t) * kTileVecs + 32 * warp + lane;
      const uint4 q = row.load(vec);
      uint4 left = q;
      float a, b;
      uint64_t sum = 0;
#pragma unroll 1
      for (int j = 0; j < Row<DT>::VEC; j += 2) {
        Row<DT>::take2(left, a, b);
        sum += weight(a) + weight(b);
      }
      uint64_t upto = warp_scan(sum);
      if (lane == 31) s.warp_mass[warp] = upto;
      __syncthreads();
      uint64_t from = before;
      for (int k = 0; k < kWarps; ++k) {
        if (k == warp) from = before;
        before += s.warp_mass[k];
      }
      upto += from;
      if (upto > goal && !(upto - sum > goal)) {
        uint64_t low = upto - sum;
        int id = row.id(vec);
        left = q;
#pragma unroll 1
        for (int j = 0; j < Row<DT>::VEC; j += 2, id += 2) {
          Row<DT>::take2(left, a, b);
          const uint64_t mid = low + weight(a), high = mid + weight(b);
          if (low + error <= goal && mid > goal + error) first.ctl.found = id;
          if (mid + error <= goal && high > goal + error) first.ctl.found = id + 1;
          low = high;
        }
      }
      __syncthreads();
      if (before > goal) break;
    }
  }
  // Warp 0: the group in which the sum of sums[] exceeds goal, and the sum before it (there is
  // one).
  __device__ __forceinline__ void find_group(const uint64_t* of_group, int n, uint64_t before, uint64_t goal) {
    const int lane = threadIdx.x & 31;
    for (int g0 = 0; g0 < n; g0 += 32) {
      const uint64_t x = g0 + lane < n ? of_group[g0 + lane] : 0;
      const uint64_t upto = before + warp_scan(x);
      const unsigned hit = __ballot_sync(kFull, upto > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) s.group = g0 + lane, s.group_before = upto - x;
        break;
      }
      before = __shfl_sync(kFull, upto, 31);
    }
  }

  // No filter: the group of tiles by the weights of chunks, then the token in it; -2 where the error of
  // sums in 32 bits leaves either open.  again: behind weigh_chunks<true>.
  __device__ __forceinline__ int draw_whole(float u, bool again) {
    constexpr float kOfUnit = 1.f / static_cast<float>(int64_t{1} << kWeightBits);
    uint64_t before_own;
    uint64_t none;
    const uint64_t all = sum_of_ranks([&](int r) { return of(r).mine.mass; }, before_own);
    const uint64_t light = sum_of_ranks([&](int r) { return of(r).mine.light; }, none);
    if (threadIdx.x == 0) {
      s.goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(all));
      // u * all, the sum before a group and (in the first try) the sum in it
      s.goal_error = static_cast<uint64_t>(2.0 * kError * static_cast<double>(light)) + 2 * kRounding * ranks;
      s.group_before = before_own;
      if (rank == 0) s.ctl.found = -2;
    }
    sync();
    const uint64_t goal = s.goal, before = s.group_before;
    if (before <= goal && before + s.mine.mass > goal) {
      __syncthreads();
      if (threadIdx.x < 32) find_group(sums, groups, before, goal);
      __syncthreads();
      const int t0 = s.group << p.span_log2, t1 = min((s.group + 1) << p.span_log2, tiles);
      if (again)
        find_exactly(t0, t1, goal - s.group_before, s.goal_error);
      else
        find_in_tiles(t0, t1, static_cast<float>(goal - s.group_before) * kOfUnit,
                      static_cast<float>(s.goal_error) * kOfUnit);
    }
    sync();
    return first.ctl.found;
  }
  static_assert(kLaneVecs == kWarps, "a tile is shared out by its vectors");

  // The id at which the running sum of f(z, id) by rising id first exceeds goal(total); -1 if it
  // never does.
  template <typename F, typename G>
  __device__ __forceinline__ int locate(F f, G goal_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t sum = 0, of_warp = 0;
    each([&](float z, int id) { sum += f(z, id); },
         [&](int unit) {
           sum = warp_sum(sum);
           if (lane == 0) sums[unit] = sum;
           of_warp += sum;
           sum = 0;
         });
    if (lane == 0) s.warp_mass[warp] = of_warp;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) of_warp += s.warp_mass[w];
      s.total[0] = of_warp;
      if (rank == 0) s.ctl.found = -1;
    }
    sync();
    uint64_t before;
    const uint64_t all = sum_of_ranks([&](int r) { return of(r).total[0]; }, before);
    set_goal([&] { s.goal = goal_of(all); });
    const uint64_t goal = s.goal;
    if (warp == 0 && before <= goal && before + s.total[0] > goal) {
      find_group(sums, tiles * kLaneVecs >> strips_log2, before, goal);
      __syncwarp();
      uint64_t upto = s.group_before;
      const int vec0 = tile0 * kTileVecs + (32 * s.group << strips_log2) + lane;
#pragma unroll 1
      for (int u = 0; u < 1 << strips_log2; ++u) {
        const int vec = vec0 + 32 * u;
        const uint4 q = row.load(vec);
        const int id = row.id(vec);
        sum = 0;
        uint4 left = q;
        float a, b;
#pragma unroll 1
        for (int j = 0; j < Row<DT>::VEC; j += 2) {
          Row<DT>::take2(left, a, b);
          sum += f(a, id + j) + f(b, id + j + 1);
        }
        const uint64_t scan = warp_scan(sum);
        uint64_t here = upto + scan - sum;
        if (!(here > goal) && here + sum > goal) {
          left = q;
#pragma unroll 1
          for (int j = 0; j < Row<DT>::VEC; j += 2) {
            Row<DT>::take2(left, a, b);
            here += f(a, id + j);
            int at = here > goal ? id + j : -1;
            here += f(b, id + j + 1);
            if (at < 0 && here > goal) at = id + j + 1;
            if (at >= 0) {
              first.ctl.found = at;
              break;
            }
          }
        }
        upto += __shfl_sync(kFull, scan, 31);
        if (upto > goal) break;
      }
    }
    sync();
    const int id = first.ctl.found;
    sync();
    return id;
  }

  // ---- the histogram of weights

  __device__ __forceinline__ uint32_t* bin_words(int b) {
    return reinterpret_cast<uint32_t*>(&fine.bins_lo_hi[b]);
  }
  // (counts: how many, too; only top_k asks for it)
  __device__ __forceinline__ void histogram(bool counts) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) fine.bins_lo_hi[b] = 0, fine.bins[b] = 0;
    __syncthreads();
    each([&](float z, int) {
      const int b = bin_of(z);
      if (b >= kBins) return;
      const uint64_t w = weight(z);
      uint32_t* words = bin_words(b);
      const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(words, lo);
      const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
      if (hi) atomicAdd(words + 1, hi);
      if (counts) atomicAdd(&fine.bins[b], 1);
    });
    sync();
    if (rank == 0 && ranks > 1) {
      for (int b = threadIdx.x; b < kBins; b += kThreads) {
        uint64_t mass = fine.bins_lo_hi[b];
        int count = fine.bins[b];
#pragma unroll
        for (int r = 1; r < kMaxRanks; ++r) {  // (all loads on their way together)
          if (r >= ranks) break;
          const Fine& o = *cg::this_cluster().map_shared_rank(&fine, r);
          mass += o.bins_lo_hi[b];
          count += o.bins[b];
        }
        fine.bins_lo_hi[b] = mass;
        fine.bins[b] = count;
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
  // Warp 0: what top_p has to reach of the sum of all weights, and how far that may be off.
  __device__ __forceinline__ void set_mass_goal() {
    uint64_t before;
    const uint64_t all = sum_of_ranks([&](int r) { return of(r).mine.mass; }, before);
    const uint64_t light = sum_of_ranks([&](int r) { return of(r).mine.light; }, before);
    if (threadIdx.x == 0) {
      s.goal = static_cast<uint64_t>(ceil(p.top_p * static_cast<double>(all)));
      s.goal_error = static_cast<uint64_t>(kError * static_cast<double>(light)) + kRounding * ranks;
    }
    __syncwarp();
  }
  // Does a prefix of this count and mass reach the goal (k candidates, or the mass x)?
  struct Goal {
    bool by_mass;
    int k;
    uint64_t x;
    __device__ __forceinline__ bool reached(int64_t count, uint64_t mass) const {
      return by_mass ? mass >= x : count >= k;
    }
  };

  // The shortest prefix that reaches `goal`; its cut and mass are in first.ctl afterwards.  The whole
  // prefix of weights above 0 where that does not reach it.
  __device__ __forceinline__ void find_cut(const Goal& goal) {
    if (rank == 0) {
      uint64_t mass = 0;
      int count = 0;
      const int b0 = threadIdx.x * kBinsPerThread;
      for (int b = b0; b < min(b0 + kBinsPerThread, kBins); ++b) mass += fine.bins_lo_hi[b], count += fine.bins[b];
      if (threadIdx.x == 0) s.ctl.bin = -1, s.ctl.listed = 0;
      block_scan(mass, count);
      for (int b = b0; b < min(b0 + kBinsPerThread, kBins); ++b) {
        const uint64_t mass1 = mass + fine.bins_lo_hi[b];
        const int count1 = count + fine.bins[b];
        if (!goal.reached(count, mass) && goal.reached(count1, mass1)) {
          s.ctl.bin = b;
          s.ctl.bin_count = fine.bins[b];
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
    int listed = in_bin;  // (0 where they were not counted)
    if (listed <= p.cap) {
      each([&](float z, int id) {
        if (bin_of(z) == bin) append(z, id);
      });
      sync();
      listed = first.ctl.listed;
    }
    if (listed <= p.cap) {
      if (rank == 0) cut_in_list(goal);
      sync();
    } else {
      cut_in_bin(goal, bin);
    }
  }
  // Largest top_k that is tried with a list.
  __device__ __forceinline__ int list_k() const { return p.cap - p.cap / 4; }
  __device__ __forceinline__ void append(float z, int id) {
    const int at = atomicAdd(&first.ctl.listed, 1);
    if (at < p.cap) first_keys[at] = static_cast<uint64_t>(~order_of(z)) << 32 | static_cast<uint32_t>(id);
  }
  __device__ __forceinline__ void sort_list(int n) {
    __syncthreads();
    sort_keys(keys, n);
  }
  __device__ __forceinline__ float listed_z(int k) const {
    return of_order(~static_cast<uint32_t>(keys[k] >> 32));
  }
  __device__ __forceinline__ int listed_id(int k) const { return static_cast<int>(keys[k] & 0xFFFFFFFFu); }

  // First CTA: the cut among the listed candidates, behind ctl.before and ctl.count_before.
  __device__ __forceinline__ void cut_in_list(const Goal& goal) {
    const int n = min(s.ctl.listed, p.cap);
    sort_list(n);
    const int each = (n + kThreads - 1) / kThreads, at0 = threadIdx.x * each, at1 = min(at0 + each, n);
    uint64_t mass = 0;
    int count = max(at1 - at0, 0);
#pragma unroll 1
    for (int at = at0; at < at1; ++at) mass += weight(listed_z(at));
    block_scan(mass, count);
    mass += s.ctl.before;
    count += s.ctl.count_before;
#pragma unroll 1
    for (int at = at0; at < at1; ++at) {
      const bool was = goal.reached(count, mass);
      mass += weight(listed_z(at));
      if (!was && goal.reached(++count, mass)) {
        s.ctl.cut = Cut{listed_z(at), listed_id(at)};
        s.ctl.mass = mass;
      }
    }
    __syncthreads();
  }

  // The cut inside a bin of more candidates than are sorted: the value by bisection, then how many of
  // the candidates with that value.
  __device__ __forceinline__ void cut_in_bin(const Goal& goal, int bin) {
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
    const uint64_t w = max(weight(z), uint64_t{1}), base = before + above;
    int64_t ties = goal.k - (count_before + count_above);
    if (goal.by_mass) {
      ties = static_cast<int64_t>((goal.x - base + w - 1) / w);
    }
    const int id = locate([&](float x, int) { return x == z ? uint64_t{1} : uint64_t{0}; },
                          [&](uint64_t) { return static_cast<uint64_t>(ties - 1); });
    if (threadIdx.x == 0 && rank == 0) {
      s.ctl.cut = Cut{z, id};
      s.ctl.mass = base + ties * w;
    }
    sync();
  }
  // Sums over all threads of the row, in every thread.
  __device__ __forceinline__ void sum_of_row(uint64_t& a, uint64_t& b) {
    const int warp = threadIdx.x >> 5;
    a = warp_sum(a);
    b = warp_sum(b);
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
    uint64_t before;
    a = sum_of_ranks([&](int r) { return of(r).total[0]; }, before);
    b = sum_of_ranks([&](int r) { return of(r).total[1]; }, before);
  }

  // The token by passes over all weights, whatever the filters keep.
  __device__ __forceinline__ int draw_any(float u) {
    Cut cut{-INFINITY, INT_MAX};
    sync();  // what the chunks' sums were is overwritten
    const bool by_k = p.top_k < p.V, by_p = p.top_p < 1.0;
    if (by_k || by_p) {
      histogram(by_k);
      if (by_k) {
        find_cut(Goal{false, p.top_k, 0});
        cut = first.ctl.cut;
      }
      if (by_p) {
        uint64_t all = first.ctl.mass;
        if (!by_k) {
          if (rank == 0) {
            uint64_t mass = 0;
            int none = 0;
            const int b0 = threadIdx.x * kBinsPerThread;
            for (int b = b0; b < min(b0 + kBinsPerThread, kBins); ++b) mass += fine.bins_lo_hi[b];
            const uint64_t own = mass;
            block_scan(mass, none);
            if (threadIdx.x == kThreads - 1) s.ctl.mass = mass + own;
          }
          sync();
          all = first.ctl.mass;
        }
        sync();
        set_goal([&] { s.goal = static_cast<uint64_t>(ceil(p.top_p * static_cast<double>(all))); });
        find_cut(Goal{true, 0, s.goal});
        cut = tighter(cut, first.ctl.cut);
        sync();
      }
    }
    if (p.log_min_p > -INFINITY) {
      set_goal([&] { s.least = __double2float_ru(static_cast<double>(m) + p.temperature * p.log_min_p); });
      cut = tighter(cut, Cut{s.least, INT_MAX});
    }
    return locate([&](float z, int id) { return kept(cut, z, id) ? weight(z) : 0; },
                  [&](uint64_t all) { return static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(all)); });
  }

  // The first pass, what the CTAs tell one another, and the token (first CTA); -1 for a row without a
  // finite logit, -2 where all weights of a row are needed to 36 bits (sample_rest_kernel).
  __device__ __forceinline__ int draw(float u) {
    const bool by_k = p.top_k < p.V, by_p = p.top_p < 1.0, by_least = p.log_min_p > -INFINITY;
    const bool by_mass = !by_k && (by_p || !by_least);  // the sum of all weights is needed
    for (int b = threadIdx.x; b < kCoarseBins; b += kThreads) s.coarse[b] = 0;
    if (threadIdx.x == 0) s.queued = 0, s.ctl.listed = 0;
    if (!by_mass)
      pass<false, true>();
    else if (p.temperature == 1.0)
      pass<true, true>();
    else
      pass<true, false>();
    // top_k: the logits that all of k, and an even share of it, of this CTA's chunks reach
    if (by_k && p.top_k <= list_k()) {
      // (thread maxima will do where there are twice as many: they are as good as k chunks)
      if (m > -INFINITY) coarse_histogram<false>(m, p.top_k <= kThreads / 2);
      if (threadIdx.x < 32) {
        int b0, b1;
        coarse_reach([&](int b) { return static_cast<float>(s.coarse[b]); },
                     static_cast<float>((p.top_k + ranks - 1) / ranks), static_cast<float>(p.top_k), b0, b1);
        if (threadIdx.x == 0) {
          s.mine.some = b0 < kCoarseBins ? logit_of(m, b0) : -INFINITY;
          s.mine.all = b1 < kCoarseBins ? logit_of(m, b1) : -INFINITY;
        }
      }
    }
    if (threadIdx.x == 0) s.mine.m = m, s.mine.sum = total;
    sync();
    if constexpr (kCluster) {
      const float2 all = joined(ranks, [&](int r) { return make_float2(of(r).mine.m, of(r).mine.sum); });
      m = all.x;
      total = all.y;
    }
    if (m == -INFINITY) return -1;
    float least = -INFINITY;
    if (by_least) {
      set_goal([&] { s.least = __double2float_ru(static_cast<double>(m) + p.temperature * p.log_min_p); });
      least = s.least;
    }

    float t = -INFINITY;  // all that the filters keep is from this logit on
    uint64_t goal = 0, error = 0;
    bool reaches = true;  // the list is not cut short by min_p
    bool sure = true;     // all that is kept is listed
    if (by_mass) {
      weigh_chunks<false>();
      if (!by_p) {
        int token;
#pragma unroll 1
        for (bool again = false;; again = true) {
          if (again) weigh_chunks<true>();
          sync();
          token = draw_whole(u, again);
          if (token != -2 || again) break;
        }
        if (kCluster && p.at_once && token == -2) return in_full(u);
        return token;
      }
      coarse_histogram<true>(m, false);
      sync();
      for (int b = threadIdx.x; b < kCoarseBins; b += kThreads) {
        int n = 0;
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r)  // (all loads on their way together)
          if (r < ranks) n += of(r).coarse[b];
        s.row_coarse[b] = n;
      }
      __syncthreads();
      if (threadIdx.x < 32) {
        set_mass_goal();
        // the maxima that reach the mass, but no more of them than the list is likely to hold (the mass
        // of all that is listed may reach it all the same)
        int b0, b1, none;
        coarse_reach(
            [&](int b) {
              return static_cast<float>(s.row_coarse[b]) * ex2(b * (-1.f / kCoarse) - 12.f);
            },
            static_cast<float>(s.goal) * 0x1.002p-42f, INFINITY, b0, none);
        coarse_reach([&](int b) { return static_cast<float>(s.row_coarse[b]) * (1.f / 3750.f); },
                     static_cast<float>(p.cap / 4), INFINITY, b1, none);
        if (threadIdx.x == 0) {
          s.from = min(b0, b1) < kCoarseBins ? logit_of(m, min(b0, b1)) : -INFINITY;
          s.sure = b0 <= b1;
        }
      }
      __syncthreads();
      goal = s.goal;
      error = s.goal_error;
      t = fmaxf(s.from, least);
      reaches = s.from > least;
      sure = s.sure || !reaches;
    } else if (by_k) {
      if (p.top_k <= list_k()) {
        const int lane = threadIdx.x & 31;
        const float some = -warp_max(lane < ranks ? -of(lane).mine.some : -INFINITY);
        const float all = warp_max(lane < ranks ? of(lane).mine.all : -INFINITY);
        // what lies further below weighs nothing
        t = fmaxf(fmaxf(some, all), logit_of(m, kCoarseBins - 1));
      }
      if (!by_p) t = fmaxf(t, least);
    } else {
      t = least;
    }
    if (t > -INFINITY || p.V <= p.cap) {
      list_from(t);
      sync();
      int n = first.ctl.listed;
      if (n > 0 && n <= p.cap) {
        for (bool again = false;; again = true) {
          if (rank == 0) {
            bool whole = true;  // all that is kept is listed
            if ((n > kFew || !sure) && (by_k || by_mass) && !again) {
              n = tightened(n, by_k, goal + error);
              whole = sure || s.from > -INFINITY;
            }
            const int token = !whole       ? -3
                              : n <= kFew ? draw_few(n, u, goal, error, least, reaches)
                                          : listed(n, u, goal, error, least, reaches);
            if (threadIdx.x == 0) s.ctl.hi = static_cast<uint32_t>(token);
          }
          if (!by_mass || (!kCluster && again)) break;
          sync();
          if (static_cast<int>(first.ctl.hi) != -2 || again) break;
          // once more, with the sum of weights known better
          weigh_chunks<true>();
          sync();
          if (threadIdx.x < 32) set_mass_goal();
          __syncthreads();
          goal = s.goal;
          error = s.goal_error;
        }
        if (kCluster && by_mass) {
          const int token = static_cast<int>(first.ctl.hi);
          if (token == -3 || (token == -2 && p.at_once)) return in_full(u);
        }
        return rank == 0 ? max(static_cast<int>(s.ctl.hi), -2) : -1;
      }
    }
    return by_mass && !kCluster ? -2 : in_full(u);
  }
  // Functions of their own, of copies: so the members stay in registers here and there.
  static __device__ __noinline__ int listed_of(const Sampler& x, int n, float u, uint64_t goal, uint64_t error,
                                               float least, bool reaches) {
    Sampler own(x);
    return own.draw_listed(n, u, goal, error, least, reaches);
  }
  static __device__ __noinline__ int tightened_of(const Sampler& x, int n, bool by_k, uint64_t goal) {
    const Sampler own(x);
    return own.drop_behind(n, by_k, goal);
  }
  static __device__ __noinline__ int in_full_of(const Sampler& x, float u) {
    Sampler own(x);
    return own.draw_any(u);
  }
  __device__ __forceinline__ int listed(int n, float u, uint64_t goal, uint64_t error, float least,
                                        bool reaches) const {
    const Sampler copy(*this);
    return listed_of(copy, n, u, goal, error, least, reaches);
  }
  __device__ __forceinline__ int tightened(int n, bool by_k, uint64_t goal) const {
    const Sampler copy(*this);
    return tightened_of(copy, n, by_k, goal);
  }
  __device__ __forceinline__ int in_full(float u) const {
    const Sampler copy(*this);
    return in_full_of(copy, u);
  }
};

template <int DT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  const int ranks = kCluster ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
  const int rank = kCluster ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  pdl_trigger();
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
  Fine& fine = *reinterpret_cast<Fine*>(dyn + sizeof(Shared));
  Sampler<DT, kCluster> x(p, s, *first, fine, logits);
  x.place(dyn, rank, ranks);
  const float u = fminf(fmaxf(p.uniform[r], 0.f), 0x1.fffffep-1f);
  const int token = x.draw(u);
  if (rank == 0 && threadIdx.x == 0) {
    const float m = x.m;
    p.out.row_max[r] = m;
    p.out.lse[r] = m == -INFINITY ? m : m + logf(x.total);
    p.out.argmax[r] = token;
    // (a row left open: what its token's probability will be multiplied by)
    p.out.conf[r] = token == -2 ? 1.f / x.total
                    : token < 0 ? 0.f
                                : ex2((load_logit(logits, DT, token) - m) * kLog2e) / x.total;
  }
  if constexpr (kCluster) x.sync();  // nobody leaves while its shared memory may be read
}

// The rows that sample_kernel left open, a cluster each: there are few of them or none, and in
// sample_kernel one of them would hold a CTA ten times as long as its neighbours.
template <int DT>
__global__ void __launch_bounds__(kThreads, 3) sample_rest_kernel(const __grid_constant__ SampleParams p,
                                                                  int rows) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ unsigned open[kWarps];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  const auto cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int own = blockIdx.x / ranks, clusters = gridDim.x / ranks;
  if (threadIdx.x < 32) s.pow2[threadIdx.x] = kPow2Table[threadIdx.x];
  pdl_wait();
  for (int64_t r0 = own; r0 < rows; r0 += static_cast<int64_t>(clusters) * kThreads) {
    const int64_t mine = r0 + static_cast<int64_t>(threadIdx.x) * clusters;
    const unsigned found = __ballot_sync(kFull, mine < rows && __ldcg(p.out.argmax + mine) == -2);
    if ((threadIdx.x & 31) == 0) open[threadIdx.x >> 5] = found;
    cluster.sync();  // all have looked before the first is done
    for (int k = 0; k < kThreads;) {
      const unsigned word = open[k >> 5] >> (k & 31);  // the next open row
      if (word == 0u) {
        k = (k | 31) + 1;
        continue;
      }
      k += __ffs(word);
      const int64_t r = r0 + static_cast<int64_t>(k - 1) * clusters;
      const char* logits = p.logits + r * p.row_stride_bytes;
      Sampler<DT, true> x(p, s, *cluster.map_shared_rank(&s, 0), *reinterpret_cast<Fine*>(dyn + sizeof(Shared)),
                          logits);
      x.place(dyn, rank, ranks);
      x.m = p.out.row_max[r];
      const int token = x.draw_any(fminf(fmaxf(p.uniform[r], 0.f), 0x1.fffffep-1f));
      if (rank == 0 && threadIdx.x == 0) {
        p.out.argmax[r] = token;
        p.out.conf[r] =
            token < 0 ? 0.f : ex2((load_logit(logits, DT, token) - x.m) * kLog2e) * p.out.conf[r];
      }
      cluster.sync();  // nobody leaves, or goes on, while its shared memory may be read
    }
    __syncthreads();
  }
}

// Shares a row of `tiles` tiles out to `ranks` CTAs; their shared memory.
// in_full: for draw_any too.
size_t lay_out(SampleParams& p, int64_t tiles, int ranks, bool in_full, int cap) {
  const int64_t own = (tiles + ranks - 1) / ranks;
  p.span_log2 = 0;
  while ((own >> p.span_log2) >= kMaxGroups) ++p.span_log2;
  const size_t groups = static_cast<size_t>((own >> p.span_log2) + 1);
  p.cap = cap;
  p.sums_at = static_cast<uint32_t>(
      sizeof(Shared) + std::max(in_full ? sizeof(Fine) : 0, align_up(groups * (2 * 128 + 4), 16)));
  p.keys_at = p.sums_at + static_cast<uint32_t>(in_full ? own * kLaneVecs : groups) * 8;
  return p.keys_at + static_cast<size_t>(cap) * (8 + 2);
}

template <int DT>
cudaError_t launch_rest(SampleParams p, int64_t rows, int64_t tiles, int sm_count,
                        cudaStream_t stream) {
  int ranks = 1;  // a tile or more each
  while (ranks < kMaxRanks && tiles > 2 * ranks) ranks *= 2;
  cudaError_t e = allow_smem<sample_rest_kernel<DT>>(200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t clusters = std::min<int64_t>(rows, std::max(1, 4 * sm_count / ranks));
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = lay_out(p, tiles, ranks, true, kCap);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_rest_kernel<DT>, p, static_cast<int>(rows));
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
  const int64_t tiles = (static_cast<int64_t>(sh.V) * es + 16 * kTileVecs - 1) / (16 * kTileVecs) + 1;
  int ranks = 1;
  while (ranks < kMaxRanks && rows * ranks * 2 <= 4 * static_cast<int64_t>(sm_count) &&
         tiles >= 2 * ranks)
    ranks *= 2;
  // Rows are left open only where the sum of all weights counts, and not by clusters of four and more or of
  // whole rows: these take the exact passes at once (32 rows of 1500 to 120000, nothing open: 8 to 9 us, with
  // the second kernel 10 to 11).  A CTA or two would take longer over a row than the second kernel's eight
  // (200 rows of 120000 with a few open: 83 us, with it 46), except where all rows are open because they are
  // flat: what clusters of two cannot list they do at once too (200 such rows: 319 us, else 482).
  p.at_once = p.top_k < p.V || (p.top_p == 1.0 && p.log_min_p > -INFINITY) || ranks >= 4 ||
              (ranks == 2 && tiles <= 4);
  const size_t smem = lay_out(p, tiles, ranks, p.at_once || ranks > 1, !p.at_once && p.top_p == 1.0 ? 0 : kCap);
  cudaError_t e;
  if (sh.dtype == DLLM_BF16)
    e = ranks > 1 ? launch<DLLM_BF16, true>(p, rows, ranks, smem, stream)
                  : launch<DLLM_BF16, false>(p, rows, ranks, smem, stream);
  else
    e = ranks > 1 ? launch<DLLM_F32, true>(p, rows, ranks, smem, stream)
                  : launch<DLLM_F32, false>(p, rows, ranks, smem, stream);
  if (e != cudaSuccess || p.at_once) return e;
  return sh.dtype == DLLM_BF16 ? launch_rest<DLLM_BF16>(p, rows, tiles, sm_count, stream)
                               : launch_rest<DLLM_F32>(p, rows, tiles, sm_count, stream);
}

}  // namespace dllm

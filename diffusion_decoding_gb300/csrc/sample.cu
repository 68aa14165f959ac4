// One token per open row of a block, drawn from the row's filtered softmax (temperature, top-k,
// top-p, min-p) with a given uniform number, beside the row's statistics.
//
// Candidates are ordered by falling logit, lower ids first among equals; every filter keeps a prefix
// of that order (a "cut": the last candidate kept), so the tightest cut holds.  The draw walks the
// kept candidates by rising id.  All comparisons of masses are of exact integer sums
// (exp_fixed.cuh), so a row's token does not depend on how its work was split.
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
constexpr int kLaneVecs = 8;                // 16-byte vectors a lane takes of a tile
constexpr int kTileVecs = 32 * kLaneVecs;   // a tile: 4 KB of a row, one warp's
constexpr int kCap = 1024;                  // candidates that are listed and ordered
constexpr int kListK = 512;                 // largest top_k that is tried with a list
constexpr int kFew = 128;                   // candidates ordered by counting, more by sorting
constexpr int kMaxGroups = 256;             // chunks of a CTA / 32
constexpr int kQueue = kCap;                // chunks that are looked through again
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
  uint32_t tops_bytes, sums_at;  // in shared memory
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
  uint64_t mass;     // weights, those of light chunks in 32 bits
  uint64_t light;    // of that: light chunks
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
  int coarse[kCoarseBins];
  uint64_t keys[kCap];      // candidates: ~order(z) << 32 | id
  ulonglong2 few[kFew];     // key, weight
  int queued;
  uint16_t queue[kQueue];   // chunks
  uint64_t goal, goal_error;  // what one thread worked out for all: a mass in units
  float least, from;
};
// The histogram of all weights, where the chunk sums were.
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
  Fine& fine;
  uint64_t* sums;   // [tiles of a CTA], behind fine
  float* tops;      // [groups * 32] maximum of a chunk
  float* masses;    // [groups * 32] weights of a chunk, to the reference refs[group]; where fine is
  float* refs;      // [groups]
  Row<DT> row;
  int rank, ranks;
  int tile0, tiles, groups;
  float m, total;   // of the row: maximum, sum of exp(z - m)
  float highest;    // of this thread's elements

  __device__ __forceinline__ Sampler(const SampleParams& p_, Shared& s_, Shared& f_, Fine& fine_,
                                     const char* r)
      : p(p_), s(s_), first(f_), fine(fine_), row(r, p_.V) {}

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
  // (A vector at a time: unrolled over a tile, an f of fifty instructions runs out of the instruction
  // cache, and a row takes 50 us instead of 20.)
  template <typename F>
  __device__ __forceinline__ void each_of_tile(int tile, F f) const {
    const int v0 = tile * kTileVecs + (threadIdx.x & 31);
    uint4 next = row.load(v0);
#pragma unroll 1
    for (int u = 0; u < kLaneVecs; ++u) {
      const uint4 q = next;
      if (u + 1 < kLaneVecs) next = row.load(v0 + 32 * (u + 1));
      float x[Row<DT>::VEC];
      unpack_vec<DT>(q, x);
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
  // 2^(x k - ref k) is computed as 2^(x k - hi) * rest.
  struct Scale {
    float k, hi, rest;
    bool far;  // hi is no use
    __device__ __forceinline__ explicit Scale(float k_) : k(k_), hi(0.f), rest(1.f), far(false) {}
    __device__ __forceinline__ void set(float r) {
      hi = r * k;
      far = !(fabsf(hi) < 0x1p100f);
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
  // (logits so large that ref * k overflows, or nearly)
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

  // The weights of this CTA's part by groups, and how much of that is known to 32 bits only: all of it,
  // or (kRefine) what lies in chunks that weigh little; the others are summed up element by element.
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
    if (lane == 0) s.warp_mass[warp] = mass, s.warp_light[warp] = light;
    __syncthreads();
    if (threadIdx.x == 0) {
      mass = light = 0;
      for (int w = 0; w < kWarps; ++w) mass += s.warp_mass[w], light += s.warp_light[w];
      s.mine.mass = mass;
      s.mine.light = light;
    }
    __syncthreads();
  }
  static constexpr float kHeavy = 0x1p-8f;  // of this CTA's weights
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
        if (at < kQueue) s.queue[at] = static_cast<uint16_t>(g * 32 + lane);
      }
    }
    __syncthreads();
    // more chunks than the list holds: no need to look
    const int queued = s.queued;
    if (queued > kQueue) {
      if (threadIdx.x == 0) atomicAdd(&first.ctl.listed, kCap + 1);
      return;
    }
    for (int k = threadIdx.x; k < queued * kLaneVecs; k += kThreads) {
      const int chunk = s.queue[k / kLaneVecs], g = chunk >> 5;
      const int t1 = min((g + 1) << p.span_log2, tiles);
      for (int tile = g << p.span_log2; tile < t1; ++tile) {
        const int vec = (tile0 + tile) * kTileVecs + 32 * (k % kLaneVecs) + (chunk & 31);
        const uint4 q = row.load(vec);
        if (!(vec_max<DT>(q) >= t)) continue;
        float x[Row<DT>::VEC];
        unpack_vec<DT>(q, x);
#pragma unroll
        for (int j = 0; j < Row<DT>::VEC; ++j)
          if (x[j] >= t && x[j] > -INFINITY) append(x[j], row.id(vec) + j);
      }
    }
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
      const uint64_t key = s.keys[threadIdx.x];
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

  // The same for up to kCap candidates, by sorting.
  __device__ __noinline__ int draw_listed(int n, float u, uint64_t goal_p, uint64_t error, float least,
                                          bool reaches) {
    constexpr int kEach = kCap / kThreads;
    sort_list(n);
    uint64_t w[kEach], mass = 0;
    int count = 0;
    if (threadIdx.x == 0) s.ctl.bin = n - 1, s.ctl.lo = 0u, s.ctl.found = -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int at = threadIdx.x * kEach + k;
      w[k] = at < n ? weight(listed_z(at)) : 0;
      mass += w[k];
    }
    block_scan(mass, count);
    const int limit = min(n, p.top_k);
    if (p.top_p < 1.0) {
      uint64_t upto = mass;
      if (p.top_k < p.V) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          upto += w[k];
          if (threadIdx.x * kEach + k == limit - 1)
            s.goal = static_cast<uint64_t>(ceil(p.top_p * static_cast<double>(upto)));
        }
        __syncthreads();
        goal_p = s.goal;
        upto = mass;
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int at = threadIdx.x * kEach + k;
        const uint64_t before = upto;
        upto += w[k];
        if (at >= n) continue;
        if (before < goal_p && upto >= goal_p) s.ctl.bin = at;
        if (error != 0 && ((upto + error >= goal_p && upto <= goal_p + error) ||
                           (reaches && at == limit - 1 && upto < goal_p + error)))
          s.ctl.lo = 1u;
      }
      __syncthreads();
      if (s.ctl.lo != 0u) return -2;
    }
    const int last = min(s.ctl.bin, limit - 1);
    __syncthreads();
    // the kept by id: key id << 32 | order(z)
    uint64_t keys[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int at = threadIdx.x * kEach + k;
      const bool keep = at <= last && listed_z(at) >= least;
      keys[k] = keep ? static_cast<uint64_t>(listed_id(at)) << 32 | order_of(listed_z(at)) : ~uint64_t{0};
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int at = threadIdx.x * kEach + k;
      if (at <= last) s.keys[at] = keys[k];
    }
    __syncthreads();
    sort_list(last + 1);
    mass = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int at = threadIdx.x * kEach + k;
      const bool there = at <= last && s.keys[at] != ~uint64_t{0};
      w[k] = there ? weight(of_order(static_cast<uint32_t>(s.keys[at]))) : 0;
      mass += w[k];
    }
    const uint64_t own = mass;
    block_scan(mass, count);
    if (threadIdx.x == kThreads - 1)
      s.goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(mass + own));
    __syncthreads();
    const uint64_t goal = s.goal;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const bool was = mass > goal;
      mass += w[k];
      if (!was && mass > goal) s.ctl.found = static_cast<int>(s.keys[threadIdx.x * kEach + k] >> 32);
    }
    __syncthreads();
    return s.ctl.found;
  }

  // The id in tiles [t, t1) at which the sum of f(z, id) by rising id, `before` before them, exceeds
  // `goal` (it does); by the whole CTA, a tile at a time, a warp each 32 of its vectors.  -2 where that
  // sum comes within `error` of the goal before or behind the token.  T: uint64_t, or float for weights
  // relative to the largest.
  template <typename T, typename F>
  __device__ __forceinline__ void find_in_tiles(int t, int t1, T before, T goal, T error, F f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* of_warp = reinterpret_cast<T*>(s.warp_mass);
    for (; t < t1; ++t) {
      const int vec = (tile0 + t) * kTileVecs + 32 * warp + lane;
      float x[Row<DT>::VEC];
      unpack_vec<DT>(row.load(vec), x);
      T w[Row<DT>::VEC], sum = 0;
#pragma unroll
      for (int j = 0; j < Row<DT>::VEC; ++j) w[j] = f(x[j], row.id(vec) + j), sum += w[j];
      T upto = warp_scan(sum);
      if (lane == 31) of_warp[warp] = upto;
      __syncthreads();
      T from = before;
      for (int k = 0; k < kWarps; ++k) {
        if (k == warp) from = before;
        before += of_warp[k];
      }
      upto += from;
      if (upto > goal && !(upto - sum > goal)) {
        upto -= sum;
#pragma unroll
        for (int j = 0; j < Row<DT>::VEC; ++j) {
          const T low = upto;
          upto += w[j];
          if (!(low > goal) && upto > goal && w[j] > 0 && (error == 0 || (upto > goal + error && low + error < goal)))
            first.ctl.found = row.id(vec) + j;
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

  // No filter: the group of tiles, then the token in it, by the weights of chunks; -2 where their error
  // leaves either open.
  template <bool kRefine>
  __device__ __forceinline__ int draw_whole(float u) {
    constexpr float kOfUnit = 1.f / static_cast<float>(int64_t{1} << kWeightBits);
    if (threadIdx.x == 0) {
      uint64_t before = 0, all = 0, light = 0;
      for (int r = 0; r < ranks; ++r) {
        const Summary& o = of(r).mine;
        if (r < rank) before += o.mass;
        all += o.mass;
        light += o.light;
      }
      s.goal = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(all));
      // u * all, the sum before a tile and the sum in it
      s.goal_error = static_cast<uint64_t>(2.0 * kError * static_cast<double>(light)) + 2 * kRounding * ranks;
      s.group_before = before;
      if (rank == 0) s.ctl.found = -2;
    }
    sync();
    const uint64_t goal = s.goal, error = s.goal_error;
    uint64_t before = s.group_before;
    if (before <= goal && before + s.mine.mass > goal) {
      __syncthreads();
      if (threadIdx.x < 32) find_group(sums, groups, before, goal);
      __syncthreads();
      const int group = s.group;
      before = s.group_before;
      const int t0 = group << p.span_log2, t1 = min((group + 1) << p.span_log2, tiles);
      if constexpr (kRefine)
        find_in_tiles<uint64_t>(t0, t1, before, goal, error, [&](float z, int) { return weight(z); });
      else
        find_in_tiles<float>(t0, t1, 0.f, static_cast<float>(goal - before) * kOfUnit,
                             static_cast<float>(error) * kOfUnit,
                             [&](float z, int) { return ex2((z - m) * p.t.hi); });
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
    set_goal([&] { s.goal = goal_of(all); });
    const uint64_t goal = s.goal;
    if (before <= goal && before + s.total[0] > goal) {
      __syncthreads();
      if (warp == 0) find_group(sums, tiles, before, goal);
      __syncthreads();
      find_in_tiles<uint64_t>(s.group, s.group + 1, s.group_before, goal, uint64_t{0}, f);
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
  __device__ __forceinline__ void histogram() {
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
      atomicAdd(&fine.bins[b], 1);
    });
    sync();
    if (rank == 0 && ranks > 1) {
      for (int b = threadIdx.x; b < kBins; b += kThreads) {
        for (int r = 1; r < ranks; ++r) {
          const Fine& o = *cg::this_cluster().map_shared_rank(&fine, r);
          fine.bins_lo_hi[b] += o.bins_lo_hi[b];
          fine.bins[b] += o.bins[b];
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
  // Warp 0: what top_p has to reach of the sum of all weights, and how far that may be off.
  __device__ __forceinline__ void set_mass_goal() {
    if (threadIdx.x == 0) {
      uint64_t all = 0, light = 0;
      for (int r = 0; r < ranks; ++r) all += of(r).mine.mass, light += of(r).mine.light;
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

  // The token by passes over all weights, whatever the filters keep.
  __device__ __noinline__ int draw_any(float u) {
    Cut cut{-INFINITY, INT_MAX};
    sync();  // what the chunks' sums were is overwritten
    const bool by_k = p.top_k < p.V, by_p = p.top_p < 1.0;
    if (by_k || by_p) {
      histogram();
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
    if (by_k && p.top_k <= kListK) {
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
    if (by_mass) {
      weigh_chunks<false>();
      if (!by_p) {
        sync();
        int token = draw_whole<false>(u);
        if (token == -2) {
          weigh_chunks<true>();
          sync();
          token = draw_whole<true>(u);
        }
        return token;
      }
      coarse_histogram<true>(m, false);
      sync();
      if (threadIdx.x < 32) {
        set_mass_goal();
        const float all = static_cast<float>(s.goal);
        int b0, b1;
        coarse_reach(
            [&](int b) {
              int n = 0;
              for (int r = 0; r < ranks; ++r) n += of(r).coarse[b];
              return static_cast<float>(n) * ex2(b * (-1.f / kCoarse) - 12.f);
            },
            all * 0x1.002p-42f, INFINITY, b0, b1);
        if (threadIdx.x == 0) s.from = b0 < kCoarseBins ? logit_of(m, b0) : -INFINITY;
      }
      __syncthreads();
      goal = s.goal;
      error = s.goal_error;
      t = fmaxf(s.from, least);
      reaches = s.from > least;
    } else if (by_k) {
      if (p.top_k <= kListK) {
        float some = INFINITY, all = -INFINITY;
        for (int r = 0; r < ranks; ++r) some = fminf(some, of(r).mine.some), all = fmaxf(all, of(r).mine.all);
        // what lies further below weighs nothing
        t = fmaxf(fmaxf(some, all), logit_of(m, kCoarseBins - 1));
      }
      if (!by_p) t = fmaxf(t, least);
    } else {
      t = least;
    }
    if (t > -INFINITY || p.V <= kCap) {
      list_from(t);
      sync();
      const int n = first.ctl.listed;
      if (n > 0 && n <= kCap) {
        if (rank == 0) {
          const int token = n <= kFew ? draw_few(n, u, goal, error, least, reaches)
                                      : listed(n, u, goal, error, least, reaches);
          if (threadIdx.x == 0) s.ctl.hi = static_cast<uint32_t>(token);
        }
        if (!by_mass) return rank == 0 ? static_cast<int>(s.ctl.hi) : -1;
        sync();
        if (static_cast<int>(first.ctl.hi) != -2) return static_cast<int>(first.ctl.hi);
        // once more, with the sum of weights known better
        weigh_chunks<true>();
        sync();
        if (rank != 0) return -1;
        if (threadIdx.x < 32) set_mass_goal();
        __syncthreads();
        goal = s.goal;
        error = s.goal_error;
        return n <= kFew ? draw_few(n, u, goal, error, least, reaches)
                         : listed(n, u, goal, error, least, reaches);
      }
      sync();
    }
    if (by_mass) return -2;
    return in_full(u);
  }
  __device__ __forceinline__ int listed(int n, float u, uint64_t goal, uint64_t error, float least,
                                        bool reaches) const {
    Sampler copy(*this);
    return copy.draw_listed(n, u, goal, error, least, reaches);
  }
  // (on a copy, so that the members stay in registers here)
  __device__ __forceinline__ int in_full(float u) const {
    Sampler copy(*this);
    return copy.draw_any(u);
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
  Fine& fine = *reinterpret_cast<Fine*>(dyn + sizeof(Shared) + p.tops_bytes);
  Sampler<DT, kCluster> x(p, s, *first, fine, logits);
  x.rank = rank;
  x.ranks = ranks;
  const int tiles = (x.row.vecs + kTileVecs - 1) / kTileVecs;
  x.tile0 = static_cast<int>(static_cast<int64_t>(tiles) * rank / ranks);
  x.tiles = static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / ranks) - x.tile0;
  x.groups = (x.tiles + (1 << p.span_log2) - 1) >> p.span_log2;
  x.tops = reinterpret_cast<float*>(dyn + sizeof(Shared));
  x.masses = reinterpret_cast<float*>(&fine);
  x.refs = x.masses + x.groups * 32;
  x.sums = reinterpret_cast<uint64_t*>(dyn + p.sums_at);
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
__global__ void __launch_bounds__(kThreads, 4) sample_rest_kernel(const __grid_constant__ SampleParams p,
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
      x.rank = rank;
      x.ranks = ranks;
      const int tiles = (x.row.vecs + kTileVecs - 1) / kTileVecs;
      x.tile0 = static_cast<int>(static_cast<int64_t>(tiles) * rank / ranks);
      x.tiles = static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / ranks) - x.tile0;
      x.sums = reinterpret_cast<uint64_t*>(dyn + sizeof(Shared) + sizeof(Fine));
      x.m = p.out.row_max[r];
      const int token = x.draw_any(fminf(fmaxf(p.uniform[r], 0.f), 0x1.fffffep-1f));
      if (rank == 0 && threadIdx.x == 0) {
        p.out.argmax[r] = token;
        p.out.conf[r] =
            token < 0 ? 0.f : ex2((load_logit(logits, DT, token) - x.m) * kLog2e) * p.out.conf[r];
      }
    }
    cluster.sync();  // nobody leaves, or looks again, while shared memory may be read
  }
}

template <int DT>
cudaError_t launch_rest(const SampleParams& p, int64_t rows, int64_t tiles, int sm_count,
                        cudaStream_t stream) {
  constexpr int kRanks = 8;
  cudaError_t e = allow_smem<sample_rest_kernel<DT>>(200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t clusters = std::min<int64_t>(rows, std::max(1, 4 * sm_count / kRanks));
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kRanks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared) + sizeof(Fine) + static_cast<size_t>(tiles / kRanks + 2) * 8;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kRanks;
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
  while (ranks < 8 && rows * ranks * 2 <= 4 * static_cast<int64_t>(sm_count) &&
         tiles >= 2 * ranks)
    ranks *= 2;
  // a CTA's tiles (rows may begin anywhere in a vector), in groups
  const int64_t own = (tiles + ranks - 1) / ranks;
  while ((own >> p.span_log2) >= kMaxGroups) ++p.span_log2;
  const size_t groups = static_cast<size_t>((own >> p.span_log2) + 1);
  p.tops_bytes = static_cast<uint32_t>(align_up(groups * 128, 16));
  const size_t shared_part = std::max(sizeof(Fine), align_up(groups * 132, 16));
  p.sums_at = static_cast<uint32_t>(sizeof(Shared) + p.tops_bytes + align_up(shared_part, 16));
  const size_t smem = p.sums_at + static_cast<size_t>(own + 1) * 8;
  cudaError_t e;
  if (sh.dtype == DLLM_BF16)
    e = ranks > 1 ? launch<DLLM_BF16, true>(p, rows, ranks, smem, stream)
                  : launch<DLLM_BF16, false>(p, rows, ranks, smem, stream);
  else
    e = ranks > 1 ? launch<DLLM_F32, true>(p, rows, ranks, smem, stream)
                  : launch<DLLM_F32, false>(p, rows, ranks, smem, stream);
  // rows are left open only where the sum of all weights counts
  const bool by_mass = p.top_k == p.V && (p.top_p < 1.0 || p.log_min_p == -INFINITY);
  if (e != cudaSuccess || !by_mass) return e;
  return sh.dtype == DLLM_BF16 ? launch_rest<DLLM_BF16>(p, rows, tiles, sm_count, stream)
                               : launch_rest<DLLM_F32>(p, rows, tiles, sm_count, stream);
}

}  // namespace dllm

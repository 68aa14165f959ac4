// Eviction from the 4-bit cache by accumulated attention weight: per sequence the `budget` entries to
// keep are chosen, and those of them that lie behind the new length move into the places of dropped
// ones before it.  Attention over a cache does not depend on the order of its entries (keys are
// rotated before they are stored), so no other entry has to move: sources lie behind the new length
// and destinations before it, and all copies are independent.
//
// kv4_evict_select_kernel, a cluster of CTAs a sequence: a histogram of the upper 11 bits of the weights'
// order finds the bin in which the K-th largest weight lies; the entries of that bin are listed and
// sorted in one CTA (a bin of more entries than the list holds is narrowed down by the other bits, and
// equal weights by counting in order), which gives the border: the last entry kept.  Kept and dropped
// entries are then numbered by counting in order, and the moves left in the workspace.
// kv4_evict_move_kernel copies 16 bytes of codes and a param word a thread and move, two moves at a time and
// the next two's loads before these are stored, and finishes slots and weights of the entries it moves.
//
// The selection is bound by its chain of barriers (one CTA a sequence 14 us for 8192 entries in registers;
// clusters of smaller CTAs 24, as each reads the others' histograms), the copies by memory in sectors: an
// entry's param words of a head are 8 bytes of a 32-byte sector.  32 sequences of up to 8192 entries cut to
// 4096: 46 us in all, 127 + 52 MB of DRAM traffic in the copies (more moves a warp at a time 46 to 90); one
// of 65536 cut to 16384 23 us; a short one 12, the host's time for two launches.
#include <limits.h>

#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dllm {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxThreads = 1024;
constexpr int kMaxRanks = 8;
constexpr int kHeld = 8;         // entries a thread keeps in registers
constexpr int kDigits = 2048;    // upper 11 bits, middle 11, lower 10
constexpr int kList = 2048;      // entries that are listed
constexpr int kSorted = 64;      // entries that are sorted as they are

struct EvictParams {
  const float* weights;
  int64_t weights_stride;
  const int32_t* lens;
  int max_len, budget, first, last;
  int32_t* slots;
  int64_t slots_stride;
  int32_t* lens_out;
  float* weights_out;
  int64_t weights_out_stride;
  // moves: entry from[b * most + k] -> to[b * most + k], k < count[b]
  int32_t* count;
  int32_t* from;
  int32_t* to;
  int64_t most;
};

// Rising order of weights as integers; a NaN comes first, both zeros are alike.  weight_of: back.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return w == w ? o : 0u;
}
__device__ __forceinline__ float weight_of(uint32_t o) {
  return o == 0u ? NAN : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

struct Shared {
  int bins[kDigits];
  uint64_t list[kList];            // ~order << 32 | entry
  int warp_total[kMaxThreads / 32];
  int digit, above, in_digit;      // the digit found, entries above it and in it
  int listed;
  int2 mine;                       // this CTA's holes and tails (or equal weights), read by the others
  int2 of_warp[kMaxThreads / 32];
  uint32_t border;                 // order of the last entry kept
  int border_entry;
};

// kHeldAll: a thread's entries fit its registers.
template <int kThreads, bool kHeldAll>
struct Selector {
  static constexpr int kWarps = kThreads / 32;
  const EvictParams& p;
  Shared& s;
  int rank, ranks, lane, warp;
  const float* w;
  int len, from, to;  // entries of this warp: [from, to)
  uint32_t held[kHeldAll ? kHeld : 1];  // order of the weights
  uint32_t open;  // bit k: entry k of the thread may be dropped

  __device__ __forceinline__ Selector(const EvictParams& p_, Shared& s_) : p(p_), s(s_) {}
  __device__ __forceinline__ Shared& of(int r) const { return *cg::this_cluster().map_shared_rank(&s, r); }
  __device__ __forceinline__ void sync() const {
    if (ranks > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  }
  // entry j may be dropped
  __device__ __forceinline__ bool may_go(int j) const {
    return static_cast<unsigned>(j - p.first) < static_cast<unsigned>(max(len - p.last - p.first, 0));
  }

  // f(j, order of the weight, whether the entry may be dropped) of the warp's entries, 32 at a time and
  // all lanes together.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (kHeldAll) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (from + 32 * k < to) f(from + 32 * k + lane, held[k], (open >> k & 1u) != 0u);
    } else {
      for (int j0 = from; j0 < to; j0 += 32) {
        const int j = j0 + lane;
        f(j, j < len ? order_of(w[j]) : 0u, may_go(j));
      }
    }
  }
  __device__ __forceinline__ void load() {
    if constexpr (kHeldAll) {
      open = 0u;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int j = from + 32 * k + lane;
        held[k] = j < min(len, to) ? order_of(w[j]) : 0u;
        open |= may_go(j) && j < to ? 1u << k : 0u;
      }
    }
  }

  // Histogram of the digit at `shift` of the open entries whose upper bits are `known`, over the row.
  __device__ __forceinline__ void histogram(uint32_t known, uint32_t mask, int shift, uint32_t digits) {
    for (int d = threadIdx.x; d < kDigits; d += kThreads) s.bins[d] = 0;
    __syncthreads();
    each([&](int, uint32_t key, bool may) {
      if (may && (key & mask) == known) atomicAdd(&s.bins[key >> shift & digits], 1);
    });
    sync();
  }
  // The digit in which the count from the top reaches `need`, and the entries above it and in it; by the
  // histograms of all CTAs, or (kOwn) this one's alone.
  template <bool kOwn>
  __device__ __forceinline__ void find_digit(int need) {
    constexpr int kEach = kDigits / kThreads;
    const int top = kDigits - 1 - threadIdx.x * kEach;  // this thread's digits from the top
    int own[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; k += 2) {
      int2 o = *reinterpret_cast<const int2*>(&s.bins[top - k - 1]);
      if (!kOwn && ranks > 1) {
        o = make_int2(0, 0);
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) {
          if (r >= ranks) break;
          // (each CTA begins with its own: they do not all read the same one's at a time)
          const int2 y = *reinterpret_cast<const int2*>(&of((rank + r) & (ranks - 1)).bins[top - k - 1]);
          o.x += y.x;
          o.y += y.y;
        }
      }
      own[k] = o.y;
      own[k + 1] = o.x;
      sum += o.x + o.y;
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s.warp_total[warp] = upto;
    __syncthreads();
    const int before = lane < warp ? s.warp_total[lane] : 0;
    int above = upto - sum + static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(before)));
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (above < need && above + own[k] >= need) s.digit = top - k, s.above = above, s.in_digit = own[k];
      above += own[k];
    }
    __syncthreads();
  }
  // Counts of this warp in the order of entries: those of the warps before it, over the whole row.
  __device__ __forceinline__ int2 before_of(int2 count) {
    if (lane == 0) s.of_warp[warp] = count;
    __syncthreads();
    int2 own = lane < kWarps ? s.of_warp[lane] : make_int2(0, 0);
    const int2 all = make_int2(static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(own.x))),
                               static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(own.y))));
    if (lane >= warp) own = make_int2(0, 0);
    if (ranks > 1) {
      if (threadIdx.x == 0) s.mine = all;
      sync();
      if (lane < rank) {
        const int2 o = of(lane).mine;
        own.x += o.x;
        own.y += o.y;
      }
    }
    return make_int2(static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(own.x))),
                     static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(own.y))));
  }

  // The last entry kept of the open ones, `need` of which are kept, to border and border_entry.
  __device__ __forceinline__ void find_border(int need, uint32_t& border, int& border_entry) {
    if (need == 0) {
      border = 0xFFFFFFFFu;
      border_entry = -1;
      return;
    }
    uint32_t mask = 0u;
    border = 0u;
    if (threadIdx.x == 0) s.listed = 0;
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
      if (mask != 0u) sync();  // the bins are counted anew
      histogram(border, mask, shift, shift == 0 ? 1023u : 2047u);
      find_digit<false>(need);
      border |= static_cast<uint32_t>(s.digit) << shift;
      mask = 0xFFFFFFFFu << shift;
      need -= s.above;
      if (s.in_digit <= kList) {
        if (ranks == 1) {
          each([&](int j, uint32_t key, bool may) {
            if (may && (key & mask) == border)
              s.list[atomicAdd(&s.listed, 1)] = static_cast<uint64_t>(~key) << 32 | static_cast<uint32_t>(j);
          });
        } else {
          list_far(border, mask);
        }
        sync();
        if (rank == 0) {
          const uint64_t last = nth_listed(need - 1);
          if (threadIdx.x == 0)
            s.border = ~static_cast<uint32_t>(last >> 32), s.border_entry = static_cast<int>(last & 0xFFFFFFFFu);
        }
        sync();
        border = of(0).border;
        border_entry = of(0).border_entry;
        return;
      }
    }
    // the need-th entry of that weight
    int equal = 0;
    each([&](int, uint32_t key, bool may) { equal += __popc(__ballot_sync(kFull, may && key == border)); });
    int seen = before_of(make_int2(equal, 0)).x;
    each([&](int j, uint32_t key, bool may) {
      const unsigned hit = __ballot_sync(kFull, may && key == border);
      const int upto = seen + __popc(hit & ((2u << lane) - 1u));
      if ((hit >> lane & 1u) && upto == need) of(0).border_entry = j;
      seen += __popc(hit);
    });
    sync();
    border_entry = of(0).border_entry;
    sync();
  }
  // The entries of that digit to the first CTA's list (a place for all of a warp's, not an atomic operation
  // on another CTA's memory for every entry).
  __device__ __forceinline__ void list_far(uint32_t known, uint32_t mask) {
    Shared& first = of(0);
    int mine = 0;
    each([&](int, uint32_t key, bool may) { mine += __popc(__ballot_sync(kFull, may && (key & mask) == known)); });
    int at = 0;
    if (lane == 0 && mine > 0) at = atomicAdd(&first.listed, mine);
    at = __shfl_sync(kFull, at, 0);
    if (mine > 0) {
      each([&](int j, uint32_t key, bool may) {
        const bool in = may && (key & mask) == known;
        const unsigned hit = __ballot_sync(kFull, in);
        if (in)
          first.list[at + __popc(hit & ((1u << lane) - 1u))] =
              static_cast<uint64_t>(~key) << 32 | static_cast<uint32_t>(j);
        at += __popc(hit);
      });
    }
  }
  // First CTA: element n of the list in rising order.  A long list is cut down to those that share the
  // n-th's middle bits first.
  __device__ __forceinline__ uint64_t nth_listed(int n) {
    int count = s.listed;
    if (count > kSorted) {
      constexpr int kEach = kList / kThreads;
      for (int d = threadIdx.x; d < kDigits; d += kThreads) s.bins[d] = 0;
      uint64_t mine[kEach];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int at = threadIdx.x + k * kThreads;
        mine[k] = at < count ? s.list[at] : 0;
        if (at < count) atomicAdd(&s.bins[~static_cast<uint32_t>(mine[k] >> 32) >> 10 & 2047u], 1);
      }
      if (threadIdx.x == 0) s.listed = 0;
      __syncthreads();
      find_digit<true>(n + 1);
      n -= s.above;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        if (threadIdx.x + k * kThreads < count &&
            (~static_cast<uint32_t>(mine[k] >> 32) >> 10 & 2047u) == static_cast<uint32_t>(s.digit))
          s.list[atomicAdd(&s.listed, 1)] = mine[k];
      }
      __syncthreads();
      count = s.listed;
    }
    int size = 32;
    while (size < count) size *= 2;
    for (int k = count + threadIdx.x; k < size; k += kThreads) s.list[k] = ~uint64_t{0};
    __syncthreads();
    for (int l = 2; l <= size; l *= 2) {
      for (int d = l / 2; d > 0; d /= 2) {
        for (int k = threadIdx.x; k < size / 2; k += kThreads) {
          const int i = 2 * k - (k & (d - 1));  // d is a power of two
          const uint64_t x = s.list[i], y = s.list[i + d];
          if ((x > y) == ((i & l) == 0)) s.list[i] = y, s.list[i + d] = x;
        }
        if (size > 64)
          __syncthreads();
        else if (warp == 0)
          __syncwarp();  // (it has all pairs)
        else
          break;
      }
    }
    __syncthreads();
    return s.list[n];
  }
};

template <int kThreads, bool kHeldAll>
__global__ void __launch_bounds__(kThreads) kv4_evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ __align__(16) Shared s;
  constexpr int kWarps = kThreads / 32;
  Selector<kThreads, kHeldAll> x{p, s};
  x.ranks = static_cast<int>(cg::this_cluster().num_blocks());
  x.rank = static_cast<int>(cg::this_cluster().block_rank());
  const int lane = x.lane = threadIdx.x & 31;
  x.warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int64_t b = blockIdx.x / x.ranks;
  x.w = p.weights + b * p.weights_stride;
  const int len = x.len = p.lens ? max(0, min(p.lens[b], p.max_len)) : p.max_len;
  const int fresh = min(len, p.budget);
  int32_t* slots = p.slots + b * p.slots_stride;
  float* out = p.weights_out ? p.weights_out + b * p.weights_out_stride : nullptr;
  // every warp has as many entries, whole 32s
  const int warps = x.ranks * kWarps, chunks = (p.max_len + 31) / 32;
  const int64_t per = 32 * static_cast<int64_t>((chunks + warps - 1) / warps);
  const int64_t start = (x.rank * kWarps + x.warp) * per;
  x.from = static_cast<int>(min(start, static_cast<int64_t>(p.max_len)));
  x.to = static_cast<int>(min(start + per, static_cast<int64_t>(p.max_len)));
  uint32_t border = 0u;
  int border_entry = INT_MAX;  // all stay
  x.load();
  if (len > p.budget) x.find_border(p.budget - p.first - p.last, border, border_entry);
  auto stays = [&](int j, uint32_t key, bool may) {
    return may && len > p.budget ? key > border || (key == border && j <= border_entry) : j < len;
  };
  const unsigned below = (1u << lane) - 1u;
  int32_t* from = p.from + b * p.most;
  int32_t* to = p.to + b * p.most;
  // (what moves is the other kernel's: its slot, its weight here and where it goes)
  auto put = [&](int j, uint32_t key, bool stay, unsigned hs, unsigned ts, int& holes, int& tails) {
    const bool hole = hs >> lane & 1u, tail = ts >> lane & 1u;
    if (hole) to[holes + __popc(hs & below)] = j;
    if (tail) from[tails + __popc(ts & below)] = j;
    holes += __popc(hs);
    tails += __popc(ts);
    if (j < x.to && !tail) {
      slots[j] = stay ? j : -1;
      if (out && !hole) out[j] = stay ? weight_of(key) : 0.f;
    }
  };
  int holes = 0, tails = 0;
  if constexpr (kHeldAll) {
    unsigned hs[kHeld], ts[kHeld], stay = 0u;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int j = x.from + 32 * k + lane;
      const bool st = stays(j, x.held[k], (x.open >> k & 1u) != 0u) && j < x.to;
      stay |= st ? 1u << k : 0u;
      hs[k] = __ballot_sync(kFull, j < min(fresh, x.to) && !st);
      ts[k] = __ballot_sync(kFull, j >= fresh && st);
      holes += __popc(hs[k]);
      tails += __popc(ts[k]);
    }
    const int2 before = x.before_of(make_int2(holes, tails));
    holes = before.x;
    tails = before.y;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (x.from + 32 * k < x.to) put(x.from + 32 * k + lane, x.held[k], stay >> k & 1u, hs[k], ts[k], holes, tails);
  } else {
    auto count = [&](auto use) {
      x.each([&](int j, uint32_t key, bool may) {
        const bool st = stays(j, key, may);
        const unsigned hs = __ballot_sync(kFull, j < fresh && !st), ts = __ballot_sync(kFull, j >= fresh && st);
        use(j, key, st, hs, ts);
      });
    };
    count([&](int, uint32_t, bool, unsigned hs, unsigned ts) { holes += __popc(hs), tails += __popc(ts); });
    const int2 before = x.before_of(make_int2(holes, tails));
    holes = before.x;
    tails = before.y;
    count([&](int j, uint32_t key, bool st, unsigned hs, unsigned ts) { put(j, key, st, hs, ts, holes, tails); });
  }
  // as many holes as kept entries behind the new length: the last warp has counted them all
  if (x.rank == x.ranks - 1 && x.warp == kWarps - 1 && lane == 0) {
    p.count[b] = tails;
    p.lens_out[b] = fresh;
  }
  if (x.ranks > 1) x.sync();  // nobody leaves while its counts may be read
}

struct MoveParams {
  uint8_t* codes[2];
  uint16_t* params[2];
  const int32_t* table;
  int table_stride, pages, page_size, heads, groups;
  int units;           // groups of an entry: heads * 2 * groups
  int lanes_log2;      // lanes that copy one move: 32, or as many as it has units
  int rounds;          // of kSteps steps: a warp's moves
  EvictParams e;
  int64_t ctas_per_seq;
};

constexpr int kMoveThreads = 256;
constexpr int kSteps = 2;  // moves, or groups of them, that a warp copies at a time

// A warp has up to 32 moves: a lane looks up where one of them comes from and goes to, then all lanes
// copy, each its unit (16 bytes of codes and a param word) of kSteps moves at a time, the loads of the
// next ones before the stores of these.  An entry of fewer than 32 units shares the warp with others.
__global__ void __launch_bounds__(kMoveThreads, 4) kv4_evict_move_kernel(const __grid_constant__ MoveParams p) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int b = static_cast<int>(blockIdx.x / p.ctas_per_seq);
  const int64_t task = (blockIdx.x - b * p.ctas_per_seq) * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const int together = 32 >> p.lanes_log2;  // moves of a step
  const int steps = min(kSteps, 1 << p.lanes_log2);  // of a round
  const int moves = p.rounds * steps * together;
  const int64_t k0 = task * moves;
  // (no __ldg of what the kernel before has written: a load of constants may be moved before the wait)
  const int count = p.e.count[b];
  if (k0 >= count) return;
  const int here = static_cast<int>(min(static_cast<int64_t>(moves), count - k0));
  int64_t row[2] = {-1, -1};  // group 0 of head 0 of the lane's move, from and to
  if (lane < here) {
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;
    const int j0 = p.e.from[b * p.e.most + k0 + lane], j1 = p.e.to[b * p.e.most + k0 + lane];
    const int t0 = j0 / p.page_size, t1 = j1 / p.page_size;
    const int page0 = __ldg(table + t0), page1 = __ldg(table + t1);
    p.e.slots[b * p.e.slots_stride + j0] = j1;
    if (p.e.weights_out) {
      p.e.weights_out[b * p.e.weights_out_stride + j1] = p.e.weights[b * p.e.weights_stride + j0];
      p.e.weights_out[b * p.e.weights_out_stride + j0] = 0.f;
    }
    if (static_cast<unsigned>(page0) < static_cast<unsigned>(p.pages) &&
        static_cast<unsigned>(page1) < static_cast<unsigned>(p.pages)) {
      row[0] = (static_cast<int64_t>(page0) * p.heads * p.page_size + j0 - t0 * p.page_size) * p.groups;
      row[1] = (static_cast<int64_t>(page1) * p.heads * p.page_size + j1 - t1 * p.page_size) * p.groups;
    }
  }
  const int of_step = lane >> p.lanes_log2, rounds = (here + steps * together - 1) / (steps * together);
  struct Held {
    uint4 c[kSteps];
    uint16_t q[kSteps];
    int64_t dst[kSteps];  // -1: nothing
    uint4* codes;
    uint16_t* params;
  };
  int round = 0, unit = lane & ((1 << p.lanes_log2) - 1), ht = unit / p.groups;
  auto load = [&](Held& x) {
    const int64_t off = static_cast<int64_t>(ht >> 1) * p.page_size * p.groups + unit - ht * p.groups;
    x.codes = reinterpret_cast<uint4*>(p.codes[ht & 1]) + off;
    x.params = p.params[ht & 1] + off;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int m = (round * steps + i) * together + of_step;
      const int64_t src = __shfl_sync(kFull, row[0], m & 31);
      x.dst[i] = __shfl_sync(kFull, row[1], m & 31);
      if (i >= steps || m >= here || unit >= p.units) x.dst[i] = -1;
      if (x.dst[i] >= 0) x.c[i] = x.codes[src], x.q[i] = x.params[src];
    }
    if (++round == rounds) {
      round = 0;
      unit += 32;
      ht = unit / p.groups;
    }
  };
  auto store = [&](const Held& x) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (x.dst[i] >= 0) x.codes[x.dst[i]] = x.c[i], x.params[x.dst[i]] = x.q[i];
  };
  const int total = rounds * ((p.units + 31) / 32);
  Held a, z;
  load(a);
  for (int it = 0; it < total; it += 2) {
    if (it + 1 < total) load(z);
    store(a);
    if (it + 2 < total) load(a);
    if (it + 1 < total) store(z);
  }
}

int64_t most_moves(int max_len) { return (static_cast<int64_t>(max_len) / 2 + 64) / 64 * 64; }

}  // namespace

size_t kv4_evict_ws_bytes(int B, int max_len) {
  return kWsHeader + align_up(static_cast<size_t>(B) * 4, 256) +
         static_cast<size_t>(B) * static_cast<size_t>(most_moves(max_len)) * 8;
}

cudaError_t launch_kv4_evict(const dllm_kv4_cache& cache, const float* weights, int64_t weights_stride,
                             const int32_t* lens, int max_len, int budget, int first, int last,
                             int32_t* slots, int64_t slots_stride, int32_t* lens_out,
                             float* weights_out, int64_t weights_out_stride, int B, void* ws,
                             int sm_count, cudaStream_t stream) {
  EvictParams p{weights, weights_stride, lens,        max_len,     budget,
                first,   last,           slots,       slots_stride, lens_out,
                weights_out, weights_out_stride};
  char* at = static_cast<char*>(ws) + kWsHeader;
  p.most = most_moves(max_len);
  p.count = reinterpret_cast<int32_t*>(at);
  p.from = reinterpret_cast<int32_t*>(at + align_up(static_cast<size_t>(B) * 4, 256));
  p.to = p.from + B * p.most;
  // a CTA has up to eight entries a thread; a short sequence fewer threads (barriers of eight warps take
  // less time than of 32)
  const int threads = max_len <= 256 * kHeld ? 256 : kMaxThreads;
  int ranks = 1;
  while (ranks < kMaxRanks && max_len > ranks * threads * kHeld) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * ranks));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e =
      threads == 256 ? cudaLaunchKernelEx(&cfg, kv4_evict_select_kernel<256, true>, p)
      : max_len <= ranks * threads * kHeld
          ? cudaLaunchKernelEx(&cfg, kv4_evict_select_kernel<kMaxThreads, true>, p)
          : cudaLaunchKernelEx(&cfg, kv4_evict_select_kernel<kMaxThreads, false>, p);
  if (e != cudaSuccess || max_len <= budget) return e;
  MoveParams m{};
  m.codes[0] = cache.k_codes, m.codes[1] = cache.v_codes;
  m.params[0] = cache.k_params, m.params[1] = cache.v_params;
  m.table = cache.page_table;
  m.table_stride = cache.table_stride, m.pages = cache.pages, m.page_size = cache.page_size;
  m.heads = cache.heads;
  m.groups = cache.head_dim / 32;
  m.units = cache.heads * 2 * m.groups;
  m.e = p;
  const int64_t most = std::min<int64_t>(max_len - budget, budget);
  if (most == 0) return cudaSuccess;
  while (m.lanes_log2 < 5 && (1 << m.lanes_log2) < m.units) ++m.lanes_log2;
  // many moves a warp where there are many (what it looks up first is then a small part of its time), few
  // where that leaves SMs idle
  const int together = 32 >> m.lanes_log2;
  const int steps = std::min(kSteps, 1 << m.lanes_log2);
  m.rounds = std::min(2, (1 << m.lanes_log2) / steps);
  while (m.rounds > 1 && B * most < static_cast<int64_t>(8) * sm_count * m.rounds * steps * together) m.rounds /= 2;
  const int64_t per_cta = (kMoveThreads / 32) * m.rounds * steps * together;
  m.ctas_per_seq = (most + per_cta - 1) / per_cta;
  return launch_dependent(kv4_evict_move_kernel, dim3(static_cast<unsigned>(B * m.ctas_per_seq)),
                          dim3(kMoveThreads), 0, stream, m);
}

}  // namespace dllm

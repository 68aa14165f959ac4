// Eviction from the 4-bit cache by accumulated attention weight: per sequence the `budget` entries to
// keep are chosen, and those of them that lie behind the new length move into the places of dropped
// ones before it.  Attention over a cache does not depend on the order of its entries (keys are
// rotated before they are stored), so no other entry has to move: sources lie behind the new length
// and destinations before it, and all copies are independent.
//
// kv4_evict_select_kernel, a cluster a sequence: the K-th largest weight by a radix search (11 + 11 +
// 10 bits of the weights' order, histograms in shared memory, summed over the cluster), the places of
// kept and dropped entries by counting in order.  It leaves the list of moves in the workspace.
// kv4_evict_move_kernel, a warp a move: codes and params of all heads.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dllm {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxRanks = 8;
constexpr int kDigits = 2048;
constexpr int kDigitsPerThread = kDigits / kThreads;

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

// Rising order of weights as integers; a NaN comes first, both zeros are alike.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Shared {
  int bins[2][kDigits];
  int warp_total[kWarps];
  int digit, above;           // the digit found, entries above it
  int ties[kWarps];           // of each warp: entries of the border weight;
  int holes[kWarps], tails[kWarps];  // dropped before, kept behind the new length
};

struct Selector {
  const EvictParams& p;
  Shared& s;
  int rank, ranks, lane, warp;
  const float* w;
  int len, from, to;  // entries of this warp: [from, to)

  __device__ __forceinline__ const Shared& of(int r) const {
    return *cg::this_cluster().map_shared_rank(&s, r);
  }
  __device__ __forceinline__ void sync() const { cg::this_cluster().sync(); }
  __device__ __forceinline__ bool fixed(int j) const { return j < p.first || j >= len - p.last; }

  // The digit in which the count from the top reaches `need`, and the entries above it.
  __device__ __forceinline__ void find_digit(int buffer, int need) {
    int own[kDigitsPerThread], sum = 0;
    const int d0 = kDigits - 1 - threadIdx.x * kDigitsPerThread;  // from the top
#pragma unroll
    for (int k = 0; k < kDigitsPerThread; ++k) {
      own[k] = 0;
      for (int r = 0; r < ranks; ++r) own[k] += of(r).bins[buffer][d0 - k];
      sum += own[k];
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s.warp_total[warp] = upto;
    __syncthreads();
    int above = upto - sum;
    for (int k = 0; k < warp; ++k) above += s.warp_total[k];
#pragma unroll
    for (int k = 0; k < kDigitsPerThread; ++k) {
      if (above < need && above + own[k] >= need) s.digit = d0 - k, s.above = above;
      above += own[k];
    }
    __syncthreads();
  }
  // Sum of one count a warp over the warps before this one, in the order of their entries.
  __device__ __forceinline__ int before(int (Shared::*counts)[kWarps]) const {
    int sum = 0;
    for (int k = lane; k < rank * kWarps + warp; k += 32) sum += (of(k / kWarps).*counts)[k % kWarps];
    return static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(sum)));
  }
};

__global__ void __launch_bounds__(kThreads) kv4_evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ Shared s;
  Selector x{p, s};
  x.ranks = static_cast<int>(cg::this_cluster().num_blocks());
  x.rank = static_cast<int>(cg::this_cluster().block_rank());
  x.lane = threadIdx.x & 31;
  x.warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / x.ranks;
  x.w = p.weights + b * p.weights_stride;
  const int len = x.len = p.lens ? max(0, min(p.lens[b], p.max_len)) : p.max_len;
  const int fresh = min(len, p.budget);
  int32_t* slots = p.slots + b * p.slots_stride;
  float* out = p.weights_out ? p.weights_out + b * p.weights_out_stride : nullptr;
  // every warp has as many entries, whole 32s
  const int warps = x.ranks * kWarps, chunks = (p.max_len + 31) / 32;
  const int per = 32 * ((chunks + warps - 1) / warps);
  const int64_t start = static_cast<int64_t>(x.rank * kWarps + x.warp) * per;
  x.from = static_cast<int>(min(start, static_cast<int64_t>(p.max_len)));
  x.to = static_cast<int>(min(start + per, static_cast<int64_t>(p.max_len)));

  // the border: entries of a weight above it stay, of the border weight the first `ties`
  uint32_t border = 0u;
  int ties = 0;
  if (len > p.budget) {
    int need = p.budget - p.first - p.last;
    if (need == 0) {
      border = 0xFFFFFFFFu;
    } else {
      int shift = 21;
      for (int pass = 0; pass < 3; ++pass) {
        const int buffer = pass & 1;
        for (int d = threadIdx.x; d < kDigits; d += kThreads) s.bins[buffer][d] = 0;
        __syncthreads();
        const uint32_t known = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + (pass == 1 ? 11 : 10));
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        for (int j = x.from + x.lane; j < min(x.to, len); j += 32) {
          if (x.fixed(j)) continue;
          const uint32_t key = order_of(x.w[j]);
          if ((key & known) == (border & known)) atomicAdd(&s.bins[buffer][key >> shift & digits], 1);
        }
        x.sync();
        x.find_digit(buffer, need);
        border |= static_cast<uint32_t>(s.digit) << shift;
        need -= s.above;
        shift = pass == 0 ? 10 : 0;
      }
      ties = need;
    }
    // entries of the border weight before this warp's
    int mine = 0;
    for (int j = x.from + x.lane; j < x.to; j += 32)
      mine += j < len && !x.fixed(j) && order_of(x.w[j]) == border ? 1 : 0;
    mine = static_cast<int>(__reduce_add_sync(kFull, static_cast<unsigned>(mine)));
    if (x.lane == 0) s.ties[x.warp] = mine;
  }
  x.sync();
  const int ties_before = len > p.budget ? x.before(&Shared::ties) : 0;

  const unsigned below = (1u << x.lane) - 1u;
  // whether entry j stays; `seen` counts the warp's entries of the border weight
  auto stays = [&](int j, float w, int& seen) {
    bool stay = j < len;
    const bool open = stay && len > p.budget && !x.fixed(j);
    const uint32_t key = open ? order_of(w) : 0u;
    const unsigned equal = __ballot_sync(kFull, open && key == border);
    if (open) stay = key > border || (key == border && seen + __popc(equal & below) < ties);
    seen += __popc(equal);
    return stay;
  };
  int holes = 0, tails = 0, seen = ties_before;
  for (int j0 = x.from; j0 < x.to; j0 += 32) {
    const int j = j0 + x.lane;
    const bool stay = stays(j, j < len ? x.w[j] : 0.f, seen);
    holes += __popc(__ballot_sync(kFull, j < fresh && !stay));
    tails += __popc(__ballot_sync(kFull, j >= fresh && stay));
  }
  if (x.lane == 0) s.holes[x.warp] = holes, s.tails[x.warp] = tails;
  x.sync();
  holes = x.before(&Shared::holes);
  tails = x.before(&Shared::tails);
  seen = ties_before;
  int32_t* from = p.from + b * p.most;
  int32_t* to = p.to + b * p.most;
  for (int j0 = x.from; j0 < x.to; j0 += 32) {
    const int j = j0 + x.lane;
    const float w = j < len ? x.w[j] : 0.f;
    const bool stay = stays(j, w, seen);
    const bool hole = j < fresh && !stay, tail = j >= fresh && stay;
    const unsigned hs = __ballot_sync(kFull, hole), ts = __ballot_sync(kFull, tail);
    if (hole) to[holes + __popc(hs & below)] = j;
    if (tail) from[tails + __popc(ts & below)] = j;
    holes += __popc(hs);
    tails += __popc(ts);
    if (j < x.to) {
      if (!tail) slots[j] = stay ? j : -1;
      if (out && stay && !tail) out[j] = w;
    }
  }
  // as many holes as kept entries behind the new length: the last warp has counted them all
  if (x.rank == x.ranks - 1 && x.warp == kWarps - 1 && x.lane == 0) {
    s.above = tails;
    p.count[b] = tails;
  }
  x.sync();
  const int moves = x.of(x.ranks - 1).above;
  for (int k = x.rank * kThreads + threadIdx.x; k < moves; k += x.ranks * kThreads) {
    const int j = from[k], hole = to[k];
    slots[j] = hole;
    if (out) out[hole] = x.w[j];
  }
  x.sync();
  if (out) {
    for (int j = x.from + x.lane; j < x.to; j += 32)
      if (j >= fresh) out[j] = 0.f;
  }
  if (x.rank == 0 && threadIdx.x == 0) p.lens_out[b] = fresh;
}

struct MoveParams {
  uint8_t* codes[2];
  uint16_t* params[2];
  const int32_t* table;
  int table_stride, pages, page_size, heads, groups;
  const int32_t* count;
  const int32_t* from;
  const int32_t* to;
  int64_t most;
  int splits;
};

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) kv4_evict_move_kernel(const __grid_constant__ MoveParams p) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.splits, part = blockIdx.x - b * p.splits;
  const int count = p.count[b];
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;
  const int stride = p.splits * (kMoveThreads / 32);
  for (int k = part * (kMoveThreads / 32) + (threadIdx.x >> 5); k < count; k += stride) {
    const int j[2] = {p.from[b * p.most + k], p.to[b * p.most + k]};
    int64_t row[2];
    bool there = true;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = j[e] / p.page_size;
      const int page = table[t];
      there &= static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
      row[e] = static_cast<int64_t>(page) * p.heads * p.page_size + (j[e] - t * p.page_size);
    }
    if (!there) continue;
    // a lane's unit: one group of one tensor of one head
    for (int u = lane; u < p.heads * 2 * p.groups; u += 32) {
      const int ht = u / p.groups, group = u - ht * p.groups, tensor = ht & 1;
      const int64_t up = static_cast<int64_t>(ht >> 1) * p.page_size;
      const int64_t src = (row[0] + up) * p.groups + group, dst = (row[1] + up) * p.groups + group;
      uint4* codes = reinterpret_cast<uint4*>(p.codes[tensor]);
      codes[dst] = codes[src];
      p.params[tensor][dst] = p.params[tensor][src];
    }
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
  int ranks = 1;
  while (ranks < kMaxRanks && max_len > ranks * kThreads * 2 &&
         static_cast<int64_t>(B) * ranks * 2 <= 2 * static_cast<int64_t>(sm_count))
    ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_evict_select_kernel, p);
  if (e != cudaSuccess || max_len <= budget) return e;
  MoveParams m{};
  m.codes[0] = cache.k_codes, m.codes[1] = cache.v_codes;
  m.params[0] = cache.k_params, m.params[1] = cache.v_params;
  m.table = cache.page_table;
  m.table_stride = cache.table_stride, m.pages = cache.pages, m.page_size = cache.page_size;
  m.heads = cache.heads;
  m.groups = cache.head_dim / 32;
  m.count = p.count, m.from = p.from, m.to = p.to;
  m.most = p.most;
  const int64_t most = std::min<int64_t>(max_len - budget, budget);
  const int64_t warps = kMoveThreads / 32;
  m.splits = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((most + warps - 1) / warps, (8 * static_cast<int64_t>(sm_count) + B - 1) / B)));
  kv4_evict_move_kernel<<<static_cast<unsigned>(static_cast<int64_t>(B) * m.splits), kMoveThreads, 0, stream>>>(m);
  return cudaGetLastError();
}

}  // namespace dllm

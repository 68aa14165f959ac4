// Attention over the 4-bit cache for many query rows per cache head (blocks, pieces of prompts), on
// the 5th-generation tensor cores.
//
// Entries are taken 64 at a time:
//   S [128 rows x 64] = Q K^T,   O [128 x D] += P V     (tcgen05.mma, fp32 accumulators in TMEM)
// Two groups of four warps each hold 128 rows, one row a thread.  With more than 128 rows in a
// segment (kShare) the groups are the two halves of a 256-row tile and both use every K and V tile;
// otherwise they hold the same rows, take the tiles in turn, and add up at the end.  (1024 tokens of
// 4 heads over 16384 entries: 387 us; with the same rows in both groups 549.)  With 192 or 256
// channels the accumulator of one group fills most of half of the tensor memory, and there is no
// second group.
//
// Warps 0-7: softmax (no shuffles), the rescaling of O when the reference moves (rarely:
// attention.cu's kSlack), and the output.  Warps 18 and 19 look the pages up and have the tiles' codes
// and params copied into a ring (bulk copies, V's and K's); they also fetch the next queries to L2 and
// leave the notes for the join.  Warps 8-15 turn codes to bf16, into rings of K and V tiles in the
// 128-byte swizzled layout, each half of them every second tile; a lane turns 32 channels (one group)
// of an entry, in an order in which no two lanes meet in a bank.  Warps 16 and 17 issue the products
// of a group each: the scores of a step as soon as the softmax warps hold those of the step before
// in registers, so that they are there when the softmax comes back for them.
//
// TMEM, 512 columns: O 2 x 128, S 2 x 64, P 2 x 32 and 64 for the queries (left operands may lie
// there): those of group 0, or of both groups where the rows are the same.  Otherwise group 1's are
// in shared memory.  Per 64 entries, 256 rows and D = 128 shared memory then moves 146 KB (K and V
// written once and read twice, the queries of group 1 read once, the codes in and out), 1150
// cycles, about as many as the products of both groups take (1152).
//
// Measured: a step of 256 rows takes 1750 to 1850 cycles, so 0.62 to 0.66 of the tensor cores' time
// (1.29 PFLOP/s on the piece above, 0.66 of the card's burst rate; 1.07 with 256 channels, 128 segments
// of 65 tiles in 65 us).  What is left is the chain scores -> softmax -> weights -> product, each
// hand-over 120 cycles, with 60 % of the issue slots busy.  One segment by itself costs about 8 us
// (launch, queries, one tile, output).  Measured slower, on the piece: two places for each group's
// scores with all queries in shared memory (444 us: its reads bind), two threads a row (478), other
// orders of the warps (402, 432), a poll with a sleep hint everywhere (418), scores unpacked for
// single multiplications (395).
// The eight channels of a code word come out as pairs (j, j + 4): Q's channels are put in the same
// order (the scores do not depend on it), and the output's are put back.
#include "attention.h"

#include <limits.h>

#include <algorithm>

#include "attention_line.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "mbarrier.cuh"
#include "vec_math.cuh"

namespace dllm {
namespace {

constexpr int kRows = 128;
constexpr int kTile = 64;  // entries of a step
// K tiles and V tiles have a ring each: a K tile is free again as soon as its scores are there, a V
// tile only when its weights have been taken off them and multiplied.
// Sizes of the rings, by what fits beside the rest.  A parity wait tells a phase from the one before
// it only.  The halves of the turning warps (and, with the same rows, the groups) take every second
// tile: with even rings they take every use of their own places and so wait for every phase of those
// barriers.
__host__ __device__ constexpr int k_tiles(int D) { return D > 128 ? 2 : 4; }
__host__ __device__ constexpr int v_tiles(int D, bool share) { return D > 128 ? 2 : share ? 4 : 6; }
constexpr int kRawTiles = 4;
constexpr int kThreads = 640;
// registers a thread: launched with 96, then shared out anew, 128 threads a figure (two groups:
// 2 x 152 + 2 x 64 + 48; one group: 152 + 24 + 2 x 128 + 48; both at most 5 x 96)
constexpr int kSoftmaxRegs = 152, kIssueRegs = 48, kIdleRegs = 24;
__host__ __device__ constexpr int turn_regs(int D) { return D > 128 ? 128 : 64; }
static_assert(2 * kSoftmaxRegs + 2 * turn_regs(128) + kIssueRegs <= 5 * 96, "");
static_assert(kSoftmaxRegs + kIdleRegs + 2 * turn_regs(256) + kIssueRegs <= 5 * 96, "");
constexpr int kTmemCols = 512;
constexpr float kSlack = 8.f;  // as in attention.cu

// ---- tcgen05, one CTA

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The products are issued by whole warps with uniform operands, one elected lane (`lead`) executing:
// in a branch of one lane the compiler has to move every operand to the uniform registers anew, and
// issuing the twelve products of a step took longer than computing them.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}
// A value that all lanes hold, in a uniform register (a reduction's result is): what is computed from
// it stays there.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(kFull, x); }
__device__ __forceinline__ int uniform(int x) {
  return static_cast<int>(uniform(static_cast<uint32_t>(x)));
}
// D [128 x N] (+)= A [128 x 16] B [16 x N], A in TMEM, B in shared memory
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// the same with A in shared memory
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// Arrive on `bar` once every tcgen05.mma issued so far by this thread has completed.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory descriptors, 128-byte swizzle: rows of 128 bytes (64 channels of one entry), the
// 16-byte piece c of row i at i * 128 + ((c ^ (i & 7)) * 16), 8-row groups 1024 bytes apart, 64
// channels further 64 rows on.  K is K-major (the product runs over the channels of a row); V is
// MN-major (it runs over the rows): its leading offset steps to the next 64 channels.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t leading) {
  return ((saddr & 0x3FFFFu) >> 4) | (leading >> 4) << 16;
}
// the descriptor `bytes` further on
__device__ __forceinline__ uint64_t desc_at(uint32_t low, uint32_t bytes) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low + (bytes >> 4)), "r"(kDescHigh));
  return d;
}
// D fp32, A and B bf16, M = 128; b_mn: B is MN-major
__host__ __device__ constexpr uint32_t idesc(int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A whole warp's wait: one vote when the phase is complete already; the same bounded wait otherwise.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int32_t* status) {
  if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  return __all_sync(kFull, wait_bar(bar, parity, abort_flag, status)) != 0;
}

// The same for waits that may end a little late (the copies, and the codes they bring): the warp
// sleeps between its looks and leaves the issue slots to the others (prompt piece 387 us, 391 without;
// 420 if the turning warps' waits for free places sleep too).
template <unsigned NS>
__device__ __forceinline__ bool wait_warp_lazy(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               int32_t* status) {
  for (int i = 0; i < 64; ++i) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    __nanosleep(NS);
  }
  return __all_sync(kFull, wait_bar(bar, parity, abort_flag, status)) != 0;
}

template <int D, bool kShare>
struct Smem {
  static constexpr uint32_t kTensor = kTile * D * 2;  // a K (or V) tile
  static constexpr uint32_t kV = k_tiles(D) * kTensor;
  static constexpr uint32_t kQ = kV + v_tiles(D, kShare) * kTensor;  // group 1's own queries
  static constexpr uint32_t kScratch = kQ + (kShare ? kRows * D * 2 : 0);  // 2 KB a softmax warp
  // codes and params as they come from the cache, kRawTiles tiles: K codes, V codes, K and V params
  static constexpr uint32_t kRaw = kScratch + (D > 128 ? 4 : 8) * 2048;
  static constexpr uint32_t kRawCodes = kTile * D / 2, kRawPar = kTile * D / 16;
  static constexpr uint32_t kRawTile = 2 * (kRawCodes + kRawPar);
  static constexpr size_t kBytes = kRaw + kRawTiles * kRawTile + 1024;  // and room to align
};

// What a CTA does with one segment.
template <int ROWS>
struct Piece {
  int units, j0, end, tiles;
  __device__ __forceinline__ Piece(const Segment<ROWS>& sg, const AttnPlan& f, int left) {
    units = min(sg.units - sg.k0, left);
    j0 = sg.k0 << f.unit_log2;
    end = min(sg.seen, (sg.k0 + units) << f.unit_log2);
    tiles = end > j0 ? (end - j0 + kTile - 1) / kTile : 0;
  }
};

template <int D, bool kShare>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPlan f) {
  using M = Smem<D, kShare>;
  constexpr bool kTwo = D <= 128;            // two groups: O of one is all that fits beyond
  constexpr bool kSame = kTwo && !kShare;    // of the same rows
  constexpr int kKTiles = k_tiles(D), kVTiles = v_tiles(D, kShare);
  static_assert(kKTiles % 2 == 0 && kVTiles % 2 == 0 && kRawTiles % 2 == 0, "");
  constexpr int kVisible = 2 * kKTiles;  // scores kKTiles on are not begun before those here are read
  constexpr int ROWS = kShare ? 2 * kRows : kRows;
  constexpr int STRIDE = kSame ? 2 : 1;  // tiles from one of a group to its next
  constexpr uint32_t SLAB = kTile * 128, QSLAB = kRows * 128;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t bars[2 * kKTiles + 2 * kVTiles + 2 * kRawTiles + 11];
  __shared__ uint32_t visible[kVisible][2];  // of a tile's 64 entries: a bit per entry
  __shared__ uint32_t raw_visible[kRawTiles][2];
  __shared__ float2 ml_s[2][kRows];         // groups with the same rows: reference and sum
  __shared__ int start_s[12];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int nan_met;  // a NaN of V on a diagonal

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t k_full0 = smem_u32(&bars[0]), k_empty0 = k_full0 + 8 * kKTiles;
  const uint32_t v_full0 = k_empty0 + 8 * kKTiles, v_empty0 = v_full0 + 8 * kVTiles;
  const uint32_t gbars = v_empty0 + 8 * kVTiles;  // of group g at + 40 g:
  // the queries are there and O may be overwritten; S is there; S has been read; P is there; the
  // product with V has been added
  constexpr uint32_t kBarQ = 0, kBarS = 8, kBarFree = 16, kBarP = 24, kBarV = 32, kGroupBars = 40;
  const uint32_t done_bar = gbars + 2 * kGroupBars;
  const uint32_t raw_full0 = done_bar + 8, raw_empty0 = raw_full0 + 8 * kRawTiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKTiles; ++s) {
      mbar_init(k_full0 + 8 * s, 4);
      mbar_init(k_empty0 + 8 * s, kShare ? 2 : 1);
    }
    for (int s = 0; s < kVTiles; ++s) {
      mbar_init(v_full0 + 8 * s, 4);
      mbar_init(v_empty0 + 8 * s, kShare ? 2 : 1);
    }
    for (int g = 0; g < 2; ++g) {
      const uint32_t bar = gbars + kGroupBars * g;
      mbar_init(bar + kBarQ, kSame ? 8 : 4);
      mbar_init(bar + kBarS, 2);  // the scores' completion, and the issuer's word that their mask is there
      mbar_init(bar + kBarFree, 4);
      mbar_init(bar + kBarP, 4);
      mbar_init(bar + kBarV, 1);
    }
    mbar_init(done_bar, kTwo ? 2 : 1);
    for (int s = 0; s < kRawTiles; ++s) {
      mbar_init(raw_full0 + 8 * s, 2 * (kTile / f.copy_span));  // the lanes that copy
      mbar_init(raw_empty0 + 8 * s, 4);  // the four warps that turn them
    }
    abort_flag = nan_met = 0;
    fence_mbar_init();
  }
  // nothing else of this CTA, its tensor memory included, is taken before the kernels it depends
  // on are done: one of them may be waiting for tensor memory
  pdl_wait();
  pdl_trigger();
  {
    Line<ROWS> line;
    line.build(p, f);
    const int u0 = line.start(blockIdx.x), u1 = line.start(blockIdx.x + 1);
    if (u0 >= u1) return;
    if (warp == 0) {
      Segment<ROWS> sg;
      sg.find(p, f, line, u0);
      if (lane == 0) {
        const int v[12] = {sg.item,  sg.b,  sg.rt, sg.h, sg.len,    sg.seen,
                           sg.units, sg.k0, u0,    u1,   line.each, line.longer};
#pragma unroll
        for (int i = 0; i < 12; ++i) start_s[i] = v[i];
      }
    }
  }
  if (warp == 16) tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort_v = &abort_flag;
  const int rows = p.n * p.G;
  auto col_o = [](int g) { return 128u * g; };
  auto col_s = [](int g) { return 256u + 64u * g; };
  auto col_p = [](int g) { return kTwo ? 384u + 32u * g : 320u; };
  constexpr uint32_t col_q = kTwo ? 448 : 384;

  // Where the CTA begins.  Each role reads it for itself once it has its own share of the registers:
  // taken across the split it was spilled, and read back in every step (128 segments of 65 tiles and 256
  // channels: 72 us in place of 65).
  Segment<ROWS> sg;
  int u0, u1;
  auto begin = [&]() {
    volatile int* v = start_s;
    sg.item = v[0], sg.b = v[1], sg.rt = v[2], sg.h = v[3], sg.len = v[4], sg.seen = v[5];
    sg.units = v[6], sg.k0 = v[7], u0 = v[8], u1 = v[9];
  };
  int step = 0;  // tiles so far
  int mine = 0;  // tiles of this group so far: the phase of its barriers
  // tile k's place in a ring of `of` places, and the parity of its use of it
  auto place = [](int k, unsigned of) { return static_cast<int>(static_cast<unsigned>(k) % of); };
  auto parity = [](int k, unsigned of) { return static_cast<unsigned>(k) / of & 1u; };

  if (!kTwo && warp >= 4 && warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIdleRegs));
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax, one row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int grp = warp >> 2, row_in = threadIdx.x & (kRows - 1);
    const uint32_t bar = gbars + kGroupBars * grp;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + col_s(grp), t_p = lanes + col_p(grp), t_o = lanes + col_o(grp);
    const uint32_t scratch = sbase + M::kScratch + warp * 2048;
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    begin();
    for (int u = u0; u < u1;) {
      const Piece<ROWS> pc(sg, f, u1 - u);
      const int b = sg.b, h = sg.h;
      const int first = kSame ? (grp ^ step) & 1 : 0;  // this group's first tile of the segment
      const int count = pc.tiles > first ? (pc.tiles - first + STRIDE - 1) / STRIDE : 0;
      const int r = sg.rt * ROWS + (kShare ? grp * kRows : 0) + row_in;
      {
        // a negative scale turns the sign of Q, one of zero makes Q zero: both exact
        const uint32_t q_flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        const uint32_t q_keep = p.scale_log2 == 0.f ? 0u : 0xffffffffu;
        // The warp loads its 32 rows, four lanes 64 bytes (32 channels) of a row, and puts them where
        // they belong: group 1's own at once, the others 32 channels at a time by way of the warp's
        // scratch, from where each thread takes those of its own row to TMEM.  Groups with the same
        // rows share the queries there, and each brings half of the channels.
        const int lr = lane >> 2, lp = lane & 3;
        constexpr int CHUNKS = kSame ? D / 64 : D / 32;
        constexpr int BLOCK = CHUNKS % 4 == 0 ? 4 : CHUNKS % 3 == 0 ? 3 : CHUNKS;
        const bool to_tmem = !kShare || grp == 0;
#pragma unroll 1
        for (int c0 = 0; c0 < CHUNKS; c0 += BLOCK) {
          const int chunk0 = (kSame ? grp * CHUNKS : 0) + c0;
          uint4 v[BLOCK][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = r - lane + e * 8 + lr;
            const int ri = token_of(p, rr);
            const uint16_t* src =
                p.q + b * p.qb + ri * p.qt + (h * p.G + rr - ri * p.G) * p.qh + chunk0 * 32 + lp * 8;
#pragma unroll
            for (int c = 0; c < BLOCK; ++c) {
              v[c][e] = make_uint4(0u, 0u, 0u, 0u);
              if (rr < rows) {
                if (f.q_aligned) {
                  v[c][e] = *reinterpret_cast<const uint4*>(src + c * 32);
                } else {
                  const uint16_t* s8 = src + c * 32;
                  v[c][e].x = s8[0] | static_cast<uint32_t>(s8[1]) << 16;
                  v[c][e].y = s8[2] | static_cast<uint32_t>(s8[3]) << 16;
                  v[c][e].z = s8[4] | static_cast<uint32_t>(s8[5]) << 16;
                  v[c][e].w = s8[6] | static_cast<uint32_t>(s8[7]) << 16;
                }
              }
            }
          }
#pragma unroll
          for (int c = 0; c < BLOCK; ++c) {
            if (to_tmem) __syncwarp();  // what was in the scratch has been taken
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t x[4] = {v[c][e].x, v[c][e].y, v[c][e].z, v[c][e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = (x[k] ^ q_flip) & q_keep;
              const int rw = e * 8 + lr, rg = (warp & 3) * 32 + rw;  // row of the warp, of the group
              const uint32_t dst =
                  to_tmem ? scratch + rw * 64 + ((lp ^ (rw >> 1 & 3)) << 4)
                          : sbase + M::kQ + (c >> 1) * QSLAB + rg * 128 +
                                ((((c & 1) * 4 + lp) ^ (rg & 7)) << 4);
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst),
                           "r"(__byte_perm(x[0], x[2], 0x5410)), "r"(__byte_perm(x[0], x[2], 0x7632)),
                           "r"(__byte_perm(x[1], x[3], 0x5410)), "r"(__byte_perm(x[1], x[3], 0x7632))
                           : "memory");
            }
            if (to_tmem) {
              __syncwarp();
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 y = ld_shared_v4(scratch + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4));
                w[4 * k] = y.x, w[4 * k + 1] = y.y, w[4 * k + 2] = y.z, w[4 * k + 3] = y.w;
              }
              tmem_st16(lanes + col_q + (chunk0 + c) * 16, w);
            }
          }
        }
        if (to_tmem)
          tmem_wait_st();
        else
          fence_async_shared();
        tc_before();
        __syncwarp();
        // only of a group with tiles here: it is held up at the end until its issuer has passed
        if (lane == 0 && count > 0) mbar_arrive(bar + kBarQ);
        // both groups read both accumulators of the segment before, and the queries are shared
        if (kSame && lane == 0 && pc.tiles > 1 - first)
          mbar_arrive(gbars + kGroupBars * (grp ^ 1) + kBarQ);
      }
      const int bound = rows_see(p, sg.len, r);             // entries this row sees
      const int all_see = rows_see(p, sg.len, r - row_in);  // what every row of the group sees
      float m = -INFINITY;
      uint64_t l2 = 0;  // two partial sums
      bool ok = true;
      int vis_at = place(step + first, kVisible);
      for (int n = 0; n < count; ++n) {
        const int t = first + n * STRIDE;
        // the scores and the mask words of their stage
        ok = wait_warp(bar + kBarS, (mine + n) & 1, abort_v, f.status);
        if (!ok) break;
        tc_after();
        float s[kTile];
        tmem_ld32(t_s, s);
        tmem_ld32(t_s + 32, s + 32);
        const uint32_t vis0 = visible[vis_at][0], vis1 = visible[vis_at][1];
        vis_at = place(vis_at + STRIDE, kVisible);
        tmem_wait_ld();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kBarFree);
        const int j = pc.j0 + t * kTile;
        if ((vis0 & vis1) != 0xffffffffu || j + kTile > all_see) {
          // what this row sees of the tile, a bit per entry
          auto below = [](int x) { return x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1u; };
          const uint32_t see[2] = {vis0 & below(bound - j), vis1 & below(bound - j - 32)};
#pragma unroll
          for (int e = 0; e < kTile; ++e) s[e] = see[e >> 5] & (1u << (e & 31)) ? s[e] : -INFINITY;
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e < kTile; e += 8) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            top[x] = e + 4 + x < kTile ? max3(top[x], s[e + x], s[e + 4 + x])
                                       : fmaxf(top[x], s[e + x]);
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
        if (__any_sync(kFull, mx > m + kSlack)) {
          const float mn = fmaxf(m, mx);
          const float keep = mn == -INFINITY ? 1.f : ex2(m - mn);
          m = mn;
          float la, lb;
          unpack2(l2, la, lb);
          l2 = pack2(la * keep, lb * keep);
          if (n > 0) {
            // the products before have been added to O
            ok = wait_warp(bar + kBarV, (mine + n - 1) & 1, abort_v, f.status);
            if (!ok) break;
            tc_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(t_o + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= keep;
              tmem_st32(t_o + c, reinterpret_cast<uint32_t*>(o));
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t scale2 = pack2(scale, scale), mu2 = pack2(-mu, -mu);
        uint32_t* pk = reinterpret_cast<uint32_t*>(s);  // in place
        // P of the step before has been read, as a rule: asked now, needed after the exponentials
        const bool p_free = n == 0 || mbar_try_wait(bar + kBarV, (mine + n - 1) & 1);
        uint64_t l_odd = 0;
#pragma unroll
        for (int e = 0; e < kTile; e += 4) {
          float a0, a1, a2, a3;
          unpack2(fma2(pack2(s[e], s[e + 1]), scale2, mu2), a0, a1);
          unpack2(fma2(pack2(s[e + 2], s[e + 3]), scale2, mu2), a2, a3);
          a0 = ex2(a0), a1 = ex2(a1), a2 = ex2(a2), a3 = ex2(a3);
          l2 = add2(l2, pack2(a0, a1));
          l_odd = add2(l_odd, pack2(a2, a3));
          pk[e / 2] = bf2_pack(a0, a1);
          pk[e / 2 + 1] = bf2_pack(a2, a3);
        }
        l2 = add2(l2, l_odd);
        if (!__all_sync(kFull, p_free)) {
          ok = wait_warp(bar + kBarV, (mine + n - 1) & 1, abort_v, f.status);
          if (!ok) break;
        }
        tc_after();
        tmem_st32(t_p, pk);
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kBarP);
      }
      float l, l_hi;
      unpack2(l2, l, l_hi);
      l += l_hi;
      const bool direct = pc.units == sg.units;
      int64_t out_row[4];  // element of p.out where the lane's piece of row 8 e + lane / 4 starts
#pragma unroll
      for (int e = 0; e < 4 && direct; ++e) {
        const int rr = r - lane + e * 8 + (lane >> 2), ri = token_of(p, rr);
        out_row[e] = rr < rows ? b * p.ob + ri * p.ot + (h * p.G + rr - ri * p.G) * p.oh +
                                     (lane & 3) * 8
                               : INT64_MIN;
      }
      // ---- output.  Groups with the same rows: each takes half of the channels of both.
      if (count > 0 && ok) ok = wait_warp(bar + kBarV, (mine + count - 1) & 1, abort_v, f.status);
      if constexpr (kSame) {
        ml_s[grp][row_in] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");  // both groups' products are complete
      }
      tc_after();
      if (ok) {
        const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (u == u0 ? 0 : 1);
        const int row_tile = r - sg.rt * ROWS;
        float keep0 = 1.f, keep1 = 0.f;  // this group's and the other's
        // An accumulator without a tile holds nothing yet; all others count however small their weight
        // is (0 * NaN is NaN).
        const bool other = kSame && pc.tiles > 1 - first;
        if constexpr (kSame) {
          const float2 ml = ml_s[grp ^ 1][row_in];
          const float mn = fmaxf(m, ml.x);
          keep0 = m == -INFINITY ? 0.f : ex2(m - mn);
          keep1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - mn);
          l = fmaf(l, keep0, ml.y * keep1);
          m = mn;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        constexpr int SPAN = kSame ? D / 2 : D;
        const int c0 = kSame ? grp * SPAN : 0;
        const uint32_t t_other = lanes + col_o(grp ^ 1);
#pragma unroll 1
        for (int c = c0; c < c0 + SPAN; c += 32) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
          if constexpr (!kSame) {
            if (count > 0) {
              tmem_ld32(t_o + c, o);
              tmem_wait_ld();
            }
          } else {
            float x[32] = {};
            if (count > 0) tmem_ld32(t_o + c, o);
            if (other) tmem_ld32(t_other + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(x[e], keep1, o[e] * keep0);
          }
          // channels back in order: the word holds 0, 4, 1, 5, 2, 6, 3, 7
          if (r < rows && !direct) {
            // four channels of a row together, rows side by side: the warp's stores are contiguous
            float4* dst = reinterpret_cast<float4*>(f.part_o) +
                          (part * (D / 4) + c / 4) * ROWS + row_tile;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              dst[(2 * k) * ROWS] = make_float4(o[8 * k], o[8 * k + 2], o[8 * k + 4], o[8 * k + 6]);
              dst[(2 * k + 1) * ROWS] =
                  make_float4(o[8 * k + 1], o[8 * k + 3], o[8 * k + 5], o[8 * k + 7]);
            }
          } else if (direct) {
            // by way of the scratch, so that four lanes store 64 contiguous bytes of a row
#pragma unroll
            for (int k = 0; k < 4; ++k)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                               scratch + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)),
                           "r"(bf2_pack(o[8 * k] * inv, o[8 * k + 2] * inv)),
                           "r"(bf2_pack(o[8 * k + 4] * inv, o[8 * k + 6] * inv)),
                           "r"(bf2_pack(o[8 * k + 1] * inv, o[8 * k + 3] * inv)),
                           "r"(bf2_pack(o[8 * k + 5] * inv, o[8 * k + 7] * inv))
                           : "memory");
            __syncwarp();
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int lr = e * 8 + (lane >> 2);
              v[e] = ld_shared_v4(scratch + lr * 64 + (((lane & 3) ^ (lr >> 1 & 3)) << 4));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (out_row[e] == INT64_MIN) continue;
              uint16_t* dst = p.out + out_row[e] + c;
              if (f.out_aligned) {
                *reinterpret_cast<uint4*>(dst) = v[e];
              } else {
                const uint32_t y[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
                for (int x = 0; x < 8; ++x) dst[x] = static_cast<uint16_t>(y[x >> 1] >> (16 * (x & 1)));
              }
            }
          }
          __syncwarp();
        }
        if (r < rows && (!kSame || grp == 0)) {
          if (!direct)
            f.part_ml[part * ROWS + row_tile] = make_float2(m, l);
          else
            store_lse(p, b, h, r, m, l);
        }
      }
      if constexpr (kSame) asm volatile("bar.sync 1, 256;" ::: "memory");  // ml_s is read
      tc_before();  // O and Q are read before the next segment's arrival on kBarQ
      mine += count;
      step += pc.tiles;
      u += pc.units;
      if (u < u1) sg.next(p, f);
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------------ codes to bf16
    // this half of the warps every second tile
    if constexpr (turn_regs(D) < 96)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(turn_regs(D)));
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(turn_regs(D)));
    constexpr int GROUPS = D / 32;  // per entry
    constexpr int PER = GROUPS / 2;  // pieces of K (and of V) a thread turns per tile
    // Piece e of the thread: entry entry0 + APART * e, group g; with 192 channels, whose six groups do
    // not divide the threads, entry entry0 and group g + 2 e.
    constexpr bool kByEntry = D == 192;
    constexpr int APART = kByEntry ? 0 : 128 / GROUPS;
    constexpr uint32_t RAW_STEP = kByEntry ? 32 : 2048, PAR_STEP = kByEntry ? 4 : 256;
    constexpr uint32_t DST_STEP = kByEntry ? SLAB : APART * 128;
    const int half = (warp >> 2) & 1, w = warp & 3;
    const int entry0 = kByEntry ? w * 16 + (lane & 15) : (w * 32 + lane) / GROUPS;
    const int g = kByEntry ? lane >> 4 : lane % GROUPS;
    const uint32_t raw0 = sbase + M::kRaw + entry0 * (D / 2) + g * 16;
    const uint32_t par0 = sbase + M::kRaw + 2 * M::kRawCodes + entry0 * (D / 16) + g * 2;
    // Word x goes to 16-byte piece (4 (g % 2) + x) ^ (entry % 8) of the entry's row in slab g / 2.
    // Lanes of slab 1 store words in the order 2, 3, 0, 1 (D = 128), those of slab s word x ^ s in
    // place of word x (D = 256): with eight lanes at a time (two entries of four groups, or one of
    // eight), all eight pieces of a 128-byte row are then hit once; eight entries of one group (D = 192)
    // do that by themselves.
    const int turn_x = D > 128 ? g >> 1 : D > 64 && g >= 2 ? 2 : 0;
    uint32_t piece_at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      piece_at[x] = sbase + (g >> 1) * SLAB + entry0 * 128 +
                    ((((g & 1) * 4 + (x ^ turn_x)) ^ (entry0 & 7)) << 4);
    auto turn = [&](const uint4& codes, uint32_t param, uint32_t dst) {
      const Kv4Scale sc = kv4_scale(__byte_perm(param, param, 0x1010));
      uint32_t wd[4] = {codes.x, codes.y, codes.z, codes.w};
      if (turn_x & 2) {
        wd[0] = codes.z, wd[1] = codes.w, wd[2] = codes.x, wd[3] = codes.y;
      }
      if (D > 128 && (turn_x & 1)) {
        const uint32_t w0 = wd[0], w2 = wd[2];
        wd[0] = wd[1], wd[1] = w0, wd[2] = wd[3], wd[3] = w2;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t a = kv4_pair<0>(wd[x], sc), c = kv4_pair<1>(wd[x], sc),
                       d = kv4_pair<2>(wd[x], sc), z = kv4_pair<3>(wd[x], sc);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + piece_at[x]), "r"(a),
                     "r"(c), "r"(d), "r"(z)
                     : "memory");
      }
    };
    begin();
    for (int u = u0; u < u1;) {
      const Piece<ROWS> pc(sg, f, u1 - u);
      // first tile that not every row sees whole
      const int t_diagonal = p.causal ? (rows_see(p, sg.len, sg.rt * ROWS) - pc.j0) >> 6 : INT_MAX;
      for (int t = (half ^ step) & 1; t < pc.tiles; t += 2) {
        const int k = step + t, rs = place(k, kRawTiles);
        if (!wait_warp_lazy<50>(raw_full0 + 8 * rs, parity(k, kRawTiles), abort_v, f.status)) break;
        const uint32_t at = raw0 + rs * M::kRawTile, par = par0 + rs * M::kRawTile;
        uint4 kc[PER], vc[PER];
        uint32_t kp[PER], vp[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          kc[e] = ld_shared_v4(at + e * RAW_STEP);
          vc[e] = ld_shared_v4(at + M::kRawCodes + e * RAW_STEP);
          kp[e] = ld_shared_u16(par + e * PAR_STEP);
          vp[e] = ld_shared_u16(par + M::kRawPar + e * PAR_STEP);
        }
        const uint32_t vis[2] = {raw_visible[rs][0], raw_visible[rs][1]};
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          // values of hidden entries are 0, whatever they hold: their weight of 0 must not meet a NaN
          const int entry = entry0 + APART * e;
          const uint32_t word = entry < 32 ? vis[0] : vis[1];
          if (!(word >> (entry & 31) & 1u)) vp[e] = 0u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(raw_empty0 + 8 * rs);
        const int ks = place(k, kKTiles), vs = place(k, kVTiles);
        if (!wait_warp(k_empty0 + 8 * ks, parity(k, kKTiles) ^ 1, abort_v, f.status)) break;
        if (w == 0 && lane < 2) visible[place(k, kVisible)][lane] = lane ? vis[1] : vis[0];
#pragma unroll
        for (int e = 0; e < PER; ++e) turn(kc[e], kp[e], ks * M::kTensor + e * DST_STEP);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full0 + 8 * ks);
        if (t >= t_diagonal) {  // (attention_line.cuh: put_nans; K's values come first, its scores wait)
          bool nan = false;
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            nan |= kv4_nan(vp[e]);
            vp[e] = kv4_nan(vp[e]) ? 0u : vp[e];
          }
          if (nan) nan_met = 1;
        }
        if (!wait_warp(v_empty0 + 8 * vs, parity(k, kVTiles) ^ 1, abort_v, f.status)) break;
#pragma unroll
        for (int e = 0; e < PER; ++e) turn(vc[e], vp[e], M::kV + vs * M::kTensor + e * DST_STEP);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full0 + 8 * vs);
      }
      step += pc.tiles;
      u += pc.units;
      if (u < u1) sg.next(p, f);
    }
  } else {
    // ------------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    const int grp = uniform(warp) - 16;
    if (!kTwo && grp == 1) {
      // no second group
    } else if (grp < 2) {
      const uint32_t lead = elect_lane();
      const uint32_t bar = gbars + kGroupBars * grp;
      const uint32_t base = uniform(tmem);
      const uint32_t t_s = base + col_s(grp), t_p = base + col_p(grp), t_o = base + col_o(grp);
      const uint32_t smem0 = uniform(sbase), q_low = desc_low(smem0 + M::kQ, 16);
      bool ok = true;
      int piece_no = 0;  // segments with tiles of this group
      begin();
      for (int u = u0; u < u1;) {
        const Piece<ROWS> pc(sg, f, u1 - u);
        const int tiles = uniform(pc.tiles);
        const int first = kSame ? (grp ^ step) & 1 : 0;
        const int count = tiles > first ? (tiles - first + STRIDE - 1) / STRIDE : 0;
        auto wait = [&](uint32_t at, uint32_t phase) {
          return wait_warp(at, phase, abort_v, f.status);
        };
        if (count > 0) ok = ok && wait(bar + kBarQ, piece_no++ & 1);
        auto scores = [&](int k) {
          const int ks = place(k, kKTiles);
          if (!wait(k_full0 + 8 * ks, parity(k, kKTiles))) return false;
          tc_after();
          const uint32_t low = desc_low(smem0 + ks * M::kTensor, 16);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint64_t kd = desc_at(low, (x >> 2) * SLAB + (x & 3) * 32);
            if (!kShare || grp == 0)
              mma_ts(lead, t_s, base + col_q + x * 8, kd, idesc(kTile, false), x > 0);
            else
              mma_ss(lead, t_s, desc_at(q_low, (x >> 2) * QSLAB + (x & 3) * 32), kd,
                     idesc(kTile, false), x > 0);
          }
          mma_commit(lead, bar + kBarS);
          mma_commit(lead, k_empty0 + 8 * ks);
          if (lead) mbar_arrive(bar + kBarS);
          return true;
        };
        if (count > 0) ok = ok && scores(step + first);
        for (int n = 0; n < count && ok; ++n) {
          const int k = step + first + n * STRIDE;
          if (n + 1 < count) {
            ok = wait(bar + kBarFree, (mine + n) & 1) && scores(k + STRIDE);
            if (!ok) break;
          }
          ok = wait(bar + kBarP, (mine + n) & 1);
          if (!ok) break;
          const int vs = place(k, kVTiles);
          ok = wait(v_full0 + 8 * vs, parity(k, kVTiles));
          if (!ok) break;
          tc_after();
          const uint32_t low = desc_low(smem0 + M::kV + vs * M::kTensor, D > 64 ? SLAB : 16);
#pragma unroll
          for (int x = 0; x < kTile / 16; ++x)
            mma_ts(lead, t_o, t_p + x * 8, desc_at(low, x * 2048), idesc(D, true), n > 0 || x > 0);
          mma_commit(lead, bar + kBarV);
          mma_commit(lead, v_empty0 + 8 * vs);
        }
        // the last scores' phase of kBarFree is passed over: it is waited for here
        if (count > 0) ok = ok && wait(bar + kBarFree, (mine + count - 1) & 1);
        mine += count;
        step += tiles;
        u += uniform(pc.units);
        if (u < u1) sg.next(p, f);
      }
      mma_commit(lead, done_bar);
    } else {
      // Copies, in as few pieces as the pages allow (each costs the issuing lane about a hundred
      // cycles): a tile lies in one page when 64 divides the page size, in two or four otherwise.
      // Lane l takes entries span * l .. of the tile; one warp K, the other V.
      const bool is_k = grp == 3;
      const uint8_t* codes = is_k ? p.k_codes : p.v_codes;
      const uint16_t* params = is_k ? p.k_params : p.v_params;
      const int span = f.copy_span, mine_from = span * lane;
      const bool copier = mine_from < kTile;
      const int step_pages = kTile / p.page_size, step_slots = kTile % p.page_size;
      const uint32_t codes_bytes = span * D / 2, par_bytes = span * D / 16;
      const uint32_t to_c = sbase + M::kRaw + (is_k ? 0 : M::kRawCodes) + lane * codes_bytes;
      const uint32_t to_p =
          sbase + M::kRaw + 2 * M::kRawCodes + (is_k ? 0 : M::kRawPar) + lane * par_bytes;
      int sent = 0;
      begin();
      for (int u = u0; u < u1;) {
        const Piece<ROWS> pc(sg, f, u1 - u);
        const int32_t* table = p.table + static_cast<int64_t>(sg.b) * p.table_stride;
        const uint8_t* mask = p.key_mask ? p.key_mask + sg.b * p.mask_stride : nullptr;
        int j = pc.j0, word = (j + mine_from) / p.page_size;
        int slot = j + mine_from - word * p.page_size;
        // page word and mask bytes of the next tile (looked at one round after they are asked for)
        int page = -1;
        uint32_t m0 = 1u, m1 = 1u;
        auto ask = [&]() {
          page = copier && j + mine_from < pc.end && word < p.table_stride ? __ldg(table + word) : -1;
          if (mask) {
            m0 = j + lane < pc.end ? __ldg(mask + j + lane) : 0u;
            m1 = j + 32 + lane < pc.end ? __ldg(mask + j + 32 + lane) : 0u;
          }
        };
        ask();
        for (int t = 0; t < pc.tiles; ++t) {
          const int k = step + t, rs = place(k, kRawTiles);
          const bool here = static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
          const unsigned there = __ballot_sync(kFull, here);  // by piece of `span` entries
          const int64_t row = (static_cast<int64_t>(page) * p.heads + sg.h) * p.page_size + slot;
          const uint32_t v0 = __ballot_sync(kFull, (there >> (lane / span) & 1u) && m0 != 0u &&
                                                       j + lane < pc.end);
          const uint32_t v1 = __ballot_sync(kFull, (there >> ((lane + 32) / span) & 1u) && m1 != 0u &&
                                                       j + 32 + lane < pc.end);
          j += kTile;
          word += step_pages;
          slot += step_slots;
          if (slot >= p.page_size) {
            slot -= p.page_size;
            ++word;
          }
          ask();
          if (!wait_warp_lazy<200>(raw_empty0 + 8 * rs, parity(k, kRawTiles) ^ 1, abort_v, f.status)) break;
          sent = k + 1;
          if (copier) {
            const uint32_t bar = raw_full0 + 8 * rs;
            if (is_k && lane == 0) {
              raw_visible[rs][0] = v0;
              raw_visible[rs][1] = v1;
            }
            if (!here) {
              mbar_arrive(bar);
            } else {
              const uint32_t at = rs * M::kRawTile;
              mbar_expect_tx(bar, codes_bytes + par_bytes);
              bulk_g2s(to_c + at, codes + row * (D / 2), codes_bytes, bar);
              bulk_g2s(to_p + at, params + row * (D / 32), par_bytes, bar);
            }
          }
          __syncwarp();
        }
        step += pc.tiles;
        if (is_k && lane == 0) {
          Line<ROWS> line;
          line.each = start_s[10], line.longer = start_s[11];
          note_segment(f, p, line, sg, u, u0, pc.units == sg.units);
        }
        u += pc.units;
        if (u >= u1) break;
        sg.next(p, f);
        if (is_k) continue;
        // the next segment's queries on their way to L2
        const int r1 = min((sg.rt + 1) * ROWS, rows);
        for (int r = sg.rt * ROWS + lane; r < r1; r += 32) {
          const int i = token_of(p, r);
          const uint16_t* src = p.q + sg.b * p.qb + i * p.qt + (sg.h * p.G + r - i * p.G) * p.qh;
#pragma unroll
          for (int c = 0; c < D; c += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src + c));
        }
      }
      // after a wait that ran out, the last copies into each place may still be under way
      if (*abort_v && lane < kRawTiles && sent > lane) {
        const int last = (sent - 1 - lane) / kRawTiles;  // rounds of this place before its last
        drain_bar(raw_full0 + 8 * lane, last & 1);
      }
    }
  }

  tc_before();
  __syncthreads();
  if (warp == 16) {
    // every product has completed before the tensor memory goes away (bounded: after a wait that
    // ran out too)
    if (lane == 0) drain_bar(done_bar, 0);
    __syncwarp();
    tc_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (nan_met) {
    begin();
    put_nans<D, ROWS, kTile, true>(p, f, sg, u0, u1);
  }
}

// Join the parts of the segments that several CTAs share, in order of their entries (the sums of
// attention_line.cuh's join; the parts lie with four channels of a row together and rows side by
// side).  A CTA takes 32 rows and 64 channels of a segment, a lane one row and 16 channels.
template <int D, int ROWS>
__global__ void __launch_bounds__(128)
    attention_tc_join_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPlan f) {
  constexpr int GROUPS = ROWS / 32, SPANS = D / 64;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int64_t seg = blockIdx.x / (GROUPS * SPANS);
  const int in = blockIdx.x % (GROUPS * SPANS);
  const int2 info = f.parts[seg];
  if (info.x < 0) return;
  const int h = static_cast<int>(seg % p.heads), item = static_cast<int>(seg / p.heads);
  const int b = item / f.row_tiles, rt = item - b * f.row_tiles;
  const int c0 = info.x >> 1, count = info.y - c0 + 1;
  const int row = in % GROUPS * 32 + lane, r = rt * ROWS + row;
  const int ch = in / GROUPS * 64 + warp * 16;
  if (r >= p.n * p.G) return;
  auto part_of = [&](int k) { return static_cast<int64_t>(k == 0 ? info.x : 2 * (c0 + k)); };
  float mx = -INFINITY;
#pragma unroll 4
  for (int k = 0; k < count; ++k) mx = fmaxf(mx, f.part_ml[part_of(k) * ROWS + row].x);
  float4 acc[4] = {};
  float sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < count; ++k) {
    const float2 v = f.part_ml[part_of(k) * ROWS + row];
    const float keep = v.x == -INFINITY ? 0.f : ex2(v.x - mx);
    sum = fmaf(v.y, keep, sum);
    const float4* src = reinterpret_cast<const float4*>(f.part_o) +
                        (part_of(k) * (D / 4) + ch / 4) * ROWS + row;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float4 o = src[x * ROWS];
      acc[x].x = fmaf(o.x, keep, acc[x].x);
      acc[x].y = fmaf(o.y, keep, acc[x].y);
      acc[x].z = fmaf(o.z, keep, acc[x].z);
      acc[x].w = fmaf(o.w, keep, acc[x].w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int i = token_of(p, r), hq = h * p.G + r - i * p.G;
  uint16_t* dst = p.out + b * p.ob + i * p.ot + hq * p.oh + ch;
#pragma unroll
  for (int x = 0; x < 4; x += 2) {
    const uint4 v = make_uint4(bf2_pack(acc[x].x * inv, acc[x].y * inv),
                               bf2_pack(acc[x].z * inv, acc[x].w * inv),
                               bf2_pack(acc[x + 1].x * inv, acc[x + 1].y * inv),
                               bf2_pack(acc[x + 1].z * inv, acc[x + 1].w * inv));
    if (f.out_aligned) {
      *reinterpret_cast<uint4*>(dst + 4 * x) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) dst[4 * x + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
  }
  if (ch == 0) store_lse(p, b, h, r, mx, sum);
}

}  // namespace

bool attention_tc_can(int n, int G, int D) {
  const int64_t least = D == 64 ? 32 : D == 128 ? 16 : 8;
  return static_cast<int64_t>(n) * G > least;
}

// Up to 32 rows only with enough to do: 24 rows of 128 channels take 50 us here and 62 in the other
// kernel (128 heads of 4000 entries), 10.8 and 14.6 (128 of 300), but 22.6 and 17.7 (8 of 8000) and
// 9.8 and 8.8 (8 of 300); 16 rows of 256 channels 69 and 78, 14.0 and 14.9, 26.6 and 23.5, 12.6 and 11.2;
// 16 rows of 192 channels 61 and 70, 12.0 and 11.7.
// 48 rows of 64 channels 46 and 61, 9.5 and 12.6, 21.3 and 16.8, 8.7 and 7.3.
bool attention_tc_takes(const AttnParams& p, int D, int sm_count) {
  if (!attention_tc_can(p.n, p.G, D)) return false;
  const int64_t segments = static_cast<int64_t>(p.B) * p.heads;
  return static_cast<int64_t>(p.n) * p.G > 32 || segments >= 64 ||
         segments * p.max_len >= int64_t{16} * kTile * sm_count;
}

namespace {
int tile_rows(int n, int G, int D) {
  return D <= 128 && static_cast<int64_t>(n) * G > kRows ? 2 * kRows : kRows;
}
}  // namespace

size_t attention_tc_ws_bytes(int B, int n, int G, int heads, int D, int sm_count) {
  const int R = tile_rows(n, G, D);
  const size_t parts = static_cast<size_t>(2) * sm_count * R;
  const size_t tiles = (static_cast<size_t>(n) * G + R - 1) / R;
  return kWsHeader + parts * D * 4 + parts * 8 + B * tiles * heads * 8;
}

// How the line of units is cut, by the tiles that the busiest CTA has to do and what it costs besides,
// as tiles (times: 128 rows a segment and 128 channels unless said otherwise).
//  - Whole segments, nothing to join.
//  - Parts, a CTA each: at least as many CTAs as there are parts.  A part more costs the join half a
//    tile.  8 segments of 65 tiles: 17.7 us in parts of 8 tiles, 18.0 of 4, 21.6 of 16; whole 49.7; in
//    equal stretches 22.4.
//  - Equal stretches: every CTA busy, but most start and end two segments, and the parts are many:
//    taken for 26 tiles.  64 segments of 256 rows and 65 tiles: 48 us, whole 68.8; 128 segments of 47
//    tiles: 46.8 us, whole 39.8; 128 of 65 tiles and 256 channels: 83 us, whole 72.
// Where the lengths may differ the mean is taken for three quarters of the longest.  Against the longest
// itself (both splits of the same call, us): 96 segments of up to 65 tiles, lengths over the last
// 0, 0.3, 0.6 and 0.9 of that: 46.8, 43.4, 39.7, 41.7; whole 50.3, 49.7, 49.3, 49.1.  256 of 44: 74.7, 67.7, 62.2,
// 63.0; whole 70.0, 69.8, 68.3, 67.5.  16 of 512: 59.9, 54.7, 50.4, 47.8; in parts 57.9, 57.5, 56.5, 56.4.  Causal:
// 256 of 44 87.4, whole 93.9.  So it costs up to 7 % where all lengths are the longest and gains up
// to 25 % where they are not.
template <int D>
static void plan_line(const AttnParams& p, int sm_count, AttnPlan* f) {
  constexpr int kLeast = 4;  // tiles of a stretch
  constexpr int kSplit = 26;
  const int64_t segments = static_cast<int64_t>(p.B) * f->row_tiles * p.heads;
  const int64_t tiles = (static_cast<int64_t>(p.max_len) + kTile - 1) / kTile;
  const int64_t whole = (segments + sm_count - 1) / sm_count * tiles;
  const int64_t mean = segments * tiles / sm_count * (p.lens || p.causal ? 3 : 4) / 4;
  const int64_t split = std::max<int64_t>(mean, kLeast) + kSplit;
  int parts_log2 = 0;
  int64_t parts = INT64_MAX;  // twice their cost
  for (int lg = 6; segments <= sm_count; ++lg) {
    const int64_t per = int64_t{1} << (lg - 6), count = (tiles + per - 1) / per;
    if (segments * count <= sm_count && (parts == INT64_MAX || 2 * per + count <= parts + 1)) {
      parts = 2 * per + count;
      parts_log2 = lg;
    }
    if (count <= 1) break;
  }
  if (whole <= split && whole <= parts / 2 + 3) {
    f->unit_log2 = 6;
    while (p.max_len > 1 << f->unit_log2) ++f->unit_log2;
    f->ctas = static_cast<int>(std::min<int64_t>(sm_count, segments));
  } else if (parts / 2 + 1 <= split) {
    f->unit_log2 = parts_log2;
    f->ctas = static_cast<int>(segments * ((p.max_len + (int64_t{1} << parts_log2) - 1) >> parts_log2));
  } else {
    f->unit_log2 = unit_log2_of(segments, p.max_len, 6);
    const int64_t units = segments * ((static_cast<int64_t>(p.max_len) >> f->unit_log2) + 1);
    f->ctas = static_cast<int>(std::min<int64_t>(sm_count, (units + kLeast - 1) / kLeast));
  }
}

template <int D, bool kShare>
static cudaError_t launch_tc(const AttnParams& p, void* ws, int sm_count, cudaStream_t stream) {
  constexpr int R = kShare ? 2 * kRows : kRows;
  AttnPlan f{};
  static_assert(1 << 6 == kTile, "");
  f.row_tiles = (p.n * p.G + R - 1) / R;
  f.copy_span = p.page_size % 64 == 0 ? 64 : p.page_size % 32 == 0 ? 32 : 16;
  plan_line<D>(p, sm_count, &f);
  f.whole = p.max_len <= 1 << f.unit_log2;
  f.q_aligned = attention_rows_aligned(p.q, p.qb, p.qt, p.qh);
  f.out_aligned = attention_rows_aligned(p.out, p.ob, p.ot, p.oh);
  f.status = static_cast<int32_t*>(ws);
  const size_t parts = static_cast<size_t>(2) * sm_count * R;
  char* at = static_cast<char*>(ws) + kWsHeader;
  f.part_o = reinterpret_cast<float*>(at);
  f.part_ml = reinterpret_cast<float2*>(at + parts * D * 4);
  f.parts = reinterpret_cast<int2*>(at + parts * D * 4 + parts * 8);
  cudaError_t e = allow_smem<attention_tc_kernel<D, kShare>>(Smem<D, kShare>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attention_tc_kernel<D, kShare>, dim3(f.ctas), dim3(kThreads),
                       Smem<D, kShare>::kBytes, stream, p, f);
  if (e != cudaSuccess || f.whole) return e;
  // (below 2^31: more than 8 rows to each of 2^30 / rows segments, 16 CTAs a segment at most)
  const int64_t joins = static_cast<int64_t>(p.B) * f.row_tiles * p.heads * (R / 32) * (D / 64);
  return launch_dependent(attention_tc_join_kernel<D, R>, dim3(static_cast<unsigned>(joins)),
                          dim3(128), 0, stream, p, f);
}

cudaError_t launch_attention_tc(const AttnParams& p, int D, void* ws, int sm_count,
                                cudaStream_t stream) {
  if (D == 256) return launch_tc<256, false>(p, ws, sm_count, stream);
  if (D == 192) return launch_tc<192, false>(p, ws, sm_count, stream);
  if (tile_rows(p.n, p.G, D) == kRows)
    return D == 64 ? launch_tc<64, false>(p, ws, sm_count, stream)
                   : launch_tc<128, false>(p, ws, sm_count, stream);
  return D == 64 ? launch_tc<64, true>(p, ws, sm_count, stream)
                 : launch_tc<128, true>(p, ws, sm_count, stream);
}

}  // namespace dllm

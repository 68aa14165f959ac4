// Attention over the 4-bit cache, one warp per query row: scores with one entry per lane, then the
// weighted sum of values with the channels spread over the lanes.
#include "attention.h"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) attention_rows_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float qs[kThreads / 32][D];
  const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
  const int64_t row = blockIdx.x * static_cast<int64_t>(kThreads / 32) + wi;
  pdl_wait();
  pdl_trigger();
  const int heads = p.heads * p.G;
  if (row >= static_cast<int64_t>(p.B) * p.n * heads) return;
  const int h = static_cast<int>(row % heads);
  const int i = static_cast<int>(row / heads % p.n), b = static_cast<int>(row / heads / p.n);
  const uint16_t* q = p.q + b * p.qb + i * p.qt + h * p.qh;
  for (int c = lane; c < D; c += 32) qs[wi][c] = __uint_as_float(static_cast<uint32_t>(q[c]) << 16);
  __syncwarp();
  const int len = p.lens ? max(0, min(__ldg(p.lens + b), p.max_len)) : p.max_len;
  const int last = p.causal ? min(len, len - p.n + i + 1) : len;  // entries below are seen
  const int kvh = h / p.G;
  float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
  for (int j0 = 0; j0 < last; j0 += 32) {
    const int j = j0 + lane;
    int page = -1;
    if (j < last && (!p.key_mask || p.key_mask[b * p.mask_stride + j]))
      page = kv4_page(p.table + static_cast<int64_t>(b) * p.table_stride, p.table_stride, p.pages,
                      p.page_size, j);
    const int64_t at = page < 0 ? 0 : (static_cast<int64_t>(page) * p.heads + kvh) * p.page_size + j % p.page_size;
    float s = -INFINITY;
    if (page >= 0) {
      s = 0.f;
      const uint32_t* kc = reinterpret_cast<const uint32_t*>(p.k_codes + at * (D / 2));
      for (int w = 0; w < D / 8; ++w) {
        const uint32_t pp = p.k_params[at * (D / 32) + w / 4];
        const Kv4Scale sc = kv4_scale(pp | pp << 16);
        const uint32_t word = kc[w];
        const uint32_t v[4] = {kv4_pair<0>(word, sc), kv4_pair<1>(word, sc), kv4_pair<2>(word, sc),
                               kv4_pair<3>(word, sc)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(qs[wi][w * 8 + e], bf16lo(v[e]), s);
          s = fmaf(qs[wi][w * 8 + e + 4], bf16hi(v[e]), s);
        }
      }
      s *= p.scale_log2;
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float keep = ex2(m - mn), e = ex2(s - mn);
    m = mn;
    l = l * keep + e;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] *= keep;
    for (int t = 0; t < 32; ++t) {
      const float pt = __shfl_sync(kFull, e, t);
      const int64_t a = __shfl_sync(kFull, at, t);
      if (!(__shfl_sync(kFull, page, t) >= 0)) continue;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t pp = p.v_params[a * (D / 32) + c];
        const float st = __uint_as_float((pp & 0xFFE0u) << 16);
        const int n = p.v_codes[a * (D / 2) + (c * 32 + lane) / 2] >> (4 * (lane & 1)) & 15;
        acc[c] = fmaf(pt, st * static_cast<float>(n - static_cast<int>(pp & 15u)), acc[c]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
  uint16_t* out = p.out + b * p.ob + i * p.ot + h * p.oh;
  for (int c = 0; c < D / 32; ++c)
    out[c * 32 + lane] = static_cast<uint16_t>(bf2_pack(l > 0.f ? acc[c] / l : 0.f, 0.f));
  if (p.lse && lane == 0)
    p.lse[(static_cast<int64_t>(b) * heads + h) * p.n + i] =
        l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t attention_ws_bytes(int B, int n, int q_heads, int heads, int D, int max_len, int sm_count) {
  (void)B, (void)n, (void)q_heads, (void)heads, (void)D, (void)max_len, (void)sm_count;
  return kWsHeader;
}

cudaError_t launch_attention(AttnParams p, int D, void* ws, int sm_count, cudaStream_t stream) {
  (void)ws, (void)sm_count;
  const int64_t rows = static_cast<int64_t>(p.B) * p.n * p.heads * p.G;
  const dim3 grid(static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32)));
  switch (D) {
    case 64: return launch_dependent(attention_rows_kernel<64>, grid, dim3(kThreads), 0, stream, p);
    case 128: return launch_dependent(attention_rows_kernel<128>, grid, dim3(kThreads), 0, stream, p);
    case 192: return launch_dependent(attention_rows_kernel<192>, grid, dim3(kThreads), 0, stream, p);
    default: return launch_dependent(attention_rows_kernel<256>, grid, dim3(kThreads), 0, stream, p);
  }
}

}  // namespace dllm

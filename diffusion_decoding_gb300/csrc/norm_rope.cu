// Norm of each query and key head and rotation to its position, in one pass (dInfer explainer,
// KV-cache manager: the keys of refreshed entries are recomputed at their positions):
//   y = x * (mean(x^2) + eps)^(-1/2) * w;  pairs (a, c) -> m * (a cos t - c sin t, c cos t + a sin t).
//
// The phase of pair i at position p is p * u_i modulo 2^64 in units of 2^-64 turns (u_i holds the
// frequency): the upper 32 bits of that product, as a signed number, are the phase within half a
// turn, at any position.  Products in fp32 would lose 2^-24 of the whole angle instead, 8e-3
// radians at position 131072.  The hardware sine and cosine then see |angle| <= pi, where their
// error is at most 2^-21.
//
// HBM-bound: 2 * heads * head_dim values move per token.  A group of head_dim / 16 lanes (padded to a
// power of two) owns a head, each lane 16 channels as two 16-byte pieces that hold whole pairs, so
// the mean is a shuffle sum over the group and the rotation stays in the lane.  A warp takes up to
// kUnits such sets of heads of one token, queries or keys, and has all their loads on the way
// before it uses the first; a lane keeps the same channels for all of them, so that sines,
// cosines and weights become 32 factors once:
//   out_a = r (a * w_a cos - c * w_c sin),  out_c = r (c * w_c cos + a * w_a sin),
// two packed fp32 operations for two channels.
//
// Measured: 16384 tokens of 32 + 8 heads of 128 channels, bf16 (336 MB): 56.5 us, 5.9 TB/s, 0.88 of the
// card's copy rate, with 64 % of the issue slots and 48 % of the integer pipe busy; with one set of
// heads a warp in place of four 84 us, with two 61.  Small calls take a launch and the chain position ->
// factors -> store: 2.2 us for one token.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "vec_math.cuh"

namespace dllm {
namespace {

constexpr int kThreads = 128;
constexpr int kUnits = 4;

struct Side {  // one tensor pair; strides in bytes
  const char* x;
  char* y;
  const char* w;
  int heads;
  int64_t xb, xt, xh, yb, yt, yh;
};

struct NormRopeParams {
  Side s[2];
  const int32_t* pos;
  int64_t pos_stride;
  const int64_t* phases;
  int n;
  int64_t tokens;  // B * n
  int D, R, interleaved, norm;
  float magnitude, eps;
  int units;       // sets of heads a warp takes, <= kUnits
  int pack_log2;   // tokens that share a warp (few heads)
  int chunks[2];   // warps per token (or tokens that share one) for the queries and for the keys
};

// cos and sin of p * u turns-in-2^-64, times m
__device__ __forceinline__ void phase_sincos(int p, int64_t u, float m, float& c, float& s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(p)) * static_cast<uint64_t>(u);
  const float a = static_cast<float>(static_cast<int32_t>(t >> 32)) * (6.283185307179586f / 4294967296.f);
  c = __cosf(a) * m;
  s = __sinf(a) * m;
}

template <int DT>
struct Piece {  // eight channels
  uint4 r[DT == DLLM_BF16 ? 1 : 2];
};

template <int DT>
__device__ __forceinline__ Piece<DT> load_piece(const char* p) {
  Piece<DT> v;
  v.r[0] = *reinterpret_cast<const uint4*>(p);
  if constexpr (DT == DLLM_F32) v.r[1] = *reinterpret_cast<const uint4*>(p + 16);
  return v;
}

template <int DT>
__device__ __forceinline__ void unpack(const Piece<DT>& v, float (&x)[8]) {
  if constexpr (DT == DLLM_BF16) {
    const uint32_t w[4] = {v.r[0].x, v.r[0].y, v.r[0].z, v.r[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  } else {
    const uint32_t w[8] = {v.r[0].x, v.r[0].y, v.r[0].z, v.r[0].w,
                           v.r[1].x, v.r[1].y, v.r[1].z, v.r[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
}

template <int DT>
__device__ __forceinline__ void store_piece(char* p, const float (&x)[8]) {
  if constexpr (DT == DLLM_BF16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf2_pack(x[0], x[1]), bf2_pack(x[2], x[3]),
                                              bf2_pack(x[4], x[5]), bf2_pack(x[6], x[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t swap2(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(hi, lo);
}

// GL lanes per head (a power of two >= D / 16); D % 16 == 0, R % 16 == 0, 16-byte aligned rows.
// kPack: tokens share a warp (a form of its own: asking costs the others 4 %).
template <int DT, int GL, bool kInter, bool kPack>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int ES = DT == DLLM_BF16 ? 2 : 4;
  constexpr int HPW = 32 / GL;  // heads a warp holds at once
  constexpr int kHpwLog2 = HPW == 1 ? 0 : HPW == 2 ? 1 : HPW == 4 ? 2 : HPW == 8 ? 3 : HPW == 16 ? 4 : 5;
  const unsigned warp = blockIdx.x * (kThreads / 32u) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const unsigned per_token = p.chunks[0] + p.chunks[1];
  const unsigned group = warp / per_token;  // of the tokens that share a warp
  int chunk = static_cast<int>(warp - group * per_token);
  const int sub = lane % GL;
  const int pack_log2 = kPack ? p.pack_log2 : 0;
  const int heads_log2 = kHpwLog2 - pack_log2;  // of a token at once
  const int slot = (lane / GL) & ((1 << heads_log2) - 1);
  const unsigned token = (group << pack_log2) + (lane / GL >> heads_log2);
  const bool valid = token < p.tokens;
  if (!kPack && !valid) return;
  const int b = static_cast<int>(token / static_cast<unsigned>(p.n));
  const int i = static_cast<int>(token) - b * p.n;
  // looked at when the loads are under way
  const int pos = kPack && !valid ? -1 : p.pos ? p.pos[b * p.pos_stride + i] : 0;
  const int side = chunk >= p.chunks[0];
  if (side) chunk -= p.chunks[0];
  const Side& s = p.s[side];

  const bool active = sub < p.D / 16;
  const bool turns = sub < p.R / 16;
  // the lane's two pieces of eight channels: both halves of its pairs, or side by side
  const int o0 = !turns || kInter ? 16 * sub : 8 * sub;
  const int o1 = !turns || kInter ? o0 + 8 : p.R / 2 + o0;
  const char* x = s.x + b * s.xb + i * s.xt;
  char* y = s.y + b * s.yb + i * s.yt;
  const int at_once = 1 << heads_log2;
  const int h0 = chunk * p.units * at_once + slot;
  Piece<DT> a0[kUnits], a1[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    a0[u] = Piece<DT>{};
    a1[u] = Piece<DT>{};
    const int h = h0 + u * at_once;
    if (u < p.units && active && (!kPack || valid) && h < s.heads) {
      a0[u] = load_piece<DT>(x + h * s.xh + o0 * ES);
      a1[u] = load_piece<DT>(x + h * s.xh + o1 * ES);
    }
  }
  if (kPack ? !__any_sync(kFull, pos >= 0) : pos < 0) return;
  // factors of a piece's own channels and of their partners' (two channels a word)
  uint64_t own[2][4], other[2][4];
  {
    float w0[8], w1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w0[e] = w1[e] = 1.f;
    if (s.w && active) {
      unpack<DT>(load_piece<DT>(s.w + o0 * ES), w0);
      unpack<DT>(load_piece<DT>(s.w + o1 * ES), w1);
    }
    if (turns) {
      float cs[8], sn[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        phase_sincos(pos, __ldg(p.phases + 8 * sub + e), p.magnitude, cs[e], sn[e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kInter) {  // a piece is four pairs
          own[0][j] = pack2(w0[2 * j] * cs[j], w0[2 * j + 1] * cs[j]);
          other[0][j] = pack2(-w0[2 * j + 1] * sn[j], w0[2 * j] * sn[j]);
          own[1][j] = pack2(w1[2 * j] * cs[4 + j], w1[2 * j + 1] * cs[4 + j]);
          other[1][j] = pack2(-w1[2 * j + 1] * sn[4 + j], w1[2 * j] * sn[4 + j]);
        } else {
          own[0][j] = pack2(w0[2 * j] * cs[2 * j], w0[2 * j + 1] * cs[2 * j + 1]);
          other[0][j] = pack2(-w1[2 * j] * sn[2 * j], -w1[2 * j + 1] * sn[2 * j + 1]);
          own[1][j] = pack2(w1[2 * j] * cs[2 * j], w1[2 * j + 1] * cs[2 * j + 1]);
          other[1][j] = pack2(w0[2 * j] * sn[2 * j], w0[2 * j + 1] * sn[2 * j + 1]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        own[0][j] = pack2(w0[2 * j], w0[2 * j + 1]);
        own[1][j] = pack2(w1[2 * j], w1[2 * j + 1]);
        other[0][j] = other[1][j] = 0;
      }
    }
  }
  const float inv_d = 1.f / static_cast<float>(p.D);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (u >= p.units) break;
    const int h = h0 + u * at_once;
    uint64_t v[2][4];
    {
      float f0[8], f1[8];
      unpack<DT>(a0[u], f0);
      unpack<DT>(a1[u], f1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[0][j] = pack2(f0[2 * j], f0[2 * j + 1]);
        v[1][j] = pack2(f1[2 * j], f1[2 * j + 1]);
      }
    }
    float r = 1.f;
    if (p.norm) {
      uint64_t q0 = 0, q1 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q0 = fma2(v[0][j], v[0][j], q0);
        q1 = fma2(v[1][j], v[1][j], q1);
      }
      float lo, hi;
      unpack2(add2(q0, q1), lo, hi);
      float ss = lo + hi;
#pragma unroll
      for (int o = GL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      r = rsqrtf(ss * inv_d + p.eps);
    }
    const uint64_t r2 = pack2(r, r);
    float out[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint64_t t;
        if (turns)
          t = fma2(v[k][j], own[k][j], mul2(kInter ? swap2(v[k][j]) : v[k ^ 1][j], other[k][j]));
        else
          t = mul2(v[k][j], own[k][j]);
        unpack2(mul2(t, r2), out[k][2 * j], out[k][2 * j + 1]);
      }
    }
    if (active && (!kPack || pos >= 0) && h < s.heads) {
      store_piece<DT>(y + h * s.yh + o0 * ES, out[0]);
      store_piece<DT>(y + h * s.yh + o1 * ES, out[1]);
    }
  }
}

__device__ __forceinline__ void store_value(char* p, int dtype, float v) {
  if (dtype == DLLM_F32)
    *reinterpret_cast<float*>(p) = v;
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(bf2_pack(v, 0.f));
}

// Any layout, one warp per head, element by element.
__global__ void __launch_bounds__(kThreads)
    norm_rope_any_kernel(const __grid_constant__ NormRopeParams p, int dtype) {
  const int es = dtype == DLLM_BF16 ? 2 : 4;
  const int64_t warp = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int total = p.s[0].heads + p.s[1].heads;
  const int64_t token = warp / total;
  if (token >= p.tokens) return;
  const int h = static_cast<int>(warp - token * total);
  const int b = static_cast<int>(token / p.n), i = static_cast<int>(token - static_cast<int64_t>(b) * p.n);
  const int pos = p.pos ? p.pos[b * p.pos_stride + i] : 0;
  if (pos < 0) return;
  const Side& s = p.s[h < p.s[0].heads ? 0 : 1];
  const int hl = h < p.s[0].heads ? h : h - p.s[0].heads;
  const char* x = s.x + b * s.xb + i * s.xt + hl * s.xh;
  char* y = s.y + b * s.yb + i * s.yt + hl * s.yh;
  float r = 1.f;
  if (p.norm) {
    float ss = 0.f;
    for (int c = lane; c < p.D; c += 32) {
      const float v = load_logit(x, dtype, c);
      ss = fmaf(v, v, ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    r = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
  }
  const bool weighted = p.norm && s.w;
  auto value = [&](int c) {
    float v = load_logit(x, dtype, c);
    if (p.norm) v *= r;
    return weighted ? v * load_logit(s.w, dtype, c) : v;
  };
  // a lane reads the channels it writes before it writes them: in place is safe
  for (int j = lane; j < p.R / 2; j += 32) {
    const int ca = p.interleaved ? 2 * j : j, cc = p.interleaved ? 2 * j + 1 : j + p.R / 2;
    float cs, sn;
    phase_sincos(pos, __ldg(p.phases + j), p.magnitude, cs, sn);
    const float a = value(ca), c = value(cc);
    store_value(y + static_cast<int64_t>(ca) * es, dtype, a * cs - c * sn);
    store_value(y + static_cast<int64_t>(cc) * es, dtype, c * cs + a * sn);
  }
  for (int c = p.R + lane; c < p.D; c += 32) store_value(y + static_cast<int64_t>(c) * es, dtype, value(c));
}

__global__ void rope_phases_kernel(dllm_rope r, int64_t* phases) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  pdl_wait();
  if (i >= r.rotary_dim / 2) return;
  const double two_pi = 6.283185307179586476925;
  const double g = pow(r.base, -2.0 * i / r.rotary_dim);
  double f = g / r.factor;
  if (r.scaling == DLLM_ROPE_BANDS) {
    const double turns = r.original_len * g / two_pi;
    const double w = fmin(1.0, fmax(0.0, (turns - r.slow_turns) / (r.fast_turns - r.slow_turns)));
    f = (1.0 - w) * f + w * g;
  }
  phases[i] = __double2ll_rn(f / two_pi * 18446744073709551616.0);
}

bool rows_aligned(const Side& s) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(s.x) | reinterpret_cast<uintptr_t>(s.y) |
                         reinterpret_cast<uintptr_t>(s.w) | static_cast<uintptr_t>(s.xb) |
                         static_cast<uintptr_t>(s.xt) | static_cast<uintptr_t>(s.xh) |
                         static_cast<uintptr_t>(s.yb) | static_cast<uintptr_t>(s.yt) |
                         static_cast<uintptr_t>(s.yh);
  return s.heads == 0 || bits % 16 == 0;
}

template <int DT, int GL>
cudaError_t launch_vec(NormRopeParams& p, int sm_count, cudaStream_t stream) {
  constexpr int HPW = 32 / GL;
  // With at most half a warp's heads, tokens share a warp (9944 tokens of 1 + 1 heads of 80 channels:
  // 5.6 us, 19.1 with a token a warp; 16384 of 2 + 1 heads of 128: 12.2, 29.2).  Otherwise as many sets of
  // heads a warp (more loads on the way, sines and cosines used more often) as leave 12 warps an SM; a
  // call with fewer tokens spreads each over more warps.  512 tokens of 32 + 8 heads take 3.9 us in 17
  // warps an SM of one set, 4.4 in 8 of two; 999 tokens of 7 + 7 heads of 80 fp32 channels 4.6 us in 13
  // warps of two, 5.4 in 26 of one.  Over 54 sizes of 128 to 4096 tokens the other thresholds come to
  // (mean, best, worst, as parts of the time with 12): 6: 0.99, 0.84, 1.28; 8: 1.01, 0.93, 1.28;
  // 16: 1.03, 0.84, 1.31; 24: 1.04, 0.79, 1.34.
  const int most = p.s[0].heads > p.s[1].heads ? p.s[0].heads : p.s[1].heads;
  p.pack_log2 = 0;
  while ((most << (p.pack_log2 + 1)) <= HPW) ++p.pack_log2;
  int64_t warps = 0;
  for (p.units = p.pack_log2 > 0 ? 1 : kUnits;; p.units /= 2) {
    const int heads = p.units * HPW >> p.pack_log2;
    for (int j = 0; j < 2; ++j) p.chunks[j] = (p.s[j].heads + heads - 1) / heads;
    warps = ((p.tokens + (1 << p.pack_log2) - 1) >> p.pack_log2) * (p.chunks[0] + p.chunks[1]);
    if (p.units == 1 || warps >= static_cast<int64_t>(sm_count) * 12) break;
  }
  const dim3 grid(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
  auto run = [&](auto kern) { return launch_dependent(kern, grid, dim3(kThreads), 0, stream, p); };
  if constexpr (HPW > 1) {
    if (p.pack_log2 > 0)
      return p.interleaved ? run(norm_rope_kernel<DT, GL, true, true>)
                           : run(norm_rope_kernel<DT, GL, false, true>);
  }
  return p.interleaved ? run(norm_rope_kernel<DT, GL, true, false>)
                       : run(norm_rope_kernel<DT, GL, false, false>);
}

template <int DT>
cudaError_t launch_vec_dt(NormRopeParams& p, int sm_count, cudaStream_t stream) {
  const int lanes = p.D / 16;
  if (lanes <= 2) return launch_vec<DT, 2>(p, sm_count, stream);
  if (lanes <= 4) return launch_vec<DT, 4>(p, sm_count, stream);
  if (lanes <= 8) return launch_vec<DT, 8>(p, sm_count, stream);
  if (lanes <= 16) return launch_vec<DT, 16>(p, sm_count, stream);
  return launch_vec<DT, 32>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const dllm_heads* q, const dllm_heads* q_out, const dllm_heads* k,
                             const dllm_heads* k_out, int B, int n, int D, const int32_t* pos,
                             int64_t pos_stride, const int64_t* phases, int R, bool interleaved,
                             float magnitude, bool norm, const void* q_weight, const void* k_weight,
                             float eps, int sm_count, cudaStream_t stream) {
  NormRopeParams p{};
  const dllm_heads* in[2] = {q, k};
  const dllm_heads* out[2] = {q_out, k_out};
  const void* w[2] = {q_weight, k_weight};
  int dtype = DLLM_F32;
  for (int j = 0; j < 2; ++j) {
    if (!in[j]) continue;
    dtype = in[j]->dtype;
    const int es = dtype == DLLM_BF16 ? 2 : 4;
    p.s[j] = Side{static_cast<const char*>(in[j]->data), static_cast<char*>(out[j]->data),
                  static_cast<const char*>(w[j]), in[j]->heads,
                  in[j]->batch_stride * es, in[j]->token_stride * es, in[j]->head_stride * es,
                  out[j]->batch_stride * es, out[j]->token_stride * es, out[j]->head_stride * es};
  }
  p.pos = pos;
  p.pos_stride = pos_stride;
  p.phases = phases;
  p.n = n;
  p.tokens = static_cast<int64_t>(B) * n;
  p.D = D;
  p.R = R;
  p.interleaved = interleaved;
  p.norm = norm;
  p.magnitude = magnitude;
  p.eps = eps;
  if (D % 16 == 0 && D <= 512 && R % 16 == 0 && rows_aligned(p.s[0]) && rows_aligned(p.s[1]))
    return dtype == DLLM_BF16 ? launch_vec_dt<DLLM_BF16>(p, sm_count, stream)
                              : launch_vec_dt<DLLM_F32>(p, sm_count, stream);
  const int64_t warps = p.tokens * (p.s[0].heads + p.s[1].heads);
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  return launch_dependent(norm_rope_any_kernel, dim3(static_cast<unsigned>(blocks)),
                          dim3(kThreads), 0, stream, p, dtype);
}

cudaError_t launch_rope_phases(const dllm_rope& rope, int64_t* phases, cudaStream_t stream) {
  return launch_dependent(rope_phases_kernel, dim3((rope.rotary_dim / 2 + 127) / 128), dim3(128), 0,
                          stream, rope, phases);
}

}  // namespace dllm

// Softmax weights as 64-bit integers, so that sums over a vocabulary are exact whatever their order.
//
// weight(z) = exp((z - m) / T) in units of 2^-42, m the row's maximum: e^x = 2^(k + j/32) * e^r with
// |r| <= ln2/64, a table of 2^(j/32) and a short series for e^r (Tang, "Table-driven implementation
// of the exponential function in IEEE floating-point arithmetic", 1989), carried in pairs of floats:
// relative error below 2^-36, and half a unit.  2^20 weights of at most one sum to less than 2^63.
//
// Why so exact: a draw compares a running sum with u * total, so a sum that is off by a share e of
// the total moves the border of every token; a vocabulary of 10^5 open candidates has as many
// borders, and sums in 32 bits (e = 10^-7 .. 10^-6) would draw another token in one row of ten to a
// hundred.  Double precision would do, but this GPU computes it at a 64th of the 32-bit rate.
#pragma once

#include "common.cuh"

namespace dllm {

constexpr int kWeightBits = 42;

// log2(e) / T as a pair of floats
struct InvTemp {
  float hi, lo;
};

// 2^(j/32), high and low part
__device__ const float2 kPow2Table[32] = {
    {0x1.000000p+0f, 0x0.0p+0f},        {0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x1.0b5586p+0f, 0x1.9f3122p-25f},  {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f},  {0x1.29e9e0p+0f, -0x1.5c0424p-25f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f},  {0x1.371a74p+0f, -0x1.18aac6p-25f},
    {0x1.3dea64p+0f, 0x1.824684p-25f},  {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f},
    {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b550p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},  {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f},  {0x1.93737cp+0f, -0x1.e64744p-25f},
    {0x1.9c4918p+0f, 0x1.51f848p-27f},  {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f},
    {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f},  {0x1.f50766p+0f, -0x1.246eb0p-26f},
};

// How far z lies below m, in octaves of weight (to 32 bits; monotone in z).  NaN for a NaN.
__device__ __forceinline__ float octaves_below(float z, float m, InvTemp t) { return (m - z) * t.hi; }

// The weight of z; 0 where it is below a unit, and for a NaN.  `table`: kPow2Table, in shared
// memory.
__device__ __forceinline__ uint64_t weight_fixed(float z, float m, InvTemp t, const float2* table) {
  const float dh = z - m;                      // z - m = dh + dl
  const float back = dh + m;
  const float dl = (z - back) + ((back - dh) - m);
  const float yh = dh * t.hi;                  // (z - m) log2(e) / T = yh + yl
  const float yl = fmaf(dh, t.hi, -yh) + fmaf(dh, t.lo, dl * t.hi);
  if (!(yh > -static_cast<float>(kWeightBits))) return 0;
  const int n = __float2int_rn(yh * 32.f);     // yh = n / 32 + g
  const float g = fmaf(static_cast<float>(n), -0.03125f, yh);
  const float2 p = table[n & 31];
  // r = (g + yl) ln2 = rh + rl;  e^r - 1 = rh + s
  constexpr float kLn2Hi = 0x1.62e430p-1f, kLn2Lo = -0x1.05c610p-29f;
  const float rh = g * kLn2Hi;
  const float rl = fmaf(g, kLn2Hi, -rh) + fmaf(g, kLn2Lo, yl * kLn2Hi);
  const float q = fmaf(rh, fmaf(rh, fmaf(rh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
  const float s = fmaf(rh * rh, q, fmaf(rl, rh, rl));
  // 2^(j/32) e^r = hi + lo
  const float a = p.x * rh;
  const float hi = p.x + a;
  const float lo = (a - (hi - p.x)) + (fmaf(p.x, rh, -a) + fmaf(p.x, s, fmaf(p.y, rh, p.y)));
  // hi is a multiple of 2^-24 in (0.98, 2.02)
  const int64_t whole = static_cast<int64_t>(static_cast<int>(hi * 0x1p24f)) * (int64_t{1} << (kWeightBits - 24)) +
                        __float2int_rn(lo * static_cast<float>(int64_t{1} << kWeightBits));
  const int down = -(n >> 5);                  // 0 .. 42
  return static_cast<uint64_t>(down > 0 ? (whole + (int64_t{1} << (down - 1))) >> down : whole);
}

}  // namespace dllm

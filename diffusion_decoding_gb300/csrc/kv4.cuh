// Device helpers of the 4-bit key/value cache (sm_103a).
//
// A group is 32 channels of one entry of one head: a step s with three significant bits and a
// zero point z; code n stands for s * (n - z).  (16 + n) and (16 + z) have five significant bits
// and s three, so (16 + n) * s, (16 + z) * s and their difference s * (n - z) (four bits and sign
// times three) are all exact in bf16: one packed bf16 fma turns two codes into two exact values.
// The bits of 16 + n are 0x4180 | n << 3, so no integer conversion is needed.
#pragma once

#include "common.cuh"

namespace dllm {

constexpr int kKv4Group = 32;
constexpr uint32_t kKv4NaNParam = 0x7FE0u;  // step of a group that held a NaN or an infinity

// The group of this param word reads as NaN (its step is no finite number).
__device__ __forceinline__ bool kv4_nan(uint32_t param) { return (param & 0x7F80u) == 0x7F80u; }

// packed bf16 arithmetic on raw words
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf2_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Step and offset of two groups from two param words in the halves of `pp`: value pair =
// fma(16 + n, step, offset).  offset = -(16 + z) * step, exact.
struct Kv4Scale {
  uint32_t step, offset;
};
__device__ __forceinline__ Kv4Scale kv4_scale(uint32_t pp) {
  Kv4Scale r;
  r.step = pp & 0xFFE0FFE0u;
  const uint32_t z16 = ((pp << 3) & 0x00780078u) | 0xC180C180u;  // -(16 + z)
  r.offset = bf2_fma(z16, r.step, 0x80008000u);                  // + (-0): keeps the product
  return r;
}

// Channels j and j + 4 of the eight in `w` (j = 0..3), as exact bf16 values.
template <int J>
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, const Kv4Scale& sc) {
  const uint32_t t = J == 0 ? (w << 3) : (w >> (4 * J - 3 < 0 ? 0 : 4 * J - 3));
  uint32_t n;  // (t & mask) | bits of 16, one instruction
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(n) : "r"(t), "r"(0x00780078u), "r"(0x41804180u));
  return bf2_fma(n, sc.step, sc.offset);
}

// Page of entry p of one sequence's table row, -1 when absent (p within the table).
__device__ __forceinline__ int kv4_page(const int32_t* table_row, int table_pages, int pages,
                                        int page_size, int p) {
  const int t = p / page_size;
  if (p < 0 || t >= table_pages) return -1;
  const int pg = __ldg(table_row + t);
  return pg >= 0 && pg < pages ? pg : -1;
}

}  // namespace dllm

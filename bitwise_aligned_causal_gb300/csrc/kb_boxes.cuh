// kb_boxes.cuh -- the whole-number grid of key-block boxes and of the queries
// that are scored against them (kb_append.cu writes boxes, kb_select.cu reads
// them).
//
// A vector with largest magnitude a lies on the grid of step 2^(E-7), E the
// smallest integer in [-100, 100] with a <= 127 * 2^(E-7); beyond the range
// values saturate.  Grid values are whole numbers of at most 7 bits times a
// power of two, so bf16 holds them, their products are exact in fp32, and so
// is every sum of 256 products (below 2^22 steps of one common power of two),
// in any order and on the tensor core.
#pragma once

#include <cstdint>

namespace kb {

__device__ __forceinline__ int grid_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 126 + ((bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);   // m > 127/128
  return min(max(e, -100), 100);
}

// 2^n for n in [-126, 127].
__device__ __forceinline__ float exp2i(int n) { return __int_as_float((n + 127) << 23); }

// rint of |x| < 2^22 (ties to even): at 1.5 * 2^23 and above fp32 has no
// fraction bits, so the sum rounds to a whole number.  Two additions, where a
// conversion instruction takes a quarter-rate pipe.
__device__ __forceinline__ float rint_small(float x) { return __fsub_rn(__fadd_rn(x, 12582912.0f), 12582912.0f); }

// The four heads' values of one channel as whole numbers of 2^(E-15), summed
// (below 2^17, so every step is exact); values beyond the grid saturate.
__device__ __forceinline__ float whole_sum(const float (&q)[4], float scale) {
  float u = 0.0f;
#pragma unroll
  for (int h = 0; h < 4; ++h)
    u = __fadd_rn(u, rint_small(fminf(fmaxf(__fmul_rn(q[h], scale), -32512.0f), 32512.0f)));
  return u;
}

// Share of a block's score of eight channels: box bounds hi, lo (bf16 pairs),
// np and nm the positive and negative parts of n.
__device__ __forceinline__ float box_dot(const uint4& hi, const uint4& lo, const float (&np)[8], const float (&nm)[8]) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = __fmaf_rn(np[2 * i], __uint_as_float(h[i] << 16), s);
    s = __fmaf_rn(nm[2 * i], __uint_as_float(l[i] << 16), s);
    s = __fmaf_rn(np[2 * i + 1], __uint_as_float(h[i] & 0xFFFF0000u), s);
    s = __fmaf_rn(nm[2 * i + 1], __uint_as_float(l[i] & 0xFFFF0000u), s);
  }
  return s;
}

}  // namespace kb

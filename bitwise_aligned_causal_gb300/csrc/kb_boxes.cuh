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

// Rounding to whole numbers without conversion instructions (a quarter-rate
// pipe): for |x| < 2^22, x + 1.5 * 2^23 has no fraction bits left, so the sum
// rounds to a whole number (ties to even) and its bit pattern is that of
// 1.5 * 2^23 plus the number.
constexpr float kWholeAt = 12582912.0f;              // 1.5 * 2^23
constexpr uint32_t kWholeBits = 0x4B400000u;         // its bit pattern
// rint(x * scale), scale a power of two.
__device__ __forceinline__ float rint_scaled(float x, float scale) { return __fsub_rn(__fmaf_rn(x, scale, kWholeAt), kWholeAt); }
// Beyond this magnitude a value lies off the grid (E stops at 100) and saturates.
constexpr float kGridMax = 127.0f * 9.903520314283042e27f;   // 127 * 2^93

// The four heads' values of one channel as whole numbers of 2^(E-15), summed
// (below 2^17, so every step is exact); values beyond the grid saturate.
__device__ __forceinline__ float whole_sum(float q0, float q1, float q2, float q3, float scale) {
  const uint32_t u = __float_as_uint(__fmaf_rn(q0, scale, kWholeAt)) + __float_as_uint(__fmaf_rn(q1, scale, kWholeAt)) +
                     __float_as_uint(__fmaf_rn(q2, scale, kWholeAt)) + __float_as_uint(__fmaf_rn(q3, scale, kWholeAt));
  return __fsub_rn(__uint_as_float(u - 3u * kWholeBits), kWholeAt);        // modulo 2^32
}
__device__ __forceinline__ float saturated(float q) { return fminf(fmaxf(q, -kGridMax), kGridMax); }
// Both bounds of a bf16 pair within the grid (127 * 2^93 is bf16 0x717E): infinities saturate, NaN becomes the least value.
// The library's own boxes lie there; others must not make scores without a place in an order.
__device__ __forceinline__ uint32_t saturated_bf16x2(uint32_t w) {
  asm("max.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0xF17EF17Eu));
  asm("min.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0x717E717Eu));
  return w;
}
// The same for a finished score: on the grid it is below 2^114 (128 * 127 * 127 * 2^93).
__device__ __forceinline__ float saturated_score(float s) {
  constexpr float kScoreMax = 1.329227995784916e36f;   // 2^120
  return fminf(fmaxf(s, -kScoreMax), kScoreMax);
}

// The bounds that count in the score of two channels (bf16 pairs): the upper
// one where n is positive, the lower one elsewhere; `up` has all bits of a
// positive channel's half set.
__device__ __forceinline__ float box_dot(const uint4& hi, const uint4& lo, const uint32_t (&up)[4], const float (&n)[8]) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (h[i] & up[i]) | (l[i] & ~up[i]);
    s = __fmaf_rn(n[2 * i], __uint_as_float(w << 16), s);
    s = __fmaf_rn(n[2 * i + 1], __uint_as_float(w & 0xFFFF0000u), s);
  }
  return s;
}

}  // namespace kb

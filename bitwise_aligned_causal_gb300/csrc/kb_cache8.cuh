// kb_cache8.cuh -- values of a KV cache held in 8 bits (kb_cache8.cu writes
// them, kb_decode.cu and kb_cache8.cu read them).
//
// A block of 128 keys of one KV head has an exponent E; its bytes are e4m3
// numbers without subnormals and stand for themselves times 2^E:
//   E = the smallest integer in [-100, 100] with max |x| <= 448 * 2^E, or 127
//       when a value is not finite (every value of the block then reads NaN)
//   x is rounded to four significant bits (ties to even), and to zero where
//       the rounded magnitude lies below 2^(E-6)
// Rounding to four bits twice is rounding once, what falls to zero depends on
// the final E alone, and the E of all keys is the largest E of any part of
// them: a block's bytes are the same for any split of its keys into appends.
// A byte times 2^E has four significant bits and lies within bf16's range, so
// the cache stands for a bf16 cache exactly.
#pragma once

#include <cstdint>

#include "kb_contract.cuh"

namespace kb {

constexpr int kExpLow = -100, kExpHigh = 100;
constexpr int kExpNaN = 127;                       // the block holds a value that is not finite
constexpr uint32_t kByteNaN = 0x7Fu;               // and its bytes

// E of a largest magnitude given by its fp32 bits.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kExpNaN;
  const int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // m > 1.75
  return min(max(e, kExpLow), kExpHigh);
}

// A block's exponent as a cache holds it.
__device__ __forceinline__ int held_exponent(int e) { return e == kExpNaN ? e : min(max(e, kExpLow), kExpHigh); }

// The byte of a value (fp32 bits) in a block of exponent E.
__device__ __forceinline__ uint32_t to_byte(uint32_t bits, int E) {
  const uint32_t mag = bits & 0x7FFFFFFFu;
  const uint32_t r = (mag + 0x7FFFFu + ((mag >> 20) & 1u)) >> 20;      // biased exponent and three mantissa bits
  const int m = static_cast<int>(r) - ((120 + E) << 3);
  const uint32_t byte = m < 8 ? 0u : static_cast<uint32_t>(min(m, 0x7E));
  return E == kExpNaN ? kByteNaN : (byte | ((bits >> 31) << 7));
}

// A byte of exponent E - d in a block whose exponent has become E (d > 0).
__device__ __forceinline__ uint32_t regrid_byte(uint32_t byte, int d) {
  const int m = static_cast<int>(byte & 0x7Fu) - 8 * d;
  return (byte & 0x80u) | (m < 8 ? 0u : static_cast<uint32_t>(m));
}

// 2^E as factors of the raw values below (bf16 pairs): `second` is 1 unless E
// lies above what one factor reaches.
struct Scale8 {
  uint32_t first, second;
  bool two;
};
__device__ __forceinline__ Scale8 scale8(int held) {
  const int E = held_exponent(held);
  Scale8 s;
  s.two = E > 7 && E != kExpNaN;
  const uint32_t f = E == kExpNaN ? 0x7FC0u : static_cast<uint32_t>((s.two ? 120 : 120 + E) + 127) << 7;
  s.first = f | (f << 16);
  const uint32_t g = static_cast<uint32_t>((s.two ? E : 0) + 127) << 7;
  s.second = g | (g << 16);
  return s;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four bytes as two bf16 pairs.  A byte's exponent and mantissa moved to the
// bf16 places give its value times 2^-120 (the biases differ by 120, and the
// product is exact for e4m3's own subnormals too).  The permutation puts eight
// copies of a byte's sign above it, so one shift and one mask place all three
// fields.
__device__ __forceinline__ uint2 values8(uint32_t w, uint32_t first) {
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));         // sign byte 1 | byte 1 | sign byte 0 | byte 0
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(b) : "r"(w));
  return make_uint2(mul_bf16x2((a << 4) & 0x87F087F0u, first), mul_bf16x2((b << 4) & 0x87F087F0u, first));
}

// Sixteen bytes as sixteen bf16 values.
__device__ __forceinline__ void values8x16(const uint4& w, uint32_t first, uint4& lo, uint4& hi) {
  const uint2 a = values8(w.x, first), b = values8(w.y, first), c = values8(w.z, first), d = values8(w.w, first);
  lo = make_uint4(a.x, a.y, b.x, b.y);
  hi = make_uint4(c.x, c.y, d.x, d.y);
}

// The same for any exponent: a second factor where one does not reach.
__device__ __forceinline__ uint4 scaled_again(const uint4& v, uint32_t second) {
  return make_uint4(mul_bf16x2(v.x, second), mul_bf16x2(v.y, second), mul_bf16x2(v.z, second), mul_bf16x2(v.w, second));
}
__device__ __forceinline__ void values8x16(const uint4& w, const Scale8& s, uint4& lo, uint4& hi) {
  values8x16(w, s.first, lo, hi);
  if (s.two) {                                     // one decision per block
    lo = scaled_again(lo, s.second);
    hi = scaled_again(hi, s.second);
  }
}

}  // namespace kb

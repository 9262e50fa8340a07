// kb_bwd.cuh -- what the dense and the block-sparse backward kernels share:
// the elementwise step from S, dP to P, dS and the paired MMA issue.
#pragma once

#include "kb_contract.cuh"

namespace kb {

constexpr float kLog2e = 1.4426950408889634f;          // log2(e), to turn a natural-log lse into base 2
constexpr float kInvSqrtD = 0.088388347648318440f;     // 1 / sqrt(128)

__device__ __forceinline__ void drain_wait_b(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 50000000ull) break;
}

// P = 2^(s c - lse2) and dS = P (dP - delta) of two adjacent columns, as
// packed f32x2 operations (the same IEEE operations, so the same bits, as the
// scalar fma, subtraction and product): `nl` and `nd` hold -lse2 and -delta.
// A masked P is zero before dS is formed, so its dS is a signed zero as in the
// scalar form.  Both values go out as one bf16 pair each.
template <bool kMask>
__device__ __forceinline__ void p_ds_pair(uint32_t s0, uint32_t s1, uint32_t dp0, uint32_t dp1, float2 c2,
                                          float2 nl, float2 nd, bool m0, bool m1, uint32_t& p_bf,
                                          uint32_t& ds_bf) {
  const float2 a = __ffma2_rn(make_float2(__uint_as_float(s0), __uint_as_float(s1)), c2, nl);
  float2 pp = make_float2(ex2_approx(a.x), ex2_approx(a.y));
  if (kMask) {
    if (m0) pp.x = 0.0f;
    if (m1) pp.y = 0.0f;
  }
  const float2 d = __fmul2_rn(pp, __fadd2_rn(make_float2(__uint_as_float(dp0), __uint_as_float(dp1)), nd));
  p_bf = pack_bf16x2(pp.x, pp.y);
  ds_bf = pack_bf16x2(d.x, d.y);
}

// dS alone of the same pair, as the sum of two bf16 values each (16 bits of
// mantissa), for a product that must not lose it to rounding.  The mask comes
// last: a row that lists nothing has lse = -inf, and its q, dO and delta may be
// anything (a padded row's NaN).
template <bool kMask>
__device__ __forceinline__ void ds_split_pair(uint32_t s0, uint32_t s1, uint32_t dp0, uint32_t dp1, float2 c2,
                                              float2 nl, float2 nd, bool m0, bool m1, uint32_t& high,
                                              uint32_t& low) {
  const float2 a = __ffma2_rn(make_float2(__uint_as_float(s0), __uint_as_float(s1)), c2, nl);
  const float2 pp = make_float2(ex2_approx(a.x), ex2_approx(a.y));
  float2 d = __fmul2_rn(pp, __fadd2_rn(make_float2(__uint_as_float(dp0), __uint_as_float(dp1)), nd));
  if (kMask) {
    if (m0) d.x = 0.0f;
    if (m1) d.y = 0.0f;
  }
  high = pack_bf16x2(d.x, d.y);
  const float2 rest = __fadd2_rn(d, make_float2(-__uint_as_float(high << 16), -__uint_as_float(high & 0xFFFF0000u)));
  low = pack_bf16x2(rest.x, rest.y);
}

// Two independent products of the same shape, their K steps interleaved
// (each accumulator still takes its eight steps in ascending order): the
// tensor pipe overlaps the two dependency chains.
__device__ __forceinline__ void issue_qk_pair(uint32_t d1, uint32_t a1, uint32_t b1, uint32_t d2, uint32_t a2,
                                              uint32_t b2) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    mma_ss(d1, desc_kmajor(a1, kk, 1024u, kSlabBytes), desc_kmajor(b1, kk, 1024u, kSlabBytes), kIdescQK,
           kk > 0 ? 1u : 0u);
    mma_ss(d2, desc_kmajor(a2, kk, 1024u, kSlabBytes), desc_kmajor(b2, kk, 1024u, kSlabBytes), kIdescQK,
           kk > 0 ? 1u : 0u);
  }
}

template <int kFrom, int kTo>
__device__ __forceinline__ void issue_pv_pair(uint32_t d1, uint32_t a1_tmem, uint32_t b1, uint32_t d2,
                                              uint32_t a2_tmem, uint32_t b2, bool first) {
#pragma unroll
  for (int kk = kFrom; kk < kTo; ++kk) {
    const uint32_t acc = (first && kk == 0) ? 0u : 1u;
    mma_ts(d1, a1_tmem + static_cast<uint32_t>(kk) * 8u, desc_v(b1, kk), kIdescPV, acc);
    mma_ts(d2, a2_tmem + static_cast<uint32_t>(kk) * 8u, desc_v(b2, kk), kIdescPV, acc);
  }
}

// 16x256b loads of 32 columns (four repetitions) from two addresses, one
// wait: thread t gets lanes t/4 and t/4 + 8, columns 8r + 2(t%4) and
// 8r + 2(t%4) + 1 of repetition r in registers 4r, 4r+1 (first lane) and
// 4r+2, 4r+3 (second lane).
__device__ __forceinline__ void tmem_ld_16x256b_x4_pair_wait(uint32_t ta, uint32_t tb, uint32_t (&ra)[16],
                                                             uint32_t (&rb)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(ra[0]), "=r"(ra[1]), "=r"(ra[2]), "=r"(ra[3]), "=r"(ra[4]), "=r"(ra[5]), "=r"(ra[6]), "=r"(ra[7]),
        "=r"(ra[8]), "=r"(ra[9]), "=r"(ra[10]), "=r"(ra[11]), "=r"(ra[12]), "=r"(ra[13]), "=r"(ra[14]), "=r"(ra[15]),
        "=r"(rb[0]), "=r"(rb[1]), "=r"(rb[2]), "=r"(rb[3]), "=r"(rb[4]), "=r"(rb[5]), "=r"(rb[6]), "=r"(rb[7]),
        "=r"(rb[8]), "=r"(rb[9]), "=r"(rb[10]), "=r"(rb[11]), "=r"(rb[12]), "=r"(rb[13]), "=r"(rb[14]), "=r"(rb[15])
      : "r"(ta), "r"(tb)
      : "memory");
}
// 16x128b store of 16 columns (four repetitions): thread t writes lanes t/4
// and t/4 + 8, column 4r + t%4 of repetition r, from registers 2r and 2r+1.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

}  // namespace kb

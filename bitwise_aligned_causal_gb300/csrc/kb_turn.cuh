// kb_turn.cuh -- the rotation of a row's planes by eight lanes, shared by the
// kernels that turn queries and keys (kb_append.cu, kb_cache8.cu).
#pragma once

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

constexpr int kRowsPerWarp = 4;                 // eight lanes per row, two 16-byte chunks each

struct Turn {
  float2 cs[kPlanesPerLane];                    // (cos, sin) of the lane's planes
};

// The two 16-byte chunks of a row that lane u of its eight holds, and whether
// they are turned: the pairs of planes 8u..8u+7, or (beyond rot_dim) two
// chunks that pass unchanged.
struct LaneChunks {
  int c0, c1;
  bool turns;
};
__device__ __forceinline__ LaneChunks lane_chunks(int u, int rot_dim, bool interleaved) {
  const int m = rot_dim >> 4;                   // chunks of one half
  if (interleaved || u >= m) return LaneChunks{2 * u, 2 * u + 1, u < m};
  return LaneChunks{u, u + m, true};
}

__device__ __forceinline__ void load_turn(Turn& t, const float* table, long long pos, int rot_dim, int u, bool inverse) {
  const float4* src = reinterpret_cast<const float4*>(table + pos * rot_dim) + 4 * u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(src + i);
    t.cs[2 * i] = make_float2(v.x, inverse ? -v.y : v.y);
    t.cs[2 * i + 1] = make_float2(v.z, inverse ? -v.w : v.w);
  }
}

// The turn of planes 8u..8u+7 with a position per axis: `axes` holds the axis
// of each of them in one byte, `pos` the row's position on each axis.  Planes
// of one axis lie together in the usual layouts, so a lane's eight mostly
// share a table row and come in four wide loads.
__device__ __forceinline__ void load_turn_axes(Turn& t, const float* table, const int (&pos)[kMaxAxes], uint64_t axes,
                                               int rot_dim, int u, bool inverse) {
  auto pos_of = [&](int a) { return a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3]; };   // no indexed registers
  const int a0 = static_cast<int>(axes & 0xFFu);
  if (axes == static_cast<uint64_t>(a0) * 0x0101010101010101ull) {
    load_turn(t, table, pos_of(a0), rot_dim, u, inverse);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPlanesPerLane; ++i) {
    const int p = pos_of(static_cast<int>(axes >> (8 * i)) & 0xFF);
    const float2 v = __ldg(reinterpret_cast<const float2*>(table + static_cast<long long>(p) * rot_dim) + 8 * u + i);
    t.cs[i] = make_float2(v.x, inverse ? -v.y : v.y);
  }
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float turn_a(float a, float b, float2 cs) {
  return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turn_b(float a, float b, float2 cs) {
  return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// Turn the lane's two chunks in place.
__device__ __forceinline__ void turn_chunks(uint4& x, uint4& y, const Turn& t, bool interleaved) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
  uint32_t* b = reinterpret_cast<uint32_t*>(&y);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = lo_of(a[i]), a1 = hi_of(a[i]), b0 = lo_of(b[i]), b1 = hi_of(b[i]);
      a[i] = pack_bf16x2(turn_a(a0, a1, t.cs[i]), turn_b(a0, a1, t.cs[i]));
      b[i] = pack_bf16x2(turn_a(b0, b1, t.cs[4 + i]), turn_b(b0, b1, t.cs[4 + i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = lo_of(a[i]), a1 = hi_of(a[i]), b0 = lo_of(b[i]), b1 = hi_of(b[i]);
      a[i] = pack_bf16x2(turn_a(a0, b0, t.cs[2 * i]), turn_a(a1, b1, t.cs[2 * i + 1]));
      b[i] = pack_bf16x2(turn_b(a0, b0, t.cs[2 * i]), turn_b(a1, b1, t.cs[2 * i + 1]));
    }
  }
}

}  // namespace kb

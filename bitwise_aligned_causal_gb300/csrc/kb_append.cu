// kb_append.cu -- position rotation, appending keys and values to a KV cache,
// and the boxes of the cache's key blocks.
//
// Rotation.  A row x of 128 values at position p is turned in rot_dim / 2
// planes; plane i holds the values x[i], x[i + rot_dim/2] (or x[2i], x[2i+1]
// when interleaved) and turns by the angle p * inv_freq[i], whose cosine and
// sine come from a table [positions, rot_dim/2, 2] in fp32:
//   a' = a cos - b sin,   b' = b cos + a sin
// each as two fp32 products and one fp32 sum, rounded to bf16 once.  The
// operations are explicit round-to-nearest intrinsics, so a key has the same
// bits whether it was appended alone, in a chunk or with its whole prompt.
// The gradient of a rotation is the rotation by the negative angle.
//
// Box of a block of 128 keys: per channel an upper and a lower bound of its
// keys, on a grid of 127 steps either way.  With E the smallest integer in
// [-100, 100] for which the largest |key| is at most 127 * 2^(E-7):
//   upper = ceil(max * 2^(7-E)) * 2^(E-7),  lower = floor(min * 2^(7-E)) * 2^(E-7)
// which bf16 holds exactly.  ceil(ceil(x) / 2) = ceil(x / 2) and the rounded
// bound never needs a larger E than the keys do, so widening a box by later
// keys gives the box of all the keys at once: any split of a sequence into
// appends leaves the same bits.
//
// Bound: memory.  Everything is read once and written once (a token: 40 rows
// of 256 B in and 40 out, 8 value rows in and out, 512 B of table); a thread
// holds eight planes of a row, so the table's 64 bytes are fetched once for
// the five or six rows it turns.  Measured: the rotation of 32 heads x 16384
// positions 43.9 us (6.3 TB/s of bytes read and written; HBM copies at 6.8);
// an append of four ragged prompts of up to 4096, 39 to 51 us from GPU to GPU
// (274 MB read and written: 5.3 TB/s at 51; above the copy rate at 39, because
// a good part of the writes is still in L2 when the kernel ends), of one token
// of 16 sequences 5.0 us, a launch's latency.
#include <algorithm>

#include "kb_boxes.cuh"
#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

constexpr int kPlanesPerLane = 8;
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

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kNegInf2 = 0xFF80FF80u, kPosInf2 = 0x7F807F80u;

}  // namespace

// ------------------------------------------------------------------- table

// One thread per (position, plane): the angle and its cosine and sine in 64
// bits, since an fp32 angle at position 10^6 is already 0.03 off.
__global__ void __launch_bounds__(256) kb_rope_table_kernel(float* table, long long n, int planes,
                                                            const double* __restrict__ inv_freq) {
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  double s, c;
  sincos(static_cast<double>(i / planes) * inv_freq[i % planes], &s, &c);
  reinterpret_cast<float2*>(table)[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
}

cudaError_t launch_rope_table(float* table, int n_pos, int rot_dim, const double* inv_freq, cudaStream_t s) {
  const long long n = static_cast<long long>(n_pos) * (rot_dim / 2);
  kb_rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(table, n, rot_dim / 2, inv_freq);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- rotation

// A warp turns four heads of four consecutive positions.
__global__ void __launch_bounds__(256) kb_rope_kernel(const RopeArgs args) {
  if (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) return;
  const int lane = threadIdx.x & 31, u = lane & 7;
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int quads = (args.H + 3) / 4, tiles = (args.L + kRowsPerWarp - 1) / kRowsPerWarp;
  const long long per_b = static_cast<long long>(quads) * tiles;
  if (item >= per_b * args.B) return;
  const int b = static_cast<int>(item / per_b);
  const int rem = static_cast<int>(item % per_b);
  const int h0 = (rem % quads) * 4, i = (rem / quads) * kRowsPerWarp + (lane >> 3);
  if (i >= args.L) return;
  const LaneChunks lc = lane_chunks(u, args.rot_dim, args.interleaved);
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.x) + b * args.sb + h0 * args.sh +
                                                    i * args.sl);
  const long long hstep = args.sh / 8;
  uint4 x[4], y[4];
  const int nh = min(4, args.H - h0);
#pragma unroll
  for (int h = 0; h < 4; ++h)
    if (h < nh) {
      x[h] = src[h * hstep + lc.c0];
      y[h] = src[h * hstep + lc.c1];
    }
  if (lc.turns) {
    Turn t;
    load_turn(t, args.table, static_cast<long long>(args.start) + i, args.rot_dim, u, args.inverse);
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (h < nh) turn_chunks(x[h], y[h], t, args.interleaved);
  }
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.out) +
                                        ((static_cast<size_t>(b) * args.H + h0) * args.L + i) * kHeadDim);
  const size_t ostep = static_cast<size_t>(args.L) * (kHeadDim / 8);
#pragma unroll
  for (int h = 0; h < 4; ++h)
    if (h < nh) {
      dst[h * ostep + lc.c0] = x[h];
      dst[h * ostep + lc.c1] = y[h];
    }
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const long long warps = static_cast<long long>(a.B) * ((a.H + 3) / 4) * ((a.L + kRowsPerWarp - 1) / kRowsPerWarp);
  kb_rope_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ append

// One CTA per (batch, KV head, key block that the call's rows touch): turns
// the block's new keys and the four query heads at their positions, copies
// the values, and widens the block's box.  A block belongs to one CTA, so
// the box needs no atomics.  kAppend false: the cache is only read and the
// boxes of its blocks are made from nothing.
template <bool kAppend>
__global__ void __launch_bounds__(512) kb_append_kernel(const AppendArgs args) {
  __shared__ uint4 part[2][16][16];                     // [max, min][warp][chunk]
  __shared__ uint32_t amax_bits[4];
  // one decision for the CTA: the word may change while its threads read it
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(args.err) != 0)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  const int u = lane & 7, r4 = lane >> 3;
  const int c = static_cast<int>(blockIdx.x) / (args.B * args.Hkv);    // which touched block
  const int bg = static_cast<int>(blockIdx.x) % (args.B * args.Hkv);
  const int b = bg / args.Hkv, g = bg % args.Hkv;

  int start = args.start, len = args.L;
  if (args.starts != nullptr) start = args.starts[b];
  if (args.lens != nullptr) len = args.lens[b];
  if (start < 0 || len < 0 || len > args.L || start > args.kv_cap - len || (args.table != nullptr && start > args.n_pos - len)) {
    if (threadIdx.x == 0 && c == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
    return;
  }
  const int end = start + len;
  const int block = start / kTileKeys + c;
  if (len == 0 || block * kTileKeys >= end) return;
  const int p0 = max(start, block * kTileKeys), p1 = min(end, (block + 1) * kTileKeys);   // positions of this CTA
  // the block's place in the cache: `plane` rows of kv_rows keys, first key at `row`
  long long plane;
  int row, plane_rows;
  if (args.block_table != nullptr) {
    const int key = block * kTileKeys;
    const int pg = args.block_table[static_cast<size_t>(b) * args.pages_per_seq + key / args.page_size];
    if (pg < 0 || pg >= args.num_pages) {
      if (threadIdx.x == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return;
    }
    plane = static_cast<long long>(pg) * args.Hkv + g;
    row = key % args.page_size;
    plane_rows = args.page_size;
  } else {
    plane = static_cast<long long>(b) * args.Hkv + g;
    row = block * kTileKeys;
    plane_rows = args.kv_cap;
  }
  const size_t cache_row0 = static_cast<size_t>(plane) * plane_rows + row - static_cast<size_t>(block) * kTileKeys;
  // (row of the cache for position p: cache_row0 + p)
  const LaneChunks lc = lane_chunks(u, args.rot_dim, args.interleaved);
  uint4 mx[2], mn[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    mx[e] = make_uint4(kNegInf2, kNegInf2, kNegInf2, kNegInf2);
    mn[e] = make_uint4(kPosInf2, kPosInf2, kPosInf2, kPosInf2);
  }
  auto widen = [&](const uint4& v, uint4& hi, uint4& lo) {
    hi.x = bf16x2_max(hi.x, v.x); hi.y = bf16x2_max(hi.y, v.y); hi.z = bf16x2_max(hi.z, v.z); hi.w = bf16x2_max(hi.w, v.w);
    lo.x = bf16x2_min(lo.x, v.x); lo.y = bf16x2_min(lo.y, v.y); lo.z = bf16x2_min(lo.z, v.z); lo.w = bf16x2_min(lo.w, v.w);
  };
  if constexpr (kAppend) {
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(args.k) + b * args.ks[0] + g * args.ks[1];
    const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(args.v) + b * args.vs[0] + g * args.vs[1];
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(args.q) + b * args.qs[0] + (g * kGroup) * args.qs[1];
    const bool has_q = args.q != nullptr;
    for (int p = p0 + warp * kRowsPerWarp + r4; p < p1; p += n_warps * kRowsPerWarp) {
      const long long i = p - start;                     // row of the call's tensors
      const uint4* ksrc = reinterpret_cast<const uint4*>(kp + i * args.ks[2]);
      const uint4* vsrc = reinterpret_cast<const uint4*>(vp + i * args.vs[2]);
      uint4 kx = ksrc[lc.c0], ky = ksrc[lc.c1];
      const uint4 vx = vsrc[u], vy = vsrc[u + 8];
      uint4 qx[kGroup], qy[kGroup];
      if (has_q) {
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
          const uint4* qsrc = reinterpret_cast<const uint4*>(qp + h * args.qs[1] + i * args.qs[2]);
          qx[h] = qsrc[lc.c0];
          qy[h] = qsrc[lc.c1];
        }
      }
      if (args.table != nullptr && lc.turns) {
        Turn t;
        load_turn(t, args.table, p, args.rot_dim, u, false);
        turn_chunks(kx, ky, t, args.interleaved);
        if (has_q) {
#pragma unroll
          for (int h = 0; h < kGroup; ++h) turn_chunks(qx[h], qy[h], t, args.interleaved);
        }
      }
      uint4* kdst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.k_cache) + (cache_row0 + p) * kHeadDim);
      uint4* vdst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.v_cache) + (cache_row0 + p) * kHeadDim);
      kdst[lc.c0] = kx;
      kdst[lc.c1] = ky;
      vdst[u] = vx;
      vdst[u + 8] = vy;
      if (has_q) {
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
          uint4* qdst = reinterpret_cast<uint4*>(
              static_cast<__nv_bfloat16*>(args.q_out) +
              ((static_cast<size_t>(b) * args.Hkv * kGroup + g * kGroup + h) * args.L + i) * kHeadDim);
          qdst[lc.c0] = qx[h];
          qdst[lc.c1] = qy[h];
        }
      }
      widen(kx, mx[0], mn[0]);
      widen(ky, mx[1], mn[1]);
    }
  } else {
    for (int p = p0 + warp * kRowsPerWarp + r4; p < p1; p += n_warps * kRowsPerWarp) {
      const uint4* ksrc = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.k_cache) +
                                                         (cache_row0 + p) * kHeadDim);
      widen(ksrc[lc.c0], mx[0], mn[0]);
      widen(ksrc[lc.c1], mx[1], mn[1]);
    }
  }
  if (args.boxes == nullptr) return;

  // the block's maxima and minima: over the warp's four row groups, then
  // over the warps; thread t of the first 128 ends with channel t
#pragma unroll
  for (int m = 8; m <= 16; m <<= 1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t* a = reinterpret_cast<uint32_t*>(&mx[e]);
      uint32_t* z = reinterpret_cast<uint32_t*>(&mn[e]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        a[w] = bf16x2_max(a[w], __shfl_xor_sync(0xffffffffu, a[w], m));
        z[w] = bf16x2_min(z[w], __shfl_xor_sync(0xffffffffu, z[w], m));
      }
    }
  }
  if (lane < 8) {
    part[0][warp][lc.c0] = mx[0];
    part[0][warp][lc.c1] = mx[1];
    part[1][warp][lc.c0] = mn[0];
    part[1][warp][lc.c1] = mn[1];
  }
  __syncthreads();
  // warp w < 4 finishes channels 32w..32w+31 (in a CTA of fewer warps each
  // takes several)
  __nv_bfloat16* box = static_cast<__nv_bfloat16*>(args.boxes) +
                       (static_cast<size_t>(plane) * ((plane_rows + kTileKeys - 1) / kTileKeys) + row / kTileKeys) * 2 * kHeadDim;
  const bool merge = kAppend && block * kTileKeys < start;      // earlier keys of the block have a box already
  float hi[4], lo[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w % n_warps != warp) continue;
    const int ch = 32 * w + lane;
    const __nv_bfloat16* mxs = reinterpret_cast<const __nv_bfloat16*>(&part[0][0][0]) + ch;
    const __nv_bfloat16* mns = reinterpret_cast<const __nv_bfloat16*>(&part[1][0][0]) + ch;
    float a = __bfloat162float(mxs[0]), z = __bfloat162float(mns[0]);
    for (int i = 1; i < n_warps; ++i) {
      a = fmaxf(a, __bfloat162float(mxs[i * 128]));
      z = fminf(z, __bfloat162float(mns[i * 128]));
    }
    if (merge) {
      a = fmaxf(a, __bfloat162float(box[ch]));
      z = fminf(z, __bfloat162float(box[kHeadDim + ch]));
    }
    hi[w] = a;
    lo[w] = z;
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(a), fabsf(z))));
    if (lane == 0) amax_bits[w] = m;
  }
  __syncthreads();
  const float amax = __uint_as_float(max(max(amax_bits[0], amax_bits[1]), max(amax_bits[2], amax_bits[3])));
  const int E = grid_exponent(amax);
  const float up = exp2i(7 - E), step = exp2i(E - 7);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w % n_warps != warp) continue;
    const int ch = 32 * w + lane;
    const float a = fminf(fmaxf(ceilf(__fmul_rn(hi[w], up)), -127.0f), 127.0f);
    const float z = fminf(fmaxf(floorf(__fmul_rn(lo[w], up)), -127.0f), 127.0f);
    box[ch] = __float2bfloat16_rn(__fmul_rn(a, step));
    box[kHeadDim + ch] = __float2bfloat16_rn(__fmul_rn(z, step));
  }
}

cudaError_t launch_append(const AppendArgs& a, bool only_boxes, int sm_count, cudaStream_t s) {
  // blocks that L rows can touch at any start (one less when the start is
  // known to sit on a block's first key)
  const bool aligned = a.starts == nullptr && a.start % kTileKeys == 0;
  const long long touched = aligned ? (a.L + kTileKeys - 1) / kTileKeys : (a.L + kTileKeys - 2) / kTileKeys + 1;
  const long long grid = touched * a.B * a.Hkv;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const int rows = a.L < kTileKeys ? a.L : kTileKeys;
  // 8 warps let two CTAs share an SM, so that one loads while the other makes
  // its box (prompts of 4 x 4096: 44.6 us, with 16 warps 46.5, with 4 46.6);
  // where every CTA has an SM to itself, 16 load faster
  const int warps = std::min((rows + kRowsPerWarp - 1) / kRowsPerWarp, grid <= sm_count ? 16 : 8);
  if (only_boxes) kb_append_kernel<false><<<static_cast<unsigned>(grid), warps * 32, 0, s>>>(a);
  else kb_append_kernel<true><<<static_cast<unsigned>(grid), warps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kb

// kb_cache8.cu -- writing a KV cache held in 8 bits, and what it stands for.
//
// The rotation is that of kb_append.cu; keys are rounded from its fp32 result
// to their bytes at once.  The cache's format is described in kb_cache8.cuh.
#include <algorithm>

#include "kb_cache8.cuh"
#include "kb_contract.cuh"
#include "kb_launch.h"
#include "kb_turn.cuh"

namespace kb {

namespace {

constexpr int kPasses = 2;                      // rows of a thread: 16 warps x 4 rows x 2 = a block

// fp32 values of a lane's two chunks, turned where they are.
__device__ __forceinline__ void turned_values(const uint4& x, const uint4& y, const Turn& t, bool turns, bool interleaved,
                                              float (&fx)[8], float (&fy)[8]) {
  const uint32_t* a = reinterpret_cast<const uint32_t*>(&x);
  const uint32_t* b = reinterpret_cast<const uint32_t*>(&y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fx[2 * i] = lo_of(a[i]);
    fx[2 * i + 1] = hi_of(a[i]);
    fy[2 * i] = lo_of(b[i]);
    fy[2 * i + 1] = hi_of(b[i]);
  }
  if (!turns) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = fx[2 * i], a1 = fx[2 * i + 1], b0 = fy[2 * i], b1 = fy[2 * i + 1];
      fx[2 * i] = turn_a(a0, a1, t.cs[i]);
      fx[2 * i + 1] = turn_b(a0, a1, t.cs[i]);
      fy[2 * i] = turn_a(b0, b1, t.cs[4 + i]);
      fy[2 * i + 1] = turn_b(b0, b1, t.cs[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a0 = fx[i], b0 = fy[i];
      fx[i] = turn_a(a0, b0, t.cs[i]);
      fy[i] = turn_b(a0, b0, t.cs[i]);
    }
  }
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The largest magnitude of eight bf16 values, as fp32 bits (as whole numbers,
// so that infinities and NaN come out on top).
__device__ __forceinline__ uint32_t magnitude8(const uint4& v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
  return m;
}

__device__ __forceinline__ uint2 bytes_of(const float (&f)[8], int E) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = to_byte(__float_as_uint(f[i]), E);
  return make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24), b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
}

__device__ __forceinline__ uint2 bytes_of(const uint4& v, int E) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_of(w[i]);
    f[2 * i + 1] = hi_of(w[i]);
  }
  return bytes_of(f, E);
}

// Bring `n16` chunks of 16 bytes from exponent E - d to E (NaN bytes where E says so).
__device__ __forceinline__ void regrid(uint8_t* base, int n16, int d, int E) {
  for (int c = threadIdx.x; c < n16; c += blockDim.x) {
    uint4 v = reinterpret_cast<uint4*>(base)[c];
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r |= (E == kExpNaN ? kByteNaN : regrid_byte((w[i] >> (8 * k)) & 0xFFu, d)) << (8 * k);
      w[i] = r;
    }
    reinterpret_cast<uint4*>(base)[c] = v;
  }
}

}  // namespace

// ------------------------------------------------------------------ append

// Two CTAs per (batch, KV head, key block that the call's rows touch): one for
// the block's keys and values, one for its queries, which wait for nothing
// (in one CTA, L2 flushed: 4 ragged prompts 58.5 us, so 54.4; 16 tokens 11.4, so
// 9.3; 4 x 40 rows 15.5, so 11.4).  A block's
// exponent needs all of the block's new keys before the first byte is written,
// so a thread keeps its rows (at most two) in registers, turns its keys once for
// the largest magnitude and once more for the bytes.  That keeps to 64
// registers, so that two CTAs of 16 warps share an SM.  Where the exponent has
// grown, the block's earlier keys are brought to it: a CTA has the block to
// itself.
__global__ void __launch_bounds__(512, 2) kb_append8_kernel(const Append8Args args) {
  __shared__ uint32_t amax[2][16];
  // one decision for the CTA: the word may change while its threads read it
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(args.a.err) != 0)) return;
  const AppendArgs& a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  const int u = lane & 7, r4 = lane >> 3;
  const int units = static_cast<int>(gridDim.x) / (a.q != nullptr ? 2 : 1);
  const bool q_part = static_cast<int>(blockIdx.x) >= units;           // the block's queries; else its keys and values
  const int c = static_cast<int>(blockIdx.x) % units / (a.B * a.Hkv);  // which touched block
  const int bg = static_cast<int>(blockIdx.x) % units % (a.B * a.Hkv);
  const int b = bg / a.Hkv, g = bg % a.Hkv;

  int start = a.start, len = a.L;
  if (a.starts != nullptr) start = a.starts[b];
  if (a.lens != nullptr) len = a.lens[b];
  if (start < 0 || len < 0 || len > a.L || start > a.kv_cap - len || (a.table != nullptr && start > a.n_pos - len)) {
    if (threadIdx.x == 0 && c == 0) atomicCAS(a.err, 0u, static_cast<uint32_t>(kDevBadInput));
    return;
  }
  const int end = start + len;
  const int block = start / kTileKeys + c;
  if (len == 0 || block * kTileKeys >= end) return;
  const int p0 = max(start, block * kTileKeys), p1 = min(end, (block + 1) * kTileKeys);   // positions of this CTA
  long long plane;
  int row, plane_rows;                                                 // the block's place: first key at `row` of `plane`
  if (a.block_table != nullptr) {
    const int key = block * kTileKeys;
    const int pg = a.block_table[static_cast<size_t>(b) * a.pages_per_seq + key / a.page_size];
    if (pg < 0 || pg >= a.num_pages) {
      if (threadIdx.x == 0) atomicCAS(a.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return;
    }
    plane = static_cast<long long>(pg) * a.Hkv + g;
    row = key % a.page_size;
    plane_rows = a.page_size;
  } else {
    plane = static_cast<long long>(b) * a.Hkv + g;
    row = block * kTileKeys;
    plane_rows = a.kv_cap;
  }
  const size_t at = (static_cast<size_t>(plane) * plane_rows + row) * kHeadDim;           // the block's first byte
  const size_t e_at = static_cast<size_t>(plane) * ((plane_rows + kTileKeys - 1) / kTileKeys) + row / kTileKeys;
  uint8_t* kb = static_cast<uint8_t*>(a.k_cache) + at;
  uint8_t* vb = static_cast<uint8_t*>(a.v_cache) + at;
  const bool merge = block * kTileKeys < start;                        // earlier keys of the block have an exponent already
  const int k_old = merge ? held_exponent(args.k_exp[e_at]) : -128, v_old = merge ? held_exponent(args.v_exp[e_at]) : -128;

  const LaneChunks lc = lane_chunks(u, a.rot_dim, a.interleaved);
  const bool turns = a.table != nullptr && lc.turns;
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k) + b * a.ks[0] + g * a.ks[1];
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + b * a.vs[0] + g * a.vs[1];
  if (q_part) {
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + b * a.qs[0] + (g * kGroup) * a.qs[1];
#pragma unroll
    for (int it = 0; it < kPasses; ++it) {
      const int p = p0 + (it * n_warps + warp) * kRowsPerWarp + r4;
      if (p >= p1) continue;
      const long long i = p - start;
      Turn t;
      if (turns) load_turn(t, a.table, p, a.rot_dim, u, false);
#pragma unroll
      for (int h0 = 0; h0 < kGroup; h0 += 2) {
        uint4 qx[2], qy[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4* qsrc = reinterpret_cast<const uint4*>(qp + (h0 + h) * a.qs[1] + i * a.qs[2]);
          qx[h] = qsrc[lc.c0];
          qy[h] = qsrc[lc.c1];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (turns) turn_chunks(qx[h], qy[h], t, a.interleaved);
          uint4* qdst = reinterpret_cast<uint4*>(
              static_cast<__nv_bfloat16*>(a.q_out) +
              ((static_cast<size_t>(b) * a.Hkv * kGroup + g * kGroup + h0 + h) * a.L + i) * kHeadDim);
          qdst[lc.c0] = qx[h];
          qdst[lc.c1] = qy[h];
        }
      }
    }
    return;
  }
  uint4 kx[kPasses], ky[kPasses], vx[kPasses], vy[kPasses];
  uint32_t k_max = 0, v_max = 0;
#pragma unroll
  for (int it = 0; it < kPasses; ++it) {
    const int p = p0 + (it * n_warps + warp) * kRowsPerWarp + r4;
    if (p >= p1) continue;
    const long long i = p - start;                                     // row of the call's tensors
    const uint4* ksrc = reinterpret_cast<const uint4*>(kp + i * a.ks[2]);
    const uint4* vsrc = reinterpret_cast<const uint4*>(vp + i * a.vs[2]);
    kx[it] = ksrc[lc.c0];
    ky[it] = ksrc[lc.c1];
    vx[it] = vsrc[u];
    vy[it] = vsrc[u + 8];
    Turn t;
    if (turns) load_turn(t, a.table, p, a.rot_dim, u, false);
    float fx[8], fy[8];
    turned_values(kx[it], ky[it], t, turns, a.interleaved, fx, fy);
#pragma unroll
    for (int e = 0; e < 8; ++e) k_max = max(k_max, max(magnitude(fx[e]), magnitude(fy[e])));
    v_max = max(v_max, max(magnitude8(vx[it]), magnitude8(vy[it])));
  }
  k_max = __reduce_max_sync(0xffffffffu, k_max);
  v_max = __reduce_max_sync(0xffffffffu, v_max);
  if (lane == 0) {
    amax[0][warp] = k_max;
    amax[1][warp] = v_max;
  }
  __syncthreads();
  for (int w = 0; w < n_warps; ++w) {
    k_max = max(k_max, amax[0][w]);
    v_max = max(v_max, amax[1][w]);
  }
  const int k_e = max(block_exponent(k_max), k_old), v_e = max(block_exponent(v_max), v_old);
  if (merge) {
    const int n16 = (start - block * kTileKeys) * (kHeadDim / 16);
    if (k_e > k_old) regrid(kb, n16, k_e - k_old, k_e);
    if (v_e > v_old) regrid(vb, n16, v_e - v_old, v_e);
  }
  if (threadIdx.x == 0) {
    args.k_exp[e_at] = static_cast<int8_t>(k_e);
    args.v_exp[e_at] = static_cast<int8_t>(v_e);
  }
#pragma unroll
  for (int it = 0; it < kPasses; ++it) {
    const int p = p0 + (it * n_warps + warp) * kRowsPerWarp + r4;
    if (p >= p1) continue;
    const size_t r = static_cast<size_t>(p - block * kTileKeys) * kHeadDim;
    Turn t;
    if (turns) load_turn(t, a.table, p, a.rot_dim, u, false);
    float fx[8], fy[8];
    turned_values(kx[it], ky[it], t, turns, a.interleaved, fx, fy);
    *reinterpret_cast<uint2*>(kb + r + 8 * lc.c0) = bytes_of(fx, k_e);
    *reinterpret_cast<uint2*>(kb + r + 8 * lc.c1) = bytes_of(fy, k_e);
    *reinterpret_cast<uint2*>(vb + r + 8 * u) = bytes_of(vx[it], v_e);
    *reinterpret_cast<uint2*>(vb + r + 8 * (u + 8)) = bytes_of(vy[it], v_e);
  }
}

cudaError_t launch_append8(const Append8Args& args, cudaStream_t s) {
  const AppendArgs& a = args.a;
  // blocks that L rows can touch at any start (one less when the start is
  // known to sit on a block's first key)
  const bool aligned = a.starts == nullptr && a.start % kTileKeys == 0;
  const long long touched = aligned ? (a.L + kTileKeys - 1) / kTileKeys : (a.L + kTileKeys - 2) / kTileKeys + 1;
  const long long grid = touched * a.B * a.Hkv * (a.q != nullptr ? 2 : 1);
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const int rows = a.L < kTileKeys ? a.L : kTileKeys;
  const int warps = std::min((rows + kRowsPerWarp - 1) / kRowsPerWarp, 16);
  kb_append8_kernel<<<static_cast<unsigned>(grid), warps * 32, 0, s>>>(args);
  return cudaGetLastError();
}

// ------------------------------------------------------------ what it stands for

// n chunks of 8 bytes of one block into 16-byte chunks, by 256 threads: eight
// bytes per load, so that a warp's stores cover whole lines.
__device__ __forceinline__ void values_of_block(const uint2* src, uint4* dst, int n, const Scale8& s) {
  uint2 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = threadIdx.x + 256 * i;
    if (c < n) w[i] = __ldg(src + c);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = threadIdx.x + 256 * i;
    if (c < n) {
      const uint2 a = values8(w[i].x, s.first), b = values8(w[i].y, s.first);
      const uint4 v = make_uint4(a.x, a.y, b.x, b.y);
      dst[c] = s.two ? scaled_again(v, s.second) : v;
    }
  }
}

// A CTA per block of 128 rows: 128 bytes of a row become 256.
__global__ void __launch_bounds__(256) kb_cache_values_kernel(const Values8Args args) {
  if (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) return;
  const long long plane = blockIdx.x / args.blocks;
  const int block = static_cast<int>(blockIdx.x % args.blocks);
  const int rows = min(kTileKeys, args.rows - block * kTileKeys);
  const size_t row0 = static_cast<size_t>(plane) * args.rows + static_cast<size_t>(block) * kTileKeys;
  const Scale8 s = scale8(args.exps[blockIdx.x]);
  const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(args.cache) + row0 * kHeadDim);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.out) + row0 * kHeadDim);
  values_of_block(src, dst, rows * 16, s);
}

cudaError_t launch_cache_values(const Values8Args& a, cudaStream_t s) {
  kb_cache_values_kernel<<<static_cast<unsigned>(a.planes * a.blocks), 256, 0, s>>>(a);
  return cudaGetLastError();
}

// A CTA per (batch, KV head, key block) of a call's visible keys, K or V:
// what the block stands for, as rows of a contiguous bf16 cache of `rows`
// positions per sequence (rows behind the sequence's last key are left as they
// are: the tile kernel masks their scores and clears their values).
__global__ void __launch_bounds__(256) kb_cache_gather_kernel(const Gather8Args args) {
  if (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) return;
  const bool is_v = blockIdx.y != 0;
  const int block = static_cast<int>(blockIdx.x % args.blocks);
  const int bg = static_cast<int>(blockIdx.x / args.blocks);
  const int b = bg / args.Hkv, g = bg % args.Hkv;
  int end = args.rows;
  if (args.starts != nullptr) {
    const int start = args.starts[b], len = args.lens == nullptr ? args.L : args.lens[b];
    // a bad length is reported by the attention that follows
    if (start < 0 || len < 0 || len > args.L || start > args.rows - len) return;
    end = len == 0 ? 0 : start + len;
  }
  const int rows = min(kTileKeys, end - block * kTileKeys);
  if (rows <= 0) return;
  size_t row0 = (static_cast<size_t>(bg) * args.kv_cap + static_cast<size_t>(block) * kTileKeys);
  size_t e_at = static_cast<size_t>(bg) * ((args.kv_cap + kTileKeys - 1) / kTileKeys) + block;
  if (args.block_table != nullptr) {
    const int key = block * kTileKeys;
    const int pg = args.block_table[static_cast<size_t>(b) * args.pages_per_seq + key / args.page_size];
    if (pg < 0 || pg >= args.num_pages) {
      if (threadIdx.x == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return;
    }
    const size_t plane = static_cast<size_t>(pg) * args.Hkv + g;
    row0 = plane * args.page_size + key % args.page_size;
    e_at = plane * (args.page_size / kTileKeys) + key % args.page_size / kTileKeys;
  }
  const Scale8 s = scale8((is_v ? args.v_exp : args.k_exp)[e_at]);
  const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? args.v : args.k) + row0 * kHeadDim);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? args.v_out : args.k_out) +
                                        (static_cast<size_t>(bg) * args.rows + static_cast<size_t>(block) * kTileKeys) * kHeadDim);
  values_of_block(src, dst, rows * 16, s);
}

cudaError_t launch_cache_gather(const Gather8Args& a, cudaStream_t s) {
  kb_cache_gather_kernel<<<dim3(static_cast<unsigned>(a.B * a.Hkv * a.blocks), 2), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kb

// kb_select.cu -- which key blocks a query row attends to: the n blocks whose
// boxes allow the largest scores.
//
// The four query heads of a KV head choose together.  Their rows are summed
// as whole numbers, so that no order of summation can move a choice: with the
// grid exponent E of the four heads' largest magnitude,
//   t_h = rint(q_h 2^(15-E)),  u = t_0 + t_1 + t_2 + t_3,
// and with E' that of u, n = rint(u 2^(7-E')), within -127..127.  The score
// of a block with box (upper, lower) is
//   sum_d max(n_d upper_d, n_d lower_d) = sum_d (n_d^+ upper_d + n_d^- lower_d),
// n+ and n- the positive and negative parts: an upper bound of n . k over the
// keys in the box, and a product of two grid vectors, so it has one value
// however it is summed (kb_boxes.cuh).  Decode, chunk and prefill therefore
// choose the same blocks for the same row.
//
// A row at position p has the blocks 0 .. p/128.  The first `keep_first` and
// the last `keep_last` of them are always taken (the last is the row's own),
// the others by score, ties to the lowest block, until n are taken.  They go
// out in ascending order, -1 behind the last when there are fewer than n.
//
// The n largest keys are found without sorting: scores become unsigned whole
// numbers of the same order, and the n-th largest is built bit by bit from
// the counts of the keys at or above a trial value.
#include "kb_boxes.cuh"
#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

constexpr uint32_t kKeyForced = 0xFFFFFFFFu;    // above every score
constexpr int kChunkKeys = 1024;                // keys a warp searches at once: 32 registers per lane

// Scores (finite) as unsigned keys of the same order; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float s) {
  const uint32_t b = __float_as_uint(__fadd_rn(s, 0.0f));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The warp's n largest of m <= 1024 keys, in place order (ties: the first
// ones), handed to emit(place among the chosen, place among the keys).
// Returns how many there are (min(n, m)).
template <class Emit>
__device__ __forceinline__ int warp_largest(const uint32_t* keys, int m, int n, int lane, Emit emit) {
  uint32_t r[kChunkKeys / 32];
#pragma unroll
  for (int i = 0; i < kChunkKeys / 32; ++i) {
    if (i * 32 >= m) break;
    r[i] = i * 32 + lane < m ? keys[i * 32 + lane] : 0u;
  }
  uint32_t T = 0;
  int ties = 0;                                   // keys equal to T that are taken; < 0: all
  if (m > n) {
    bool exact = false;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = T | (1u << bit);
      int c = 0;
#pragma unroll
      for (int i = 0; i < kChunkKeys / 32; ++i) {
        if (i * 32 >= m) break;
        c += r[i] >= trial ? 1 : 0;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= n) T = trial;
      if (c == n) { exact = true; break; }
    }
    if (exact) {
      ties = -1;
    } else {
      int above = 0;
#pragma unroll
      for (int i = 0; i < kChunkKeys / 32; ++i) {
        if (i * 32 >= m) break;
        above += r[i] > T ? 1 : 0;
      }
      ties = n - __reduce_add_sync(0xffffffffu, above);
    }
  } else {
    ties = -1;
  }
  int taken = 0, tied = 0;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < kChunkKeys / 32; ++i) {
    if (i * 32 >= m) break;
    const bool in = i * 32 + lane < m;
    bool take = in && r[i] >= T;
    if (ties >= 0) {
      const bool eq = in && r[i] == T;
      const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
      if (eq) take = tied + __popc(eqs & below) < ties;
      tied += __popc(eqs);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, take);
    if (take) emit(taken + __popc(mask & below), i * 32 + lane);
    taken += __popc(mask);
  }
  return taken;
}

// Position of row i of sequence b, or -1 when the row does not exist; a bad
// start or length is recorded.
__device__ __forceinline__ int row_position(const SelectArgs& a, int b, int i) {
  int start = a.start, len = a.L;
  if (a.starts != nullptr) {
    start = a.starts[b];
    if (a.lens != nullptr) len = a.lens[b];
    if (start < 0 || len < 0 || len > a.L || start > a.kv_cap - len) {
      if (threadIdx.x == 0) atomicCAS(a.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return -1;
    }
  }
  return i < len ? start + i : -1;
}

// Box of block j of sequence b, KV head g, or null for a page out of range.
__device__ __forceinline__ const __nv_bfloat16* box_of(const SelectArgs& a, int b, int g, int j) {
  const __nv_bfloat16* boxes = static_cast<const __nv_bfloat16*>(a.boxes);
  if (a.block_table == nullptr)
    return boxes + ((static_cast<size_t>(b) * a.Hkv + g) * a.blocks_per_plane + j) * 2 * kHeadDim;
  const int pg = a.block_table[static_cast<size_t>(b) * a.pages_per_seq + j / a.blocks_per_plane];
  if (pg < 0 || pg >= a.num_pages) {
    atomicCAS(a.err, 0u, static_cast<uint32_t>(kDevBadInput));
    return nullptr;
  }
  return boxes + ((static_cast<size_t>(pg) * a.Hkv + g) * a.blocks_per_plane + j % a.blocks_per_plane) * 2 * kHeadDim;
}

__device__ __forceinline__ bool always_taken(const SelectArgs& a, int j, int nb) {
  return j < a.keep_first || j >= nb - a.keep_last;
}

}  // namespace

// ----------------------------------------------------------- a row per CTA
//
// One CTA of 16 warps per (row, batch, KV head); 16 lanes score a block (eight
// channels of both bounds each), so a warp has two blocks of 512 bytes in
// flight per step.
constexpr int kSelectRowThreads = 512;

__global__ void __launch_bounds__(kSelectRowThreads, 1) kb_select_row_kernel(const SelectArgs args) {
  extern __shared__ uint32_t sel_smem[];
  __shared__ float whole[kHeadDim];               // n
  __shared__ uint32_t amax_bits[8];
  if (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = blockIdx.x;
  const int g = static_cast<int>(item % args.Hkv);
  const int b = static_cast<int>(item / args.Hkv % args.B);
  const int i = static_cast<int>(item / (static_cast<long long>(args.Hkv) * args.B));
  const int pos = row_position(args, b, i);
  if (pos < 0) return;
  const int nb = pos / kTileKeys + 1;
  int* out = args.blocks + ((static_cast<size_t>(b) * args.Hkv + g) * args.L + i) * args.n;
  if (nb <= args.n) {
    for (int t = threadIdx.x; t < args.n; t += kSelectRowThreads) out[t] = t < nb ? t : -1;
    return;
  }
  // the whole-number query: thread d < 128 holds channel d
  float q[kGroup];
  if (warp < 4) {
    float m = 0.0f;
#pragma unroll
    for (int h = 0; h < kGroup; ++h) {
      q[h] = __bfloat162float(static_cast<const __nv_bfloat16*>(
          args.q)[((static_cast<size_t>(b) * args.Hkv + g) * kGroup + h) * args.L * kHeadDim +
                  static_cast<size_t>(i) * kHeadDim + threadIdx.x]);
      m = fmaxf(m, fabsf(q[h]));
    }
    const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if (lane == 0) amax_bits[warp] = mb;
  }
  __syncthreads();
  float u = 0.0f;
  if (warp < 4) {
    const uint32_t mb = max(max(amax_bits[0], amax_bits[1]), max(amax_bits[2], amax_bits[3]));
    u = whole_sum(q, exp2i(15 - grid_exponent(__uint_as_float(mb))));
    const uint32_t ub = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(u)));
    if (lane == 0) amax_bits[4 + warp] = ub;
  }
  __syncthreads();
  if (warp < 4) {
    const uint32_t ub = max(max(amax_bits[4], amax_bits[5]), max(amax_bits[6], amax_bits[7]));
    whole[threadIdx.x] = rintf(__fmul_rn(u, exp2i(7 - grid_exponent(__uint_as_float(ub)))));
  }
  __syncthreads();
  // scores
  const int c = lane & 15;
  float np[8], nm[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float w = whole[8 * c + e];
    np[e] = fmaxf(w, 0.0f);
    nm[e] = fminf(w, 0.0f);
  }
  for (int j0 = warp * 2; j0 < nb; j0 += kSelectRowThreads / 16) {
    const int j = j0 + (lane >> 4);
    float s = 0.0f;
    const bool scored = j < nb && !always_taken(args, j, nb);
    if (scored) {
      const __nv_bfloat16* box = box_of(args, b, g, j);
      if (box != nullptr) {
        const uint4 hi = __ldg(reinterpret_cast<const uint4*>(box) + c);
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(box + kHeadDim) + c);
        s = box_dot(hi, lo, np, nm);
      }
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, m));
    if (c == 0 && j < nb) sel_smem[j] = scored ? order_key(s) : kKeyForced;
  }
  __syncthreads();
  // rounds: every warp reduces chunks of 1024 keys to their n largest, until
  // one chunk is left.  Round 0 reads the keys in block order, later rounds
  // (key, block) pairs in the same order.
  int m = nb;
  uint32_t* keys = sel_smem;
  int* ids = nullptr;
  const int half = (args.max_blocks + kChunkKeys - 1) / kChunkKeys * args.n;     // pairs a round can leave
  int which = 0;
  while (m > kChunkKeys) {
    uint32_t* nk = sel_smem + args.max_blocks + which * 2 * half;
    int* ni = reinterpret_cast<int*>(nk + half);
    const int chunks = (m + kChunkKeys - 1) / kChunkKeys;
    for (int k = warp; k < chunks; k += kSelectRowThreads / 32) {
      const int from = k * kChunkKeys, mk = min(kChunkKeys, m - from);
      warp_largest(keys + from, mk, args.n, lane, [&](int to, int at) {
        nk[k * args.n + to] = keys[from + at];
        ni[k * args.n + to] = ids == nullptr ? from + at : ids[from + at];
      });
    }
    const int last = m - (chunks - 1) * kChunkKeys;
    m = (chunks - 1) * args.n + min(args.n, last);
    keys = nk;
    ids = ni;
    which ^= 1;
    __syncthreads();
  }
  if (warp == 0) {
    warp_largest(keys, m, args.n, lane, [&](int to, int at) { out[to] = ids == nullptr ? at : ids[at]; });
  }
}

cudaError_t launch_select(const SelectArgs& a, int device, cudaStream_t s) {
  static bool configured[64] = {};
  if (!configured[device]) {
    const cudaError_t e = cudaFuncSetAttribute(kb_select_row_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  const int rounds = (a.max_blocks + kChunkKeys - 1) / kChunkKeys;
  const size_t smem = (static_cast<size_t>(a.max_blocks) + (a.max_blocks > kChunkKeys ? 4u * rounds * a.n : 0u)) * 4u;
  const long long rows = static_cast<long long>(a.B) * a.Hkv * a.L;
  if (rows > 0x7FFFFFFFLL || smem > 200u * 1024u) return cudaErrorInvalidValue;
  kb_select_row_kernel<<<static_cast<unsigned>(rows), kSelectRowThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kb

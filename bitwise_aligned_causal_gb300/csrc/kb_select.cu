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
// The n largest scores are found without sorting: a trial value halves the
// range between the smallest and the largest score until exactly n scores are
// at or above it; only ties keep the search going until the range is a single
// value, of which the first blocks are then taken.
#include "kb_boxes.cuh"
#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

constexpr int kChunkKeys = 1024;                // scores a warp searches at once: 32 registers per lane

// Scores (finite) as unsigned keys of the same order; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float s) {
  const uint32_t b = __float_as_uint(__fadd_rn(s, 0.0f));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k); }

// Search for the value that exactly `need` scores are at or above: the range
// [lo, hi) of keys with count(>= lo) >= need > count(>= hi).
struct CutSearch {
  uint32_t lo, hi;
  bool exact;                                   // exactly `need` scores are at or above lo's value
  __device__ __forceinline__ bool done() const { return exact || hi - lo <= 1u; }
  // The next key to try: the middle of the values, and after 40 halvings that
  // of their bit patterns (32 more end any search).
  __device__ __forceinline__ uint32_t trial(int iter) const {
    const float a = key_value(lo), b = key_value(hi);
    const uint32_t mid = order_key(__fmaf_rn(0.5f, __fsub_rn(b, a), a));
    return iter < 40 && mid > lo && mid < hi ? mid : lo + ((hi - lo) >> 1);
  }
  __device__ __forceinline__ void counted(uint32_t key, int count, int need) {
    if (count >= need) lo = key;
    else hi = key;
    exact = count == need;
  }
  __device__ __forceinline__ float cut() const { return key_value(lo); }
};
constexpr int kMaxTrials = 80;

// The warp's n largest of m <= 1024 scores, in place order (ties: the first
// ones), handed to emit(place among the chosen, place among the scores).
template <class Emit>
__device__ __forceinline__ void warp_largest(const float* scores, int m, int n, int lane, Emit emit) {
  float r[kChunkKeys / 32];
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < kChunkKeys / 32; ++i) {
    if (i * 32 >= m) break;
    const bool in = i * 32 + lane < m;
    r[i] = in ? scores[i * 32 + lane] : -INFINITY;          // below every trial
    hi = fmaxf(hi, r[i]);
    lo = fminf(lo, in ? r[i] : INFINITY);
  }
  CutSearch c{__reduce_min_sync(0xffffffffu, order_key(lo)), __reduce_max_sync(0xffffffffu, order_key(hi)) + 1u, m <= n};
  for (int iter = 0; iter < kMaxTrials && !c.done(); ++iter) {
    const uint32_t key = c.trial(iter);
    const float t = key_value(key);
    int count = 0;
#pragma unroll
    for (int i = 0; i < kChunkKeys / 32; ++i) {
      if (i * 32 >= m) break;
      count += r[i] >= t ? 1 : 0;
    }
    c.counted(key, __reduce_add_sync(0xffffffffu, count), n);
  }
  const float cut = c.cut();
  int ties = 0;                                             // scores equal to the cut that are taken
  if (!c.exact) {
    int above = 0;
#pragma unroll
    for (int i = 0; i < kChunkKeys / 32; ++i) {
      if (i * 32 >= m) break;
      above += r[i] > cut ? 1 : 0;
    }
    ties = n - __reduce_add_sync(0xffffffffu, above);
  }
  int taken = 0, tied = 0;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < kChunkKeys / 32; ++i) {
    if (i * 32 >= m) break;
    bool take = i * 32 + lane < m && r[i] >= cut;
    if (!c.exact) {
      const bool eq = take && r[i] == cut;
      const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
      if (eq) take = tied + __popc(eqs & below) < ties;
      tied += __popc(eqs);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, take);
    if (take) emit(taken + __popc(mask & below), i * 32 + lane);
    taken += __popc(mask);
  }
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

}  // namespace

// ----------------------------------------------------------- a row per CTA
//
// One CTA of 16 warps per (row, batch, KV head); 16 lanes score a block (eight
// channels of both bounds each), so a warp has eight blocks of 512 bytes in
// flight, the first of them while the query is still on its way to whole
// numbers.  For one token the boxes are read once and nothing else counts.
constexpr int kSelectRowThreads = 512;
constexpr int kSelectRowMax = 16;               // query rows per sequence up to which this kernel runs

__global__ void __launch_bounds__(kSelectRowThreads, 1) kb_select_row_kernel(const SelectArgs args) {
  extern __shared__ float sel_smem[];
  __shared__ float whole[kHeadDim];               // n
  __shared__ uint32_t amax_bits[8];
  const bool failed = *reinterpret_cast<volatile uint32_t*>(args.err) != 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = blockIdx.x;
  const int g = static_cast<int>(item % args.Hkv);
  const int b = static_cast<int>(item / args.Hkv % args.B);
  const int i = static_cast<int>(item / (static_cast<long long>(args.Hkv) * args.B));
  const int pos = row_position(args, b, i);
  const int nb = pos < 0 ? 0 : pos / kTileKeys + 1;
  const int c0 = args.keep_first, m = nb - args.keep_first - args.keep_last;   // blocks c0 .. c0+m-1 are chosen by score
  const int need = args.n - args.keep_first - args.keep_last;
  // the first boxes and the query leave together
  constexpr int kAtOnce = 4, kStep = kSelectRowThreads / 16;
  const int c = lane & 15;
  uint4 hi[kAtOnce], lo[kAtOnce];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a) {
      const int j = j0 + a * kStep;
      const __nv_bfloat16* box = j < m ? box_of(args, b, g, c0 + j) : nullptr;
      hi[a] = lo[a] = make_uint4(0u, 0u, 0u, 0u);
      if (box != nullptr) {
        hi[a] = __ldg(reinterpret_cast<const uint4*>(box) + c);
        lo[a] = __ldg(reinterpret_cast<const uint4*>(box + kHeadDim) + c);
      }
    }
  };
  const int j_first = warp * 2 + (lane >> 4);
  const bool scored = nb > args.n && need > 0;
  float q[kGroup];
  if (scored) {
    fetch(j_first);
    if (warp < 4) {
      float mx = 0.0f;
#pragma unroll
      for (int h = 0; h < kGroup; ++h) {
        q[h] = __bfloat162float(static_cast<const __nv_bfloat16*>(
            args.q)[((static_cast<size_t>(b) * args.Hkv + g) * kGroup + h) * args.L * kHeadDim +
                    static_cast<size_t>(i) * kHeadDim + threadIdx.x]);
        mx = fmaxf(mx, fabsf(q[h]));
      }
      const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
      if (lane == 0) amax_bits[warp] = mb;
    }
  }
  // one decision for the CTA: the word may change while its threads read it
  if (__syncthreads_or(failed) || pos < 0) return;
  int* out = args.blocks + ((static_cast<size_t>(b) * args.Hkv + g) * args.L + i) * args.n;
  if (!scored) {
    if (nb > args.n)                              // nothing is scored, but a bad page is still found
      for (int j = threadIdx.x; j < m; j += kSelectRowThreads) (void)box_of(args, b, g, c0 + j);
    for (int t = threadIdx.x; t < args.n; t += kSelectRowThreads)
      out[t] = nb <= args.n ? (t < nb ? t : -1) : t < args.keep_first ? t : nb - args.n + t;
    return;
  }
  // the whole-number query: thread d < 128 holds channel d
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
    whole[threadIdx.x] = rint_small(__fmul_rn(u, exp2i(7 - grid_exponent(__uint_as_float(ub)))));
  }
  __syncthreads();
  float np[8], nm[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float w = whole[8 * c + e];
    np[e] = fmaxf(w, 0.0f);
    nm[e] = fminf(w, 0.0f);
  }
  for (int j0 = j_first; j0 < m + (lane >> 4); j0 += kStep * kAtOnce) {        // uniform over the warp
    float s[kAtOnce];
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a) s[a] = box_dot(hi[a], lo[a], np, nm);
    if (j0 + kStep * kAtOnce < m + (lane >> 4)) fetch(j0 + kStep * kAtOnce);
#pragma unroll
    for (int k = 8; k >= 1; k >>= 1)
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) s[a] = __fadd_rn(s[a], __shfl_xor_sync(0xffffffffu, s[a], k));
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a)
      if (c == 0 && j0 + a * kStep < m) sel_smem[j0 + a * kStep] = s[a];
  }
  __syncthreads();
  // rounds: every warp reduces chunks of 1024 scores to their `need` largest,
  // until one chunk is left.  Round 0 reads the scores in block order, later
  // rounds (score, block) pairs in the same order.
  int left = m;
  float* scores = sel_smem;
  int* ids = nullptr;
  const int half = (args.max_blocks + kChunkKeys - 1) / kChunkKeys * args.n;     // pairs a round can leave
  int which = 0;
  while (left > kChunkKeys) {
    float* nk = sel_smem + args.max_blocks + which * 2 * half;
    int* ni = reinterpret_cast<int*>(nk + half);
    const int chunks = (left + kChunkKeys - 1) / kChunkKeys;
    for (int k = warp; k < chunks; k += kSelectRowThreads / 32) {
      const int from = k * kChunkKeys;
      warp_largest(scores + from, min(kChunkKeys, left - from), need, lane, [&](int to, int at) {
        nk[k * need + to] = scores[from + at];
        ni[k * need + to] = ids == nullptr ? from + at : ids[from + at];
      });
    }
    left = (chunks - 1) * need + min(need, left - (chunks - 1) * kChunkKeys);
    scores = nk;
    ids = ni;
    which ^= 1;
    __syncthreads();
  }
  if (warp == 0) {
    warp_largest(scores, left, need, lane, [&](int to, int at) { out[c0 + to] = c0 + (ids == nullptr ? at : ids[at]); });
  } else if (warp == 1) {
    for (int t = lane; t < args.keep_first + args.keep_last; t += 32)
      if (t < args.keep_first) out[t] = t;
      else out[args.n - args.keep_last + t - args.keep_first] = nb - args.keep_last + t - args.keep_first;
  }
}

// ------------------------------------------------------ 128 rows per CTA
//
// One CTA per (batch, KV head, 128 positions from a multiple of 128 on), so
// its rows share their blocks 0 .. t.  Scores are one product of grid vectors,
// [n+ | n-] (128 rows x 256) times [upper | lower] (blocks x 256), on the
// tensor core, exact like every other order of summation.  They stay in TMEM
// (a row per lane, a block per column).  Two threads search a row, each over
// half of its blocks, the first 64 of which it keeps in registers; they add
// their counts through shared memory.  Rows whose blocks exceed TMEM go on in
// passes of 256 blocks, the winners of the earlier ones carried along in
// shared memory.
// Bound: q is read once (1 KB a row and KV head); 96 KB of shared memory and
// half of TMEM let two CTAs share an SM, so one loads while the other
// searches.
struct SelectTileCfg {
  static constexpr int kThreads = 256;
  static constexpr int kChunk = 64;                         // blocks per MMA
  static constexpr int kPass = 256;                         // blocks in TMEM at a time
  static constexpr uint32_t kTmemCols = 256;
  static constexpr uint32_t kASlab = 128 * 128;             // 64 of the 256 columns of n, 128 rows
  static constexpr uint32_t kBSlab = kChunk * 128;
  static constexpr uint32_t kAOff = 0;
  static constexpr uint32_t kBOff = 4 * kASlab;
  static constexpr uint32_t kBarOff = kBOff + 4 * kBSlab;
  static constexpr uint32_t kMiscOff = kBarOff + 16;
  static constexpr uint32_t kCountOff = kMiscOff + 16;      // [parity][half][row] counts
  static constexpr uint32_t kListOff = kCountOff + 2 * 2 * 128 * 4;   // several passes: score and block per winner and row
  static constexpr int kMaxListed = 32;
};

__global__ void __launch_bounds__(SelectTileCfg::kThreads, 2) kb_select_tile_kernel(const SelectArgs args, int n_tiles) {
  using Cfg = SelectTileCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  const uint32_t bar = sbase + Cfg::kBarOff;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // one decision for the CTA: the word may change while its threads read it
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(args.err) != 0)) return;
  const int bg = static_cast<int>(blockIdx.x) / n_tiles;
  const int b = bg / args.Hkv, g = bg % args.Hkv;
  int start = args.start, len = args.L;
  if (args.starts != nullptr) {
    start = args.starts[b];
    if (args.lens != nullptr) len = args.lens[b];
    if (start < 0 || len < 0 || len > args.L || start > args.kv_cap - len) {
      if (threadIdx.x == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return;
    }
  }
  const int t = start / kTileKeys + n_tiles - 1 - static_cast<int>(blockIdx.x) % n_tiles;   // last positions first
  const int i0 = t * kTileKeys - start;                     // row index of the tile's first position (may be negative)
  if (len == 0 || i0 >= len) return;
  const int nb = t + 1;
  const size_t out_row0 = (static_cast<size_t>(b) * args.Hkv + g) * args.L;
  const int cand0 = args.keep_first, cand1 = nb - args.keep_last;      // blocks that are chosen by score
  const int need = args.n - args.keep_first - args.keep_last;
  if (nb <= args.n || need == 0) {
    if (nb > args.n)                                        // nothing is scored, but a bad page is still found
      for (int j = cand0 + threadIdx.x; j < cand1; j += Cfg::kThreads) (void)box_of(args, b, g, j);
    for (int e = threadIdx.x; e < kTileKeys * args.n; e += Cfg::kThreads) {
      const int i = i0 + e / args.n, k = e % args.n;
      if (i >= 0 && i < len)
        args.blocks[(out_row0 + i) * args.n + k] = nb <= args.n ? (k < nb ? k : -1) : k < args.keep_first ? k : nb - args.n + k;
    }
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    misc[1] = 0u;
    fence_mbar_init();
  }
  // by a warp that has not just branched on one thread: the allocation is one
  // instruction of a whole, converged warp
  if (warp == 4) {
    __syncwarp();
    tmem_alloc(sbase + Cfg::kMiscOff, Cfg::kTmemCols);
    tmem_relinquish();
  }
  // boxes of the 64 blocks from j0 on into the B operand (a box is a row of it)
  auto load_boxes = [&](int j0, int j1) {
    uint4 val[Cfg::kChunk * 32 / Cfg::kThreads];
#pragma unroll
    for (int k = 0; k < Cfg::kChunk * 32 / Cfg::kThreads; ++k) {
      const int e = threadIdx.x + k * Cfg::kThreads, j = j0 + (e >> 5);
      const __nv_bfloat16* box = j < j1 ? box_of(args, b, g, j) : nullptr;
      val[k] = box != nullptr ? __ldg(reinterpret_cast<const uint4*>(box) + (e & 31)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < Cfg::kChunk * 32 / Cfg::kThreads; ++k) {
      const int e = threadIdx.x + k * Cfg::kThreads, r = e >> 5, c = e & 31;
      *reinterpret_cast<uint4*>(smem + Cfg::kBOff + (c >> 3) * Cfg::kBSlab + (r >> 3) * 1024 + (r & 7) * 128 +
                                (((c & 7) ^ (r & 7)) << 4)) = val[k];
    }
  };
  load_boxes(0, min(cand1, Cfg::kPass));

  // n of the tile's rows: 16 lanes per row, eight channels of the four heads
  // each, written as the two halves n+ and n- of the A operand
  {
    const int c = lane & 15;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.q) +
                                                    (static_cast<size_t>(b) * args.Hkv + g) * kGroup * args.L * kHeadDim);
    const size_t head_step = static_cast<size_t>(args.L) * (kHeadDim / 8);
    constexpr int kAtOnce = 2;                              // rows in flight per lane
#pragma unroll 1
    for (int m0 = 2 * warp + (lane >> 4); m0 < kTileKeys; m0 += 16 * kAtOnce) {
      uint4 x[kAtOnce][kGroup];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int i = i0 + m0 + 16 * a;
#pragma unroll
        for (int h = 0; h < kGroup; ++h)
          x[a][h] = i >= 0 && i < len ? __ldg(q + h * head_step + static_cast<size_t>(i) * (kHeadDim / 8) + c)
                                      : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        float amax = 0.0f;
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
          const uint32_t w[4] = {x[a][h].x, x[a][h].y, x[a][h].z, x[a][h].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const float scale = exp2i(15 - grid_exponent(amax));
        float u[8], umax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v[kGroup];
#pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            const uint32_t w = e < 2 ? x[a][h].x : e < 4 ? x[a][h].y : e < 6 ? x[a][h].z : x[a][h].w;
            v[h] = __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
          }
          u[e] = whole_sum(v, scale);
          umax = fmaxf(umax, fabsf(u[e]));
        }
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) umax = fmaxf(umax, __shfl_xor_sync(0xffffffffu, umax, m));
        const float fit = exp2i(7 - grid_exponent(umax));
        uint32_t np[4], nm[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w0 = rint_small(__fmul_rn(u[2 * e], fit)), w1 = rint_small(__fmul_rn(u[2 * e + 1], fit));
          np[e] = pack_bf16x2(fmaxf(w0, 0.0f), fmaxf(w1, 0.0f));
          nm[e] = pack_bf16x2(fminf(w0, 0.0f), fminf(w1, 0.0f));
        }
        const int m = m0 + 16 * a;
        uint8_t* at = smem + Cfg::kAOff + (c >> 3) * Cfg::kASlab + (m >> 3) * 1024 + (m & 7) * 128 + (((c & 7) ^ (m & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = make_uint4(np[0], np[1], np[2], np[3]);
        *reinterpret_cast<uint4*>(at + 2 * Cfg::kASlab) = make_uint4(nm[0], nm[1], nm[2], nm[3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];

  const int passes = (cand1 + Cfg::kPass - 1) / Cfg::kPass;
  const int row = 32 * (warp & 3) + lane, side = warp >> 2;            // the thread's row, and which half of its blocks
  int* counts = reinterpret_cast<int*>(smem + Cfg::kCountOff);
  int turn = 0;
  // both sides' values of the row, side 0's in .x
  auto exchange = [&](int mine) {
    counts[(turn * 2 + side) * 128 + row] = mine;
    __syncwarp();
    named_bar_sync(1u + (warp & 3), 64u);
    const int2 v = make_int2(counts[turn * 2 * 128 + row], counts[(turn * 2 + 1) * 128 + row]);
    turn ^= 1;                                                           // the other buffer next: one barrier is enough
    return v;
  };
  float* list_s = reinterpret_cast<float*>(smem + Cfg::kListOff);        // [winner][row]
  int* list_j = reinterpret_cast<int*>(smem + Cfg::kListOff) + Cfg::kMaxListed * 128;
  int* staged = reinterpret_cast<int*>(smem + Cfg::kAOff);             // [row][n + 1], once A is no longer read
  int listed = 0;                                                      // winners carried from earlier passes (every row's)
  uint32_t phase = 0;
  bool ok = true;
  for (int pass = 0; pass < passes; ++pass) {
    const int c0 = pass * Cfg::kPass, c1 = min(cand1, c0 + Cfg::kPass);
    for (int j0 = c0; j0 < c1; j0 += Cfg::kChunk) {
      if (j0 > 0) load_boxes(j0, c1);
      fence_proxy_async_smem();
      __syncthreads();
      if (threadIdx.x == 7 * 32) {
        tc_fence_after();
        constexpr uint32_t kIdesc = idesc_bf16_f32(128, Cfg::kChunk, 0);
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
          mma_ss(tmem_base + static_cast<uint32_t>(j0 - c0), desc_kmajor(sbase + Cfg::kAOff, kk, 1024u, Cfg::kASlab),
                 desc_kmajor(sbase + Cfg::kBOff, kk, 1024u, Cfg::kBSlab), kIdesc, kk > 0 ? 1u : 0u);
        tc_commit(bar);
      }
      ok = mbar_wait(bar, phase, abort_flag, args.err, kDevTimeoutMma);   // the scores are there, B may be replaced
      phase ^= 1u;
      ok = __syncthreads_and(ok);
      if (!ok) break;
    }
    if (!ok) break;
    tc_fence_after();
    {
      // side 0 has the winners of earlier passes and columns skip .. mid-1 of
      // this one, side 1 columns mid .. cols-1
      const uint32_t s_tmem = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
      const int cols = c1 - c0, skip = max(0, cand0 - c0);
      const int mid = min(cols, (cols / 2 + 31) & ~31);
      const int k0 = side ? mid : 0, k1 = side ? cols : mid;
      const int carried = side ? 0 : listed;
      auto load32 = [&](int k, uint32_t (&x)[32]) {
        __syncwarp();                                                     // TMEM is read by the whole warp together
        tmem_ld32_wait(s_tmem + static_cast<uint32_t>(k), x);
        if (k < skip || k + 32 > k1) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (k + e < skip || k + e >= k1) x[e] = 0xFF800000u;          // -inf: below every trial
        }
      };
      uint32_t x0[32], x1[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) x0[e] = x1[e] = 0xFF800000u;
      if (k0 < k1) load32(k0, x0);
      if (k0 + 32 < k1) load32(k0 + 32, x1);
      // fn(column of x[0], x) over the side's columns; the whole warp together
      auto each32 = [&](auto fn) {
        fn(k0, x0);
        if (k0 + 32 < k1) fn(k0 + 32, x1);
        for (int k = k0 + 64; k < k1; k += 32) {
          uint32_t x[32];
          load32(k, x);
          fn(k, x);
        }
      };
      float hi = -INFINITY, lo = INFINITY;
      each32([&](int, const uint32_t (&x)[32]) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float v = __uint_as_float(x[e]);
          hi = fmaxf(hi, v);
          lo = fminf(lo, v == -INFINITY ? INFINITY : v);
        }
      });
      for (int w = 0; w < carried; ++w) {
        const float v = list_s[w * 128 + row];
        hi = fmaxf(hi, v);
        lo = fminf(lo, v);
      }
      const int2 his = exchange(__float_as_int(hi)), los = exchange(__float_as_int(lo));
      hi = fmaxf(__int_as_float(his.x), __int_as_float(his.y));
      lo = fminf(__int_as_float(los.x), __int_as_float(los.y));
      // the pass's winners: all of them when there are at most `need`, else
      // those above the cut; ties at the cut from the lowest block on
      const int have = cols - min(cols, skip) + listed;
      CutSearch c{order_key(lo), order_key(hi) + 1u, have <= need};
      for (int iter = 0; iter < kMaxTrials; ++iter) {
        const bool done = c.done();
        if (__all_sync(0xffffffffu, done)) break;                         // the same on both sides: they hold the same rows
        const uint32_t key = c.trial(iter);
        const float trial = key_value(key);
        int count = 0;
        each32([&](int, const uint32_t (&x)[32]) {
#pragma unroll
          for (int e = 0; e < 32; ++e) count += __uint_as_float(x[e]) >= trial ? 1 : 0;
        });
        for (int w = 0; w < carried; ++w) count += list_s[w * 128 + row] >= trial ? 1 : 0;
        const int2 both = exchange(count);
        if (!done) c.counted(key, both.x + both.y, need);
      }
      const float cut = c.cut();
      // counts of the scores above the cut and at it, and of side 0's share
      int above = 0, equal = 0;
      each32([&](int, const uint32_t (&x)[32]) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          above += __uint_as_float(x[e]) > cut ? 1 : 0;
          equal += __uint_as_float(x[e]) == cut ? 1 : 0;
        }
      });
      for (int w = 0; w < carried; ++w) {
        above += list_s[w * 128 + row] > cut ? 1 : 0;
        equal += list_s[w * 128 + row] == cut ? 1 : 0;
      }
      const int2 aboves = exchange(above), equals = exchange(equal);
      const int ties_all = c.exact ? equals.x + equals.y : need - aboves.x - aboves.y;
      const int ties0 = min(ties_all, equals.x);
      int ties = side ? ties_all - ties0 : ties0;
      int at = side ? aboves.x + ties0 : 0;                               // place of the side's first winner
      const bool last = pass == passes - 1;
      int* const mine = staged + row * (args.n + 1) + args.keep_first;
      auto take = [&](float v, int j) {
        if (v == cut && ties-- <= 0) return;
        if (last) {
          mine[at] = j;
        } else {
          list_s[at * 128 + row] = v;
          list_j[at * 128 + row] = j;
        }
        ++at;
      };
      // carried winners first (side 0 moves them down in place), then the
      // columns: their winners as a mask, so only those cost a store
      for (int w = 0; w < carried; ++w) {
        const float v = list_s[w * 128 + row];
        if (v >= cut) take(v, list_j[w * 128 + row]);
      }
      __syncwarp();
      if (!last) named_bar_sync(1u + (warp & 3), 64u);                    // side 1 writes behind them
      each32([&](int k, const uint32_t (&x)[32]) {
        uint32_t mask = 0u;
#pragma unroll
        for (int e = 0; e < 32; ++e) mask |= __uint_as_float(x[e]) >= cut ? 1u << e : 0u;
        while (mask != 0u) {
          const int e = __ffs(mask) - 1;
          mask &= mask - 1u;
          float v = cut;
          if (!last || !c.exact) {                                        // the score is only needed for these
#pragma unroll
            for (int f = 0; f < 32; ++f) v = f == e ? __uint_as_float(x[f]) : v;
          } else {
            v = INFINITY;
          }
          take(v, c0 + k + e);
        }
      });
      listed = min(need, have);
    }
    tc_fence_before();
    __syncthreads();                                                     // TMEM has been read, the lists are written
    tc_fence_after();
  }
  if (ok) {
    // lists out, the kept blocks around the chosen ones
    for (int e = threadIdx.x; e < kTileKeys * args.n; e += Cfg::kThreads) {
      const int r = e / args.n, k = e % args.n, i = i0 + r;
      if (i < 0 || i >= len) continue;
      args.blocks[(out_row0 + i) * args.n + k] = k < args.keep_first ? k
                                                 : k >= args.n - args.keep_last ? nb - args.n + k
                                                                                : staged[r * (args.n + 1) + k];
    }
  }
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

cudaError_t launch_select(const SelectArgs& a, int device, cudaStream_t s) {
  using Cfg = SelectTileCfg;
  constexpr int kRowSmem = 200 * 1024, kTileSmem = static_cast<int>(Cfg::kListOff) + Cfg::kMaxListed * 128 * 8 + 1024;
  static bool configured[64] = {};
  if (!configured[device]) {
    cudaError_t e = cudaFuncSetAttribute(kb_select_row_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kb_select_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  // A CTA of 128 rows pays from about 16 rows per sequence on.  Its lists of
  // earlier passes hold 32 winners, so longer ones stay with it only while
  // all blocks fit one pass.
  const bool several = a.max_blocks - a.keep_last > Cfg::kPass;
  if (a.L > kSelectRowMax && (!several || a.n - a.keep_first - a.keep_last <= Cfg::kMaxListed)) {
    const int n_tiles = a.starts != nullptr ? (a.L + kTileKeys - 2) / kTileKeys + 1
                                            : (a.start + a.L - 1) / kTileKeys - a.start / kTileKeys + 1;
    const long long grid = static_cast<long long>(a.B) * a.Hkv * n_tiles;
    const int smem = several ? kTileSmem : static_cast<int>(Cfg::kListOff) + 1024;
    kb_select_tile_kernel<<<static_cast<unsigned>(grid), Cfg::kThreads, smem, s>>>(a, n_tiles);
    return cudaGetLastError();
  }
  const int rounds = (a.max_blocks + kChunkKeys - 1) / kChunkKeys;
  const size_t smem = (static_cast<size_t>(a.max_blocks) + (a.max_blocks > kChunkKeys ? 4u * rounds * a.n : 0u)) * 4u;
  const long long rows = static_cast<long long>(a.B) * a.Hkv * a.L;
  if (rows > 0x7FFFFFFFLL || smem > kRowSmem) return cudaErrorInvalidValue;
  kb_select_row_kernel<<<static_cast<unsigned>(rows), kSelectRowThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kb

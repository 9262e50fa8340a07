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
// at or above it (about 7 trials for a row, 12 for the slowest of 32; trials
// placed by the counts at both ends took as many); only ties keep the search
// going until the range is a single value, of which the first blocks are then
// taken.
#include "kb_boxes.cuh"
#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

// Search for the value that exactly `need` scores are at or above: the range
// [lo, hi) of values with count(>= lo) >= need > count(>= hi).
struct CutSearch {
  float lo, hi;
  bool exact;                                   // exactly `need` scores are at or above lo
  __device__ __forceinline__ CutSearch(float least, float most, bool all)
      : lo(least), hi(next_above(most)), exact(all) {}
  __device__ __forceinline__ static float next_above(float x) {
    const int b = __float_as_int(__fadd_rn(x, 0.0f));       // -0 counts as +0
    return __int_as_float(b >= 0 ? b + 1 : b - 1);
  }
  __device__ __forceinline__ float trial() const { return __fmaf_rn(0.5f, __fsub_rn(hi, lo), lo); }
  // No value lies between lo and hi, or the cut is exact.
  __device__ __forceinline__ bool done(float t) const { return exact || !(t > lo && t < hi); }
  __device__ __forceinline__ void counted(float t, int count, int need) {
    if (count >= need) lo = t;
    else hi = t;
    exact = count == need;
  }
};
// Scores are whole multiples of a power of two and below 2^22 of them, so
// halving ends within a few dozen steps of 22 bits, except around zero, where
// floats go on down to 2^-149: 264 halvings at most, 271 between the bounds to
// which scores of boxes that are no boxes saturate.  Scores must be finite:
// with an infinite or NaN one the range has no middle, or fewer than `need`
// scores reach any value, and a row's winners would not fill its places exactly.
constexpr int kMaxTrials = 300;

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

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));       // NaN goes through
  return r;
}
// All ones in the half of every negative value of a bf16 pair.
__device__ __forceinline__ uint32_t bf16x2_sign_mask(uint32_t w) {
  return ((w & 0x8000u) ? 0x0000FFFFu : 0u) | ((w & 0x80000000u) ? 0xFFFF0000u : 0u);
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
// channels of both bounds each), so a warp has twelve blocks of 512 bytes
// in flight, the first of them while the query is still on its way to whole
// numbers.  For one token the boxes are read once and nothing else counts:
// 16 sequences of 64K (33.6 MB) take 13.0 to 13.7 us, 128 CTAs whose loads,
// search and start follow one another.
//
// It also runs for longer calls that the tile kernel does not take (more than
// 256 blocks to choose from and more than 32 of them by score): there every row
// reads its boxes again, 872 us for 2048 rows at 64K and 35 blocks a row, where
// the tile kernel takes 136 us for 34.
constexpr int kSelectRowThreads = 512;
// Query rows per sequence up to which this kernel runs, whatever the batch and
// the number of blocks.  Measured at 16 blocks a row, this kernel against the
// tile kernel (a replayed graph, L2 flushed): B = 1 and 64 blocks, 16 rows 13.5
// us against 21.6, 64 rows 27.8 against 21.6; 512 blocks, 16 rows 15.5 against
// 116, 64 rows 40 against 119; B = 16 and 64 blocks, 1 row 13.5 against 21.6, 4
// rows 27.8 against 21.6, 16 rows 77 against 23.6; 512 blocks, 12 rows 95 against
// 116, 16 rows 120 against 114.  One number meets the last of these; a batch of
// short contexts pays from 4 rows on, one long context not before 64.
constexpr int kSelectRowMax = 16;

__global__ void __launch_bounds__(kSelectRowThreads, 1) kb_select_row_kernel(const SelectArgs args) {
  extern __shared__ float sel_smem[];
  __shared__ float whole[kHeadDim];               // n
  __shared__ uint32_t amax_bits[8];
  __shared__ int warp_sums[2][kSelectRowThreads / 32];
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
  constexpr int kAtOnce = 6, kStep = kSelectRowThreads / 16;
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
        q[h] = saturated(__bfloat162float(static_cast<const __nv_bfloat16*>(
            args.q)[((static_cast<size_t>(b) * args.Hkv + g) * kGroup + h) * args.L * kHeadDim +
                    static_cast<size_t>(i) * kHeadDim + threadIdx.x]));
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
    u = whole_sum(q[0], q[1], q[2], q[3], exp2i(15 - grid_exponent(__uint_as_float(mb))));
    const uint32_t ub = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(u)));
    if (lane == 0) amax_bits[4 + warp] = ub;
  }
  __syncthreads();
  if (warp < 4) {
    const uint32_t ub = max(max(amax_bits[4], amax_bits[5]), max(amax_bits[6], amax_bits[7]));
    whole[threadIdx.x] = rint_scaled(u, exp2i(7 - grid_exponent(__uint_as_float(ub))));
  }
  __syncthreads();
  float n[8];
  uint32_t up[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) n[e] = whole[8 * c + e];
#pragma unroll
  for (int e = 0; e < 4; ++e) up[e] = (n[2 * e] > 0.0f ? 0x0000FFFFu : 0u) | (n[2 * e + 1] > 0.0f ? 0xFFFF0000u : 0u);
  for (int j0 = j_first; j0 < m + (lane >> 4); j0 += kStep * kAtOnce) {        // uniform over the warp
    float s[kAtOnce];
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a) s[a] = box_dot(hi[a], lo[a], up, n);
    if (j0 + kStep * kAtOnce < m + (lane >> 4)) fetch(j0 + kStep * kAtOnce);
#pragma unroll
    for (int k = 8; k >= 1; k >>= 1)
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) s[a] = __fadd_rn(s[a], __shfl_xor_sync(0xffffffffu, s[a], k));
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a)
      if (c == 0 && j0 + a * kStep < m) sel_smem[j0 + a * kStep] = saturated_score(s[a]);
  }
  __syncthreads();
  // the cut, by all threads: thread t holds scores t, t + 512, ..
  int turn = 0;
  auto sum_of = [&](int mine) {                   // over the CTA
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) warp_sums[turn][warp] = mine;
    __syncthreads();
    const int all = __reduce_add_sync(0xffffffffu, lane < kSelectRowThreads / 32 ? warp_sums[turn][lane] : 0);
    turn ^= 1;                                    // the other buffer next: one barrier is enough
    return all;
  };
  float least = INFINITY, most = -INFINITY;
  for (int j = threadIdx.x; j < m; j += kSelectRowThreads) {
    least = fminf(least, sel_smem[j]);
    most = fmaxf(most, sel_smem[j]);
  }
  {
    // extremes over the CTA, as unsigned numbers of the same order
    auto key = [](float x) {
      const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
      return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    };
    auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k); };
    const uint32_t klo = __reduce_min_sync(0xffffffffu, key(least)), khi = __reduce_max_sync(0xffffffffu, key(most));
    if (lane == 0) {
      warp_sums[0][warp] = static_cast<int>(klo);
      warp_sums[1][warp] = static_cast<int>(khi);
    }
    __syncthreads();
    const int from = lane & (kSelectRowThreads / 32 - 1);
    least = value(__reduce_min_sync(0xffffffffu, static_cast<uint32_t>(warp_sums[0][from])));
    most = value(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(warp_sums[1][from])));
    __syncthreads();
  }
  CutSearch s(least, most, m <= need);
#pragma unroll 1
  for (int iter = 0; iter < kMaxTrials; ++iter) {
    const float t = s.trial();
    if (s.done(t)) break;                         // the same in every thread
    int count = 0;
    for (int j = threadIdx.x; j < m; j += kSelectRowThreads) count += sel_smem[j] >= t ? 1 : 0;
    s.counted(t, sum_of(count), need);
  }
  int ties = 0;                                   // scores equal to the cut that are taken
  if (!s.exact) {
    int above = 0;
    for (int j = threadIdx.x; j < m; j += kSelectRowThreads) above += sel_smem[j] > s.lo ? 1 : 0;
    ties = need - sum_of(above);
  }
  // winners out in block order: a place is the number of winners before it
  int before = 0, tied_before = 0;                // of the blocks of earlier slabs of 512
  const uint32_t below = (1u << lane) - 1u;
  for (int j0 = 0; j0 < m; j0 += kSelectRowThreads) {
    const int j = j0 + static_cast<int>(threadIdx.x);
    const float v = j < m ? sel_smem[j] : -INFINITY;
    const bool tied = !s.exact && v == s.lo;
    const uint32_t win = __ballot_sync(0xffffffffu, v >= s.lo && !tied), eq = __ballot_sync(0xffffffffu, tied);
    if (lane == 0) warp_sums[turn][warp] = __popc(win) | (__popc(eq) << 16);
    __syncthreads();
    const int theirs = lane < kSelectRowThreads / 32 ? warp_sums[turn][lane] : 0;
    const int earlier = __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0);      // two sums in one word: at most 512 each
    const int all = __reduce_add_sync(0xffffffffu, theirs);
    turn ^= 1;
    const int n_win = before + (earlier & 0xFFFF) + __popc(win & below);
    const int n_eq = tied_before + (earlier >> 16) + __popc(eq & below);
    if (tied ? n_eq < ties : v >= s.lo) out[c0 + n_win + min(n_eq, ties)] = c0 + j;
    before += all & 0xFFFF;
    tied_before += all >> 16;
  }
  for (int t = threadIdx.x; t < args.keep_first + args.keep_last; t += kSelectRowThreads)
    if (t < args.keep_first) out[t] = t;
    else out[args.n - args.keep_last + t - args.keep_first] = nb - args.keep_last + t - args.keep_first;
}

// ------------------------------------------------------ 128 rows per CTA
//
// One CTA per (batch, KV head, 128 positions from a multiple of 128 on), so
// its rows share their blocks 0 .. t.  Scores are one product of grid vectors,
// [n+ | n-] (128 rows x 256) times [upper | lower] (blocks x 256), on the
// tensor core, exact like every other order of summation.  They stay in TMEM
// (a row per lane, a block per column).  A quad of threads searches a row: the
// 16x256b TMEM load gives thread u columns 8r + 2u and 8r + 2u + 1 of every
// group of 8, for two rows, so counts are added by two shuffles, and 128
// blocks of both rows are 64 registers.  Rows whose blocks exceed TMEM go on
// in passes of 256 blocks, the winners of the earlier ones carried along in
// shared memory.
// Bound: q is read once (1 KB a row and KV head); 96 KB of shared memory and
// half of TMEM let two CTAs share an SM, so one loads while the other
// searches.  A 16K prompt (134 MB of q) takes 92 us, 1.5 TB/s: rounding q to
// whole numbers and the search are instructions (56 % of issue slots), and a
// tile's slowest row holds up its CTA.  Sixteen rows per warp with register
// products of 16 x 8 in place of tcgen05, so that no warp waits for another,
// took 141 us.
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
  static constexpr uint32_t kMaskOff = kMiscOff + 16;       // [row][9] chosen columns of a pass, 32 to a word
  static constexpr uint32_t kListOff = kMaskOff + 128 * 9 * 4;        // several passes: score and block per winner and row
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
    for (int r = warp; r < kTileKeys; r += Cfg::kThreads / 32) {
      const int i = i0 + r;
      if (i < 0 || i >= len) continue;
      for (int k = lane; k < args.n; k += 32)
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
  // boxes of the 64 blocks from j0 on: into registers, then into the B operand
  // (a box is a row of it)
  constexpr int kBoxLoads = Cfg::kChunk * 32 / Cfg::kThreads;
  auto fetch_boxes = [&](int j0, int j1, uint4 (&val)[kBoxLoads]) {
#pragma unroll
    for (int k = 0; k < kBoxLoads; ++k) {
      const int e = threadIdx.x + k * Cfg::kThreads, j = j0 + (e >> 5);
      const __nv_bfloat16* box = j < j1 ? box_of(args, b, g, j) : nullptr;
      val[k] = box != nullptr ? __ldg(reinterpret_cast<const uint4*>(box) + (e & 31)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto put_boxes = [&](const uint4 (&val)[kBoxLoads]) {
#pragma unroll
    for (int k = 0; k < kBoxLoads; ++k) {
      const int e = threadIdx.x + k * Cfg::kThreads, r = e >> 5, c = e & 31;
      *reinterpret_cast<uint4*>(smem + Cfg::kBOff + (c >> 3) * Cfg::kBSlab + (r >> 3) * 1024 + (r & 7) * 128 +
                                (((c & 7) ^ (r & 7)) << 4)) =
          make_uint4(saturated_bf16x2(val[k].x), saturated_bf16x2(val[k].y), saturated_bf16x2(val[k].z), saturated_bf16x2(val[k].w));
    }
  };
  {
    uint4 val[kBoxLoads];
    fetch_boxes(0, min(cand1, Cfg::kPass), val);
    put_boxes(val);
  }

  // n of the tile's rows: 16 lanes per row, eight channels of the four heads
  // each, written as the two halves n+ and n- of the A operand
  {
    const int c = lane & 15;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.q) +
                                                    (static_cast<size_t>(b) * args.Hkv + g) * kGroup * args.L * kHeadDim);
    const size_t head_step = static_cast<size_t>(args.L) * (kHeadDim / 8);
    constexpr int kAtOnce = 2;                              // rows in flight per lane
    auto fetch = [&](int m0, uint4 (&x)[kAtOnce][kGroup]) {
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int i = i0 + m0 + 16 * a;
        const bool in = m0 + 16 * a < kTileKeys && i >= 0 && i < len;
#pragma unroll
        for (int h = 0; h < kGroup; ++h)
          x[a][h] = in ? __ldg(q + h * head_step + static_cast<size_t>(i) * (kHeadDim / 8) + c) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    uint4 x[kAtOnce][kGroup], ahead[kAtOnce][kGroup];
    fetch(2 * warp + (lane >> 4), ahead);
#pragma unroll 1
    for (int m0 = 2 * warp + (lane >> 4); m0 < kTileKeys; m0 += 16 * kAtOnce) {
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a)
#pragma unroll
        for (int h = 0; h < kGroup; ++h) x[a][h] = ahead[a][h];
      fetch(m0 + 16 * kAtOnce, ahead);                      // the next rows are on their way while these are rounded
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        uint32_t top = 0u;                                  // largest magnitudes, a bf16 pair
#pragma unroll
        for (int h = 0; h < kGroup; ++h) {
          const uint32_t w[4] = {x[a][h].x, x[a][h].y, x[a][h].z, x[a][h].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = bf16x2_max_nan(top, w[e] & 0x7FFF7FFFu);
        }
        uint32_t top32 = max(top << 16, top & 0xFFFF0000u);  // as fp32 bits, whose order is that of the magnitudes
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) top32 = max(top32, __shfl_xor_sync(0xffffffffu, top32, m));
        const float amax = __uint_as_float(top32);
        const float scale = exp2i(15 - grid_exponent(amax));
        const bool off_grid = !(amax <= kGridMax);          // beyond the grid, infinite or NaN
        float u[8], umax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v[kGroup];
#pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            const uint32_t w = e < 2 ? x[a][h].x : e < 4 ? x[a][h].y : e < 6 ? x[a][h].z : x[a][h].w;
            v[h] = __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
            if (off_grid) v[h] = saturated(v[h]);
          }
          u[e] = whole_sum(v[0], v[1], v[2], v[3], scale);
          umax = fmaxf(umax, fabsf(u[e]));
        }
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) umax = fmaxf(umax, __shfl_xor_sync(0xffffffffu, umax, m));
        const float fit = exp2i(7 - grid_exponent(umax));
        uint32_t np[4], nm[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = pack_bf16x2(rint_scaled(u[2 * e], fit), rint_scaled(u[2 * e + 1], fit));
          const uint32_t neg = bf16x2_sign_mask(w);         // n- has the negative channels, n+ the others
          np[e] = w & ~neg;
          nm[e] = w & neg;
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
  // rows of this thread: rA and rA + 8 of the warp's 16, shared by its quad
  const int lane_base = 32 * (warp & 3) + 16 * (warp >> 2);
  const int u4 = lane & 3, rA = lane_base + (lane >> 2);
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + Cfg::kMaskOff);
  float* list_s = reinterpret_cast<float*>(smem + Cfg::kListOff);        // [winner][row]
  int* list_j = reinterpret_cast<int*>(smem + Cfg::kListOff) + Cfg::kMaxListed * 128;
  int* staged = reinterpret_cast<int*>(smem + Cfg::kAOff);             // [row][n + 1], once A is no longer read
  int listed = 0;                                                      // winners carried from earlier passes (every row's)
  uint32_t phase = 0;
  bool ok = true;
  for (int pass = 0; pass < passes; ++pass) {
    const int c0 = pass * Cfg::kPass, c1 = min(cand1, c0 + Cfg::kPass);
    uint4 val[kBoxLoads];
    for (int j0 = c0; j0 < c1; j0 += Cfg::kChunk) {
      if (j0 > 0) {
        fetch_boxes(j0, c1, val);
        put_boxes(val);
      }
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
      const uint32_t s_tmem = tmem_base + (static_cast<uint32_t>(lane_base) << 16);
      const int cols = c1 - c0, skip = max(0, cand0 - c0);               // columns skip .. cols-1 are candidates
      // 64 columns from k on: x[4r], x[4r+1] of row A, x[4r+2], x[4r+3] of row
      // B, columns k + 8r + 2 u4 and the next; other columns as -inf, below
      // every trial.  The whole warp reads TMEM together.
      auto load64 = [&](int k, uint32_t (&x)[32]) {
        __syncwarp();
        tmem_ld_16x256b_x8_wait(s_tmem + static_cast<uint32_t>(k), x);
        if (k < skip || k + 64 > cols) {
#pragma unroll
          for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = k + 8 * r + 2 * u4 + e;
              if (col < skip || col >= cols) x[4 * r + e] = x[4 * r + 2 + e] = 0xFF800000u;
            }
        }
      };
      uint32_t x0[32], x1[32];
      load64(0, x0);
      if (cols > 64) load64(64, x1);
      // fn(first column, x) over the pass's columns; the first 128 stay in registers
      auto each64 = [&](auto fn) {
        fn(0, x0);
        if (cols > 64) fn(64, x1);
        for (int k = 128; k < cols; k += 64) {
          uint32_t x[32];
          load64(k, x);
          fn(k, x);
        }
      };
      auto quad_sum = [](int v) {
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        return v + __shfl_xor_sync(0xffffffffu, v, 2);
      };
      // carried winners of a row: the quad takes every fourth
      auto carried = [&](int r, auto fn) {
        for (int w = u4; w < listed; w += 4) fn(list_s[w * 128 + r], list_j[w * 128 + r]);
      };
      float hiA = -INFINITY, hiB = -INFINITY, loA = INFINITY, loB = INFINITY;
      each64([&](int, const uint32_t (&x)[32]) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = __uint_as_float(x[4 * r + e]), z = __uint_as_float(x[4 * r + 2 + e]);
            hiA = fmaxf(hiA, a);
            hiB = fmaxf(hiB, z);
            loA = fminf(loA, a == -INFINITY ? INFINITY : a);
            loB = fminf(loB, z == -INFINITY ? INFINITY : z);
          }
      });
      carried(rA, [&](float v, int) { hiA = fmaxf(hiA, v); loA = fminf(loA, v); });
      carried(rA + 8, [&](float v, int) { hiB = fmaxf(hiB, v); loB = fminf(loB, v); });
      __syncwarp();
#pragma unroll
      for (int k = 1; k <= 2; k <<= 1) {
        hiA = fmaxf(hiA, __shfl_xor_sync(0xffffffffu, hiA, k));
        hiB = fmaxf(hiB, __shfl_xor_sync(0xffffffffu, hiB, k));
        loA = fminf(loA, __shfl_xor_sync(0xffffffffu, loA, k));
        loB = fminf(loB, __shfl_xor_sync(0xffffffffu, loB, k));
      }
      // the pass's winners: all of them when there are at most `need`, else
      // those above the cut; ties at the cut from the lowest block on
      const int have = cols - min(cols, skip) + listed;
      CutSearch sA(loA, hiA, have <= need), sB(loB, hiB, have <= need);
      for (int iter = 0; iter < kMaxTrials; ++iter) {
        const float tA = sA.trial(), tB = sB.trial();
        const bool doneA = sA.done(tA), doneB = sB.done(tB);
        if (__all_sync(0xffffffffu, doneA && doneB)) break;
        int nA = 0, nB = 0;
        each64([&](int, const uint32_t (&x)[32]) {
#pragma unroll
          for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              nA += __uint_as_float(x[4 * r + e]) >= tA ? 1 : 0;
              nB += __uint_as_float(x[4 * r + 2 + e]) >= tB ? 1 : 0;
            }
        });
        if (listed > 0) {
          carried(rA, [&](float v, int) { nA += v >= tA ? 1 : 0; });
          carried(rA + 8, [&](float v, int) { nB += v >= tB ? 1 : 0; });
          __syncwarp();
        }
        nA = quad_sum(nA | (nB << 16));                                   // two counts of at most 288 in one word
        if (!doneA) sA.counted(tA, nA & 0xFFFF, need);
        if (!doneB) sB.counted(tB, nA >> 16, need);
      }
      // the chosen columns as bit masks, a word for 32 columns: a thread's
      // share of a word are bits 8(r%4) + 2 u4 + e; the quad's shares are ORed
      // and thread u4 stores the words u4, u4 + 4, ..
      const bool tied = __any_sync(0xffffffffu, !sA.exact || !sB.exact);
      auto put_masks = [&](int k, const uint32_t (&x)[32], int half, bool strict, int word0) {
        // half 0: row A, 1: row B; strict: above the cut only, else at or above
        const float cut = half ? sB.lo : sA.lo;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w = 0u;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float v = __uint_as_float(x[4 * (4 * h + r) + 2 * half + e]);
              if (strict ? v > cut : v >= cut) w |= 1u << (8 * r + e);
            }
          w <<= 2 * u4;
          w |= __shfl_xor_sync(0xffffffffu, w, 1);
          w |= __shfl_xor_sync(0xffffffffu, w, 2);
          const int word = word0 + k / 32 + h;
          if (u4 == (word & 3)) masks[(rA + 8 * half) * 9 + word] = w;
        }
      };
      auto write_masks = [&](bool strict) {
        each64([&](int k, const uint32_t (&x)[32]) {
          put_masks(k, x, 0, strict, 0);
          put_masks(k, x, 1, strict, 0);
        });
        __syncwarp();
      };
      const bool last = pass == passes - 1;
      const int words = (cols + 31) / 32;
      write_masks(false);
      if (tied) {
        // rows whose cut is tied: the words now hold the columns at or above
        // it; keep the strict ones and the first of the tied ones.  Rare, so
        // thread 0 and 1 of a quad do it serially, a row each.
        uint32_t at_or_above[8];
        const int rr = rA + 8 * u4;
        if (u4 < 2)
#pragma unroll
          for (int k = 0; k < 8; ++k) at_or_above[k] = k < words ? masks[rr * 9 + k] : 0u;
        __syncwarp();
        write_masks(true);
        if (u4 < 2) {
          const bool exact = u4 ? sB.exact : sA.exact;
          const float cut = u4 ? sB.lo : sA.lo;
          int above = 0;
          for (int k = 0; k < words; ++k) above += __popc(masks[rr * 9 + k]);
          for (int w = 0; w < listed; ++w) above += list_s[w * 128 + rr] > cut ? 1 : 0;
          int left = exact ? 0x7FFFFFFF : need - above;
          for (int w = 0; w < listed; ++w)                                // carried ones come first
            if (list_s[w * 128 + rr] == cut && left-- <= 0) list_s[w * 128 + rr] = -INFINITY;
          left = max(left, 0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k >= words) break;
            uint32_t eq = at_or_above[k] & ~masks[rr * 9 + k], keep = 0u;
            for (; eq != 0u && left > 0; --left) {
              keep |= eq & (0u - eq);
              eq &= eq - 1u;
            }
            masks[rr * 9 + k] |= keep;
          }
        }
        __syncwarp();
      }
      if (last) {
        // a row's winners in block order: carried ones (thread 0 of the quad),
        // then those of words u4 and u4 + 4
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int r = rA + 8 * half;
          const float cut = half ? sB.lo : sA.lo;
          int* const mine = staged + r * (args.n + 1);
          for (int k = u4; k < args.keep_first; k += 4) mine[k] = k;
          for (int k = u4; k < args.keep_last; k += 4) mine[args.n - 1 - k] = nb - 1 - k;
          int at = args.keep_first;
          for (int w = 0; w < listed; ++w)
            if (list_s[w * 128 + r] >= cut) {
              if (u4 == 0) mine[at] = list_j[w * 128 + r];
              ++at;
            }
          for (int k = 0; k < words; ++k) {
            uint32_t m = masks[r * 9 + k];
            if ((k & 3) != u4) {
              at += __popc(m);
              continue;
            }
            for (; m != 0u; m &= m - 1u) mine[at++] = c0 + 32 * k + __ffs(m) - 1;
          }
          __syncwarp();
        }
      } else {
        // carry the winners on: the earlier ones move down (in place, by
        // thread 0), then each column's score goes to its place
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = rA + 8 * half;
          const float cut = half ? sB.lo : sA.lo;
          int kept = 0;
          if (u4 == 0)
            for (int w = 0; w < listed; ++w) {
              const float v = list_s[w * 128 + r];
              if (v < cut) continue;
              list_s[kept * 128 + r] = v;
              list_j[kept * 128 + r] = list_j[w * 128 + r];
              ++kept;
            }
          __syncwarp();
          kept = __shfl_sync(0xffffffffu, kept, lane & ~3);
          each64([&](int k, const uint32_t (&x)[32]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int col = k + 8 * i + 2 * u4 + e;
                if (col >= cols || !((masks[r * 9 + col / 32] >> (col & 31)) & 1u)) continue;
                int at = kept + __popc(masks[r * 9 + col / 32] & ((1u << (col & 31)) - 1u));
                for (int w = 0; w < col / 32; ++w) at += __popc(masks[r * 9 + w]);
                list_s[at * 128 + r] = __uint_as_float(x[4 * i + 2 * half + e]);
                list_j[at * 128 + r] = c0 + col;
              }
          });
          __syncwarp();
        }
      }
      listed = min(need, have);
    }
    if (pass + 1 < passes) {
      tc_fence_before();
      __syncthreads();                                                   // TMEM has been read
      tc_fence_after();
    }
  }
  if (ok) {
    // the warp's sixteen lists out, one after another
    for (int rr = lane / args.n, k = lane % args.n; rr < 16;) {
      const int i = i0 + lane_base + rr;
      if (i >= 0 && i < len) args.blocks[(out_row0 + i) * args.n + k] = staged[(lane_base + rr) * (args.n + 1) + k];
      rr += 32 / args.n;
      k += 32 % args.n;
      if (k >= args.n) {
        k -= args.n;
        ++rr;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

cudaError_t launch_select(const SelectArgs& a, int device, cudaStream_t s) {
  using Cfg = SelectTileCfg;
  constexpr int kRowSmem = 128 * 1024, kTileSmem = static_cast<int>(Cfg::kListOff) + Cfg::kMaxListed * 128 * 8 + 1024;
  static bool configured[64] = {};
  if (!configured[device]) {
    cudaError_t e = cudaFuncSetAttribute(kb_select_row_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kb_select_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  // A CTA of 128 rows pays from some number of rows per sequence on (measured
  // at kSelectRowMax).  Its lists of earlier passes hold 32 winners, so longer
  // ones stay with it only while all blocks fit one pass.
  const bool several = a.max_blocks - a.keep_last > Cfg::kPass;
  if (a.L > kSelectRowMax && (!several || a.n - a.keep_first - a.keep_last <= Cfg::kMaxListed)) {
    const int n_tiles = a.starts != nullptr ? (a.L + kTileKeys - 2) / kTileKeys + 1
                                            : (a.start + a.L - 1) / kTileKeys - a.start / kTileKeys + 1;
    const long long grid = static_cast<long long>(a.B) * a.Hkv * n_tiles;
    const int smem = several ? kTileSmem : static_cast<int>(Cfg::kListOff) + 1024;
    kb_select_tile_kernel<<<static_cast<unsigned>(grid), Cfg::kThreads, smem, s>>>(a, n_tiles);
    return cudaGetLastError();
  }
  const size_t smem = static_cast<size_t>(a.max_blocks) * 4u;
  const long long rows = static_cast<long long>(a.B) * a.Hkv * a.L;
  if (rows > 0x7FFFFFFFLL || smem > kRowSmem) return cudaErrorInvalidValue;
  kb_select_row_kernel<<<static_cast<unsigned>(rows), kSelectRowThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kb

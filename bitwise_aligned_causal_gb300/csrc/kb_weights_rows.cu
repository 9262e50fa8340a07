// kb_weights_rows.cu -- the attention weight that each cached key gets from
// many query rows (more than the packed kernel of kb_weights.cu holds):
//   w_j += sum over rows i and heads h of 2^(s c - lse log2 e),
// s = q_i . k_j, c = log2(e) / sqrt(128).
//
// S = Q K^T with a query row per TMEM lane: a thread's offset -lse log2(e) is a
// register, and its 64 keys' sums stay in registers while tiles of query rows
// stream by; lanes meet once per pair of key tiles.  (With a key per lane the
// offsets came from shared memory, whose loads and the MMA's operands together
// were the bound: 8K prompt 298 us.)  Two key tiles are the B operand of one
// MMA with N = 256, so the product reads 96 bytes of shared memory a clock, not
// 128.  The rows of a group's four heads are one sequence of 4 L rows in memory
// and are cut into tiles as such, across heads.
//   warps 0..15   weights: warp w takes lanes 32 (w % 4) .. +31, keys 64 (w / 4) .. +63
//   warp 16       TMA producer      warp 17   TMEM allocator + MMA issuer (one lane)
//   warp 18       per tile of rows: their offsets (-inf for a row that gives nothing)
//                 and what the weight warps have to know of the tile, in shared
//                 memory (their registers are full of sums)
// TMEM: two score buffers of 256 columns.  Shared memory: two pairs of key
// tiles, three tiles of query rows.
//
// A CTA takes key pairs first, first + splits, ...; where there are few pairs,
// a cluster of CTAs shares one, each every ctas-th tile of rows, and their sums
// meet in the first CTA's shared memory in the order of ranks, so a call gives
// the same bits every time.  A register adds one term per tile of rows: a sum
// over R rows rounds at most R / 32 + 16 times.
//
// Measured: 8K prompt 236 us, of which the products alone take 210 (0.77 us
// each, 87% of the rate of a large library product) and the longest CTA, the
// first keys' 256 tiles, sets the time where the average is 219; 2048 rows over
// their own keys 33 us (63 without clusters), over 32K 425.
#include <algorithm>

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

struct RowsCfg {
  static constexpr int kSumWarps = 16;
  static constexpr int kSumThreads = kSumWarps * 32;
  static constexpr int kThreads = kSumThreads + 96;
  static constexpr int kPairKeys = 2 * kTileKeys;
  static constexpr uint32_t kPairBytes = 2 * kTileBytes;
  static constexpr int kKSlots = 2, kQSlots = 3;
  static constexpr uint32_t kKOff = 0;
  static constexpr uint32_t kQOff = kKSlots * kPairBytes;
  static constexpr uint32_t kPartOff = kQOff + kQSlots * kTileBytes;      // float per key of a pair: the quarters' sums
  static constexpr uint32_t kRowOff = kPartOff + kPairKeys * 4;           // float -lse log2 e x 128, per score buffer
  static constexpr uint32_t kHeadOff = kRowOff + 2 * kTileRows * 4;       // int r0, flags, per score buffer
  static constexpr int kMasked = 1, kLast = 2;            // flags of a tile: some row does not see some key; the pair's last
  static constexpr uint32_t kBarOff = kHeadOff + 16;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kKSlots;
  static constexpr int kBarQFull = kBarKEmpty + kKSlots;
  static constexpr int kBarQEmpty = kBarQFull + kQSlots;
  static constexpr int kBarDFull = kBarQEmpty + kQSlots;  // per score buffer: product and rows' offsets there
  static constexpr int kBarDEmpty = kBarDFull + 2;        // ... read by all of the weight threads
  static constexpr int kBarDrain = kBarDEmpty + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr uint32_t kMiscOff = kBarOff + (kNumBars + 1) / 2 * 16;
  static constexpr uint32_t kSmemUsed = kMiscOff + 16;
  static constexpr uint32_t kSmemBytes = kSmemUsed;
  static_assert(kSmemBytes <= 227u * 1024u, "shared memory budget");
};

// Tiles of the group's 4 L query rows that a pair of key tiles meets.
struct RowTiles {
  int t, r0;                   // the tile; the row (of its head) that it begins with
  int n, L, rows, step, inc;   // tiles in all, rows per head, of them live, tiles to the next, and rows (mod L)
  int key0, pos0;              // first key of the pair; position of row 0
  __device__ __forceinline__ bool cross() const { return r0 + kTileRows > L; }       // begins in one head, ends in another (or behind the last)
  __device__ __forceinline__ bool live() const {
    return (cross() || r0 < rows) && pos0 + (cross() ? rows : min(r0 + kTileRows, rows)) - 1 >= key0;
  }
  __device__ __forceinline__ bool masked() const {
    return cross() || r0 + kTileRows > rows || pos0 + r0 < key0 + RowsCfg::kPairKeys - 1;
  }
  __device__ __forceinline__ void skip() {
    while (t < n && !live()) move();
  }
  __device__ __forceinline__ void move() {
    t += step;
    r0 += inc;
    if (r0 >= L) r0 -= L;
  }
  __device__ __forceinline__ void next() {
    move();
    skip();
  }
};

__device__ __forceinline__ void rows_drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 50000000ull) break;
}

// A thread's row over its 64 keys: off its -lse log2 e; kMasked: it gives
// nothing to keys behind the seen-th.  (Four warps a scheduler cover the loads'
// latency; a second buffer would not fit beside the sums.)
template <bool kMasked>
__device__ __forceinline__ void add64(uint32_t d, float off, int seen, float2 (&acc)[32]) {
  const float c = score_scale_log2();
  const float2 c2 = make_float2(c, c), off2 = make_float2(off, off);
#pragma unroll
  for (int at = 0; at < 32; at += 8) {
    uint32_t x[16];
    tmem_ld16_wait(d + 2 * at, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, off2);
      float2 w = make_float2(ex2_approx(a.x), ex2_approx(a.y));
      if (kMasked) {
        if (2 * (at + i) > seen) w.x = 0.0f;
        if (2 * (at + i) + 1 > seen) w.y = 0.0f;
      }
      acc[at + i] = __fadd2_rn(acc[at + i], w);
    }
  }
}

// Keys `key` and `key` + 1 of sequence b.
__device__ __forceinline__ void add_to_weights(const WeightsArgs& a, int b, int bg, int seq_kv, int key, const float2& sum) {
  if (a.block_table != nullptr && key < seq_kv) {         // (a tile without a page got zeros for keys: nothing is added)
    const int pg = __ldg(a.block_table + static_cast<size_t>(b) * a.pages_per_seq + key / a.page_size);
    if (pg < 0 || pg >= a.num_pages) return;
  }
  float* w = a.weights + static_cast<size_t>(bg) * a.kv_cap + key;
  if (key < seq_kv) w[0] = __fadd_rn(w[0], sum.x);
  if (key + 1 < seq_kv) w[1] = __fadd_rn(w[1], sum.y);
}

}  // namespace

__global__ void __launch_bounds__(RowsCfg::kThreads, 1)
kb_weights_rows_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const WeightsArgs args) {
  using Cfg = RowsCfg;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return smem_addr(bars + i); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ctas = args.ctas;
  const int rank = static_cast<int>(blockIdx.x) % ctas;   // in the cluster
  const int unit = static_cast<int>(blockIdx.x) / ctas;
  const int bg = unit % (args.B * args.Hkv);
  const int first = unit / (args.B * args.Hkv);
  const int b = bg / args.Hkv, g = bg % args.Hkv;
  int pos0 = args.start, rows = args.L;
  if (args.starts != nullptr) {
    pos0 = args.starts[b];
    rows = args.lens[b];
    if (pos0 < 0 || rows < 0 || rows > args.L || pos0 > args.kv_cap - rows) {
      if (threadIdx.x == 0 && first == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return;                                             // (the whole cluster)
    }
  }
  const int seq_kv = pos0 + rows;
  const int n_pairs = rows == 0 ? 0 : (seq_kv - 1) / Cfg::kPairKeys + 1;
  if (first >= n_pairs) return;                           // (the whole cluster)
  auto tiles_of = [&](int j) {
    RowTiles t{rank, rank * kTileRows % args.L, (kGroup * args.L + kTileRows - 1) / kTileRows, args.L, rows,
               ctas, ctas * kTileRows % args.L, j * Cfg::kPairKeys, pos0};
    t.skip();
    return t;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kNumBars; ++i)
      mbar_init(bar(i), i >= Cfg::kBarDEmpty && i < Cfg::kBarDrain ? Cfg::kSumWarps : i >= Cfg::kBarDFull && i < Cfg::kBarDEmpty ? 2u : 1u);
    if (sbase % 1024u != 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));    // (the swizzle's unit; never so)
    misc[1] = (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) ? 1u : 0u;
    fence_mbar_init();
  }
  if (warp == Cfg::kSumWarps + 1) {
    tmem_alloc(sbase + Cfg::kMiscOff, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (ctas > 1) cluster_arrive();                         // (waited for before another CTA's memory is written)
  const uint32_t tmem_base = misc[0];
  const bool skip = *abort_flag != 0;

  if (warp == Cfg::kSumWarps) {
    // ----------------------------------------------------------- producer
    if (lane == 0 && !skip) {
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_q);
      int K = 0, T = 0;                                   // pairs, tiles of rows
      bool ok = true;
      for (int j = first; j < n_pairs && ok; j += args.splits) {
        RowTiles it = tiles_of(j);
        if (it.t >= it.n) continue;
        const int ks = K % Cfg::kKSlots;
        if (K >= Cfg::kKSlots) ok = mbar_wait(bar(Cfg::kBarKEmpty + ks), (K / Cfg::kKSlots - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
        if (!ok) break;
        // (a second tile wholly behind the sequence is not read: no row sees its keys)
        const int live_tiles = (2 * j + 1) * kTileKeys < seq_kv ? 2 : 1;
        mbar_arrive_expect_tx(bar(Cfg::kBarKFull + ks), live_tiles * kTileBytes);
        for (int i = 0; i < live_tiles; ++i) {
          int row = (2 * j + i) * kTileKeys, plane = bg;
          if (args.block_table != nullptr) {
            int pg = args.block_table[static_cast<size_t>(b) * args.pages_per_seq + row / args.page_size];
            if (pg < 0 || pg >= args.num_pages) {
              atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
              pg = args.num_pages;                        // beyond the map: the TMA unit reads zeros
            }
            row = row % args.page_size;
            plane = pg * args.Hkv + g;
          }
          for (int h = 0; h < 2; ++h)
            tma_load_half(sbase + Cfg::kKOff + ks * Cfg::kPairBytes + h * kTileBytes + i * kSlabBytes, &tmap_k, row, h, plane,
                          bar(Cfg::kBarKFull + ks));
        }
        ++K;
        for (; it.t < it.n; it.next(), ++T) {
          const int qs = T % Cfg::kQSlots;
          if (T >= Cfg::kQSlots) ok = mbar_wait(bar(Cfg::kBarQEmpty + qs), (T / Cfg::kQSlots - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(Cfg::kBarQFull + qs), kTileBytes);
          tma_load_tile(sbase + Cfg::kQOff + qs * kTileBytes, &tmap_q, it.t * kTileRows, bg, bar(Cfg::kBarQFull + qs));
        }
      }
      if (!ok) {
        for (int x = max(K - Cfg::kKSlots, 0); x < K; ++x) rows_drain_wait(bar(Cfg::kBarKFull + x % Cfg::kKSlots), (x / Cfg::kKSlots) & 1);
        for (int x = max(T - Cfg::kQSlots, 0); x < T; ++x) rows_drain_wait(bar(Cfg::kBarQFull + x % Cfg::kQSlots), (x / Cfg::kQSlots) & 1);
      }
    }
  } else if (warp == Cfg::kSumWarps + 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0 && !skip) {
      const uint32_t idesc = idesc_bf16_f32(kTileRows, Cfg::kPairKeys, 0);
      int K = 0, T = 0;
      bool ok = true;
      for (int j = first; j < n_pairs && ok; j += args.splits) {
        RowTiles it = tiles_of(j);
        if (it.t >= it.n) continue;
        const int ks = K % Cfg::kKSlots;
        ok = mbar_wait(bar(Cfg::kBarKFull + ks), (K / Cfg::kKSlots) & 1, abort_flag, args.err, kDevTimeoutTma);
        for (; it.t < it.n && ok; it.next(), ++T) {
          const int qs = T % Cfg::kQSlots, db = T & 1;
          ok = mbar_wait(bar(Cfg::kBarQFull + qs), (T / Cfg::kQSlots) & 1, abort_flag, args.err, kDevTimeoutTma);
          if (ok && T >= 2) ok = mbar_wait(bar(Cfg::kBarDEmpty + db), (T / 2 - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem_base + db * 256u, desc_kmajor(sbase + Cfg::kQOff + qs * kTileBytes, kk, 1024u, kSlabBytes),
                   desc_kmajor(sbase + Cfg::kKOff + ks * Cfg::kPairBytes, kk, 1024u, 2 * kSlabBytes), idesc, kk > 0 ? 1u : 0u);
          tc_commit(bar(Cfg::kBarDFull + db));
          tc_commit(bar(Cfg::kBarQEmpty + qs));
        }
        if (!ok) break;
        tc_commit(bar(Cfg::kBarKEmpty + ks));
        ++K;
      }
      if (!ok) {
        tc_commit(bar(Cfg::kBarDrain));
        rows_drain_wait(bar(Cfg::kBarDrain), 0);
      }
    }
  } else if (warp == Cfg::kSumWarps + 2) {
    // ------------------------------------------------- the rows' offsets
    if (!skip) {
      constexpr float kLog2e = 1.44269504088896341f;
      const float* lse = args.lse + static_cast<size_t>(bg) * kGroup * args.L;
      int T = 0;
      bool ok = true;
      for (int j = first; j < n_pairs && ok; j += args.splits) {
        RowTiles it = tiles_of(j);
        while (it.t < it.n) {
          const int db = T & 1, r0 = it.r0;
          // the rows' log-sum-exps are on their way while the buffer is waited for
          float l[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = 32 * i + lane, m = it.t * kTileRows + x;
            l[i] = m < kGroup * args.L && (r0 + x) % args.L < rows ? __ldg(lse + m) : INFINITY;
          }
          int flags = it.masked() ? Cfg::kMasked : 0;
          it.next();
          if (it.t >= it.n) flags |= Cfg::kLast;
          if (T >= 2) {
            ok = mbar_wait(bar(Cfg::kBarDEmpty + db), (T / 2 - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          float* off = reinterpret_cast<float*>(smem + Cfg::kRowOff) + db * kTileRows;
#pragma unroll
          for (int i = 0; i < 4; ++i)      // a row that saw nothing (-inf) has no weights to give
            off[32 * i + lane] = l[i] == -INFINITY ? -INFINITY : __fmul_rn(-l[i], kLog2e);
          if (lane == 0) reinterpret_cast<int2*>(smem + Cfg::kHeadOff)[db] = make_int2(r0, flags);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Cfg::kBarDFull + db));
          ++T;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ weights
    const int quarter = warp & 3, group = warp >> 2;
    const int me = 32 * quarter + lane;                   // TMEM lane = row of a tile
    const uint32_t d_tmem = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + 64u * group;
    const float* row_off = reinterpret_cast<const float*>(smem + Cfg::kRowOff) + me;
    float2* part = reinterpret_cast<float2*>(smem + Cfg::kPartOff) + 32 * group + lane;
    int T = 0;
    bool ok = !skip;
    for (int j = first; j < n_pairs; j += args.splits) {
      float2 acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = make_float2(0.0f, 0.0f);
      bool more = true;
      if (ctas > 1) {                                     // (a CTA of a cluster may have no tile)
        const RowTiles it = tiles_of(j);
        more = it.t < it.n;
      }
      while (ok && more) {
        const int db = T & 1;
        ok = mbar_wait(bar(Cfg::kBarDFull + db), (T / 2) & 1, abort_flag, args.err, kDevTimeoutMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = d_tmem + db * 256u;
        const int2 head = reinterpret_cast<const int2*>(smem + Cfg::kHeadOff)[db];
        const float off = row_off[db * kTileRows];
        // (some row of these 32 does not see some key, or gives nothing; told by the
        // offsets' warp, the latter cost the 8K prompt 11 us)
        if ((head.y & Cfg::kMasked) || __any_sync(0xffffffffu, off == -INFINITY)) {
          int r = head.x + me;
          while (r >= args.L) r -= args.L;
          // a row that gives nothing (whatever stands in q) sees no key
          add64<true>(d, off, off == -INFINITY ? -1 : pos0 + r - (j * Cfg::kPairKeys + 64 * group), acc);
        } else {
          add64<false>(d, off, 0, acc);
        }
        more = (head.y & Cfg::kLast) == 0;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Cfg::kBarDEmpty + db));
        ++T;
      }
      // over the lanes, halving the keys each time: lane l ends with keys 2l and 2l + 1 of the 64
#pragma unroll
      for (int w = 16, n = 16; w >= 1; w >>= 1, n >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float2 mine = up ? acc[i + n] : acc[i], other = up ? acc[i] : acc[i + n];
          acc[i] = make_float2(__fadd_rn(mine.x, __shfl_xor_sync(0xffffffffu, other.x, w)),
                               __fadd_rn(mine.y, __shfl_xor_sync(0xffffffffu, other.y, w)));
        }
      }
      // one decision for the sixteen warps: all go on, or none does (and the part before has been read)
      if (named_bar_or(1, Cfg::kSumThreads, !ok)) break;
      float2 sum = acc[0];
      for (int i = 0; i < 4; ++i) {                       // over the quarters, in their order
        if (i == quarter) {
          if (i > 0) {
            const float2 v = *part;
            sum = make_float2(__fadd_rn(v.x, sum.x), __fadd_rn(v.y, sum.y));
          }
          if (i < 3 || ctas > 1) *part = sum;
        }
        if (i < 3) named_bar_sync(1, Cfg::kSumThreads);
      }
      if (quarter == 3 && ctas == 1) add_to_weights(args, b, bg, seq_kv, j * Cfg::kPairKeys + 64 * group + 2 * lane, sum);
    }
  }
  if (ctas > 1) {
    // One pair: its sums go to the first CTA's free slot of key tiles.  (A CTA
    // that gave up has set the error word; then nothing is added.)
    __syncthreads();
    cluster_wait();
    const int t = static_cast<int>(threadIdx.x);
    const uint32_t slot = sbase + Cfg::kKOff + Cfg::kPairBytes + t * 8u;
    const float2* part = reinterpret_cast<const float2*>(smem + Cfg::kPartOff);
    if (rank > 0 && t < kTileKeys) st_cluster_f32x2(smem_addr_in_cta(slot + rank * Cfg::kPairKeys * 4u, 0u), part[t]);
    cluster_sync();
    if (rank == 0 && t < kTileKeys && *reinterpret_cast<volatile uint32_t*>(args.err) == 0) {
      float2 sum = part[t];
      for (int r = 1; r < ctas; ++r) {
        const float2 v = reinterpret_cast<const float2*>(smem + Cfg::kKOff + Cfg::kPairBytes + r * Cfg::kPairKeys * 4)[t];
        sum = make_float2(__fadd_rn(sum.x, v.x), __fadd_rn(sum.y, v.y));
      }
      add_to_weights(args, b, bg, seq_kv, first * Cfg::kPairKeys + 2 * t, sum);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kSumWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

cudaError_t launch_weights_rows(const CUtensorMap& tq, const CUtensorMap& tk, WeightsArgs a, int max_keys, int sm_count, cudaStream_t s) {
  using Cfg = RowsCfg;
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kb_weights_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Cfg::kSmemBytes));
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const int pairs = (max_keys - 1) / Cfg::kPairKeys + 1;
  const int tiles = (kGroup * a.L + kTileRows - 1) / kTileRows;          // of rows: steps of a pair
  const long long units = static_cast<long long>(a.B) * a.Hkv * pairs;
  a.ctas = 1;
  a.splits = pairs;
  if (units <= sm_count) {
    // few pairs: a cluster each, while SMs are idle and a CTA keeps four steps
    while (a.ctas < 4 && units * a.ctas <= sm_count && tiles >= 8 * a.ctas) a.ctas *= 2;
  } else if (tiles < 64) {
    // short pairs: as many CTAs as are resident, so that a CTA's start (4 us, 7 steps) comes once
    const int per_cta = static_cast<int>((units + sm_count - 1) / sm_count);
    a.splits = (pairs + per_cta - 1) / per_cta;
  }
  const long long grid = static_cast<long long>(a.splits) * a.B * a.Hkv * a.ctas;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kb_weights_rows_kernel, tq, tk, a);
}

}  // namespace kb

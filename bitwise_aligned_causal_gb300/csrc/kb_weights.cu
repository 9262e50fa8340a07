// kb_weights.cu -- the attention weight that each cached key gets from a
// call's query rows: w_j += sum over rows i and heads h of 2^(s c - lse log2 e),
// s = q_i . k_j, c = log2(e) / sqrt(128), with the row's log-sum-exp given.
//
// A key tile is the A operand and a tile of query rows the B operand, so the
// product S^T = K Q^T has a key per TMEM lane: a thread sums its key's weights
// over the columns alone, without a shuffle.  Two warps share a key (columns
// 0..63 and 64..127 of a step); their sums meet once per key tile.
//   warp 0       TMA producer of the K ring (and of the Q ring)
//   warp 1       TMEM allocator + MMA issuer (one lane)
//   warp 2       per step: -lse log2(e) and the position of every column, in
//                shared memory (-inf and -1 for a column without a row)
//   warps 4..11  weights: warp w takes lanes 32 (w % 4) .. +31, column half (w - 4) / 4
// Each step's 128 x 64 exponentials per half are summed in fp32 before they
// join the key's running sum, so a sum over 65536 rows rounds some 500 times
// at its full size, not 65536.
//
// kPacked (at most 32 rows): the rows of a group's four heads are one B tile of
// 16 .. 128 columns that stays in shared memory while key tiles stream by: HBM
// bounds it.  Otherwise B tiles are 128 rows of one head, streamed (from L2)
// against each key tile: the exponentials bound it.  Two CTAs share an SM, so
// one's weights run while the other waits.
#include <algorithm>

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

struct WeightsCfg {
  static constexpr int kThreads = 12 * 32;
  static constexpr int kSumWarp0 = 4;
  static constexpr int kSumThreads = 256;
  static constexpr int kStages = 3;                       // tiles in the ring: K and Q tiles as they come (packed: K, one Q)
  static constexpr uint32_t kTmemCols = 256;              // two score buffers
  static constexpr uint32_t kRingOff = 0;
  static constexpr uint32_t kBarOff = kStages * kTileBytes;
  static constexpr int kBarKFull = 0;                     // per K slot
  static constexpr int kBarKEmpty = 2;
  static constexpr int kBarQFull = 4;                     // per Q slot
  static constexpr int kBarQEmpty = 6;
  static constexpr int kBarDFull = 8;                     // per score buffer
  static constexpr int kBarDEmpty = 10;                   // ... read by all of the weight threads
  static constexpr int kBarLFull = 12;                    // ... and its columns' log-sum-exps staged
  static constexpr int kBarDrain = 14;
  static constexpr int kNumBars = 15;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8 + 8;
  static constexpr uint32_t kColOff = kMiscOff + 16;      // float -lse log2 e x 128 x 2 buffers, then int position the same
  static constexpr uint32_t kPartOff = kColOff + 2 * 128 * 8;   // float x 128 x 2: the upper half's sums of a key tile
  static constexpr uint32_t kSmemUsed = kPartOff + 2 * 128 * 4;
  static constexpr uint32_t kSmemBytes = kSmemUsed + 1024;
};
static_assert(WeightsCfg::kColOff % 16 == 0, "columns are read in 16-byte words");
static_assert(2 * WeightsCfg::kSmemBytes <= 226u * 1024u, "two CTAs share an SM");

__device__ __forceinline__ void weights_drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 50000000ull) break;
}

// Weights of one key for 16 columns of a step: x scores, off -lse log2 e of the
// columns, pos their positions (kMasked: a column gives nothing to a key behind it).
template <bool kMasked>
__device__ __forceinline__ void sum16(const uint32_t (&x)[16], const float* off, const int* pos, int key, float2 (&sum)[2]) {
  const float c = score_scale_log2();
  const float2 c2 = make_float2(c, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(off)[i];
    const float2 a0 = __ffma2_rn(make_float2(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])), c2, make_float2(v.x, v.y));
    const float2 a1 = __ffma2_rn(make_float2(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])), c2, make_float2(v.z, v.w));
    float2 w0 = make_float2(ex2_approx(a0.x), ex2_approx(a0.y)), w1 = make_float2(ex2_approx(a1.x), ex2_approx(a1.y));
    if (kMasked) {
      const int4 p = reinterpret_cast<const int4*>(pos)[i];
      if (key > p.x) w0.x = 0.0f;
      if (key > p.y) w0.y = 0.0f;
      if (key > p.z) w1.x = 0.0f;
      if (key > p.w) w1.y = 0.0f;
    }
    sum[0] = __fadd2_rn(sum[0], w0);
    sum[1] = __fadd2_rn(sum[1], w1);
  }
}

}  // namespace

template <bool kPacked>
__global__ void __launch_bounds__(WeightsCfg::kThreads, 2)
kb_weights_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const WeightsArgs args) {
  using Cfg = WeightsCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return smem_addr(bars + i); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bg = static_cast<int>(blockIdx.x) % (args.B * args.Hkv);
  const int first = static_cast<int>(blockIdx.x) / (args.B * args.Hkv);   // key tiles first, first + splits, ...
  const int b = bg / args.Hkv, g = bg % args.Hkv;
  int pos0 = args.start, rows = args.L;
  if (args.starts != nullptr) {
    pos0 = args.starts[b];
    rows = args.lens[b];
    if (pos0 < 0 || rows < 0 || rows > args.L || pos0 > args.kv_cap - rows) {
      if (threadIdx.x == 0 && first == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
      return;
    }
  }
  const int seq_kv = pos0 + rows;
  const int n_kv = rows == 0 ? 0 : (seq_kv + kTileKeys - 1) / kTileKeys;
  if (first >= n_kv) return;

  // K tiles in two slots (packed) or one, Q tiles in one slot (packed) or two
  constexpr int kKSlots = kPacked ? 2 : 1, kQSlots = kPacked ? 1 : 2;
  const uint32_t k_ring = sbase + Cfg::kRingOff, q_ring = k_ring + kKSlots * kTileBytes;
  // packed: columns m = head * rows + row; N covers them in sixteens
  const int n_cols = kPacked ? (kGroup * rows + 15) / 16 * 16 : 128;
  const int q_tiles = kPacked ? 1 : (rows + kTileRows - 1) / kTileRows;
  // first query tile that sees key tile j (its steps: four heads from there on)
  auto first_tile = [&](int j) { return kPacked ? 0 : max(0, j * kTileKeys - pos0) / kTileRows; };
  auto steps_of = [&](int j) { return kPacked ? 1 : (q_tiles - first_tile(j)) * kGroup; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kNumBars; ++i) {
      uint32_t count = 1u;
      if (i >= Cfg::kBarDEmpty && i < Cfg::kBarDEmpty + 2) count = Cfg::kSumThreads;
      if (i >= Cfg::kBarLFull && i < Cfg::kBarLFull + 2) count = 32u;
      if (kPacked && i == Cfg::kBarQFull) count = Cfg::kSumThreads;
      mbar_init(bar(i), count);
    }
    misc[1] = (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) ? 1u : 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + Cfg::kMiscOff, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];
  const bool skip = *abort_flag != 0;

  if (warp == 0) {
    // ----------------------------------------------------------- producer
    if (lane == 0 && !skip) {
      tma_prefetch_desc(&tmap_k);
      if (!kPacked) tma_prefetch_desc(&tmap_q);
      int K = 0, T = 0;                                   // key tiles, steps
      bool ok = true;
      for (int j = first; j < n_kv && ok; j += args.splits) {
        int row = j * kTileKeys, plane = bg;
        if (args.block_table != nullptr) {
          int pg = args.block_table[static_cast<size_t>(b) * args.pages_per_seq + row / args.page_size];
          if (pg < 0 || pg >= args.num_pages) {
            atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
            pg = args.num_pages;                          // beyond the map: the TMA unit reads zeros
          }
          row = row % args.page_size;
          plane = pg * args.Hkv + g;
        }
        const int ks = K % kKSlots;
        if (K >= kKSlots) ok = mbar_wait(bar(Cfg::kBarKEmpty + ks), (K / kKSlots - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(Cfg::kBarKFull + ks), kTileBytes);
        tma_load_tile(k_ring + ks * kTileBytes, &tmap_k, row, plane, bar(Cfg::kBarKFull + ks));
        ++K;
        if constexpr (!kPacked) {
          const int t0 = first_tile(j), n = steps_of(j);
          for (int s = 0; s < n; ++s, ++T) {
            const int qs = T % kQSlots;
            if (T >= kQSlots) ok = mbar_wait(bar(Cfg::kBarQEmpty + qs), (T / kQSlots - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
            if (!ok) break;
            mbar_arrive_expect_tx(bar(Cfg::kBarQFull + qs), kTileBytes);
            tma_load_tile(q_ring + qs * kTileBytes, &tmap_q, (t0 + s / kGroup) * kTileRows,
                          b * args.Hkv * kGroup + g * kGroup + s % kGroup, bar(Cfg::kBarQFull + qs));
          }
        }
      }
      if (!ok) {
        for (int x = max(K - kKSlots, 0); x < K; ++x) weights_drain_wait(bar(Cfg::kBarKFull + x % kKSlots), (x / kKSlots) & 1);
        for (int x = max(T - kQSlots, 0); x < T; ++x) weights_drain_wait(bar(Cfg::kBarQFull + x % kQSlots), (x / kQSlots) & 1);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0 && !skip) {
      const uint32_t idesc = idesc_bf16_f32(128, static_cast<uint32_t>(n_cols), 0);
      int K = 0, T = 0;
      bool ok = true;
      for (int j = first; j < n_kv && ok; j += args.splits, ++K) {
        const int ks = K % kKSlots;
        ok = mbar_wait(bar(Cfg::kBarKFull + ks), (K / kKSlots) & 1, abort_flag, args.err, kDevTimeoutTma);
        const int n = steps_of(j);
        for (int s = 0; s < n && ok; ++s, ++T) {
          const int qs = kPacked ? 0 : T % kQSlots, db = T & 1;
          if (!kPacked || T == 0)
            ok = mbar_wait(bar(Cfg::kBarQFull + qs), kPacked ? 0 : (T / kQSlots) & 1, abort_flag, args.err, kDevTimeoutTma);
          if (ok && T >= 2) ok = mbar_wait(bar(Cfg::kBarDEmpty + db), (T / 2 - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem_base + db * 128u, desc_kmajor(k_ring + ks * kTileBytes, kk, 1024u, kSlabBytes),
                   desc_kmajor(q_ring + qs * kTileBytes, kk, 1024u, kSlabBytes), idesc, kk > 0 ? 1u : 0u);
          tc_commit(bar(Cfg::kBarDFull + db));
          if (!kPacked) tc_commit(bar(Cfg::kBarQEmpty + qs));
          if (s == n - 1) tc_commit(bar(Cfg::kBarKEmpty + ks));
        }
      }
      if (!ok) {
        tc_commit(bar(Cfg::kBarDrain));
        weights_drain_wait(bar(Cfg::kBarDrain), 0);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------- the columns' offsets
    if (!skip) {
      constexpr float kLog2e = 1.44269504088896341f;
      int T = 0;
      bool ok = true;
      for (int j = first; j < n_kv && ok; j += args.splits) {
        const int t0 = first_tile(j), n = steps_of(j);
        for (int s = 0; s < n && ok; ++s, ++T) {
          const int db = T & 1;
          // the rows' log-sum-exps are on their way while the buffer is waited for
          float l[4];
          int p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int col = 32 * i + lane;
            const int head = kPacked ? col / rows : s % kGroup;
            const int r = kPacked ? col % rows : (t0 + s / kGroup) * kTileRows + col;
            const bool used = kPacked ? head < kGroup : r < rows;
            p[i] = used ? pos0 + r : -1;
            l[i] = used ? __ldg(args.lse + (static_cast<size_t>(b) * args.Hkv * kGroup + g * kGroup + head) * args.L + r) : INFINITY;
          }
          if (T >= 2) {
            ok = mbar_wait(bar(Cfg::kBarDEmpty + db), (T / 2 - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          float* off = reinterpret_cast<float*>(smem + Cfg::kColOff) + db * 128;
          int* pos = reinterpret_cast<int*>(smem + Cfg::kColOff + 1024) + db * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {    // a row that saw nothing (-inf) has no weights to give
            off[32 * i + lane] = l[i] == -INFINITY ? -INFINITY : __fmul_rn(-l[i], kLog2e);
            pos[32 * i + lane] = p[i];
          }
          mbar_arrive(bar(Cfg::kBarLFull + db));
        }
      }
    }
  } else if (warp >= Cfg::kSumWarp0) {
    // ------------------------------------------------------------ weights
    const int st = static_cast<int>(threadIdx.x) - 32 * Cfg::kSumWarp0;
    if constexpr (kPacked) {
      // Q: column m = head * rows + row, zero behind, in the swizzled layout
      for (int idx = st; idx < n_cols * 16; idx += Cfg::kSumThreads) {
        const int m = idx >> 4, c = idx & 15;
        uint4 val = make_uint4(0u, 0u, 0u, 0u);
        if (m < kGroup * rows)
          val = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.q) +
                      ((static_cast<size_t>(b) * args.Hkv * kGroup + g * kGroup + m / rows) * args.L + m % rows) * kHeadDim) + c);
        *reinterpret_cast<uint4*>(smem + Cfg::kRingOff + kKSlots * kTileBytes + (c >> 3) * kSlabBytes + (m >> 3) * 1024 +
                                  (m & 7) * 128 + (((c & 7) ^ (m & 7)) << 4)) = val;
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(Cfg::kBarQFull));
    }
    const int half = (warp - Cfg::kSumWarp0) >> 2;
    const int key = 32 * (warp & 3) + lane;               // TMEM lane = key of the tile
    const uint32_t d_tmem = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const float* col_off = reinterpret_cast<const float*>(smem + Cfg::kColOff);
    const int* col_pos = reinterpret_cast<const int*>(smem + Cfg::kColOff + 1024);
    float* part = reinterpret_cast<float*>(smem + Cfg::kPartOff);
    int T = 0, K = 0;
    bool ok = !skip;
    for (int j = first; j < n_kv && ok; j += args.splits, ++K) {
      const int t0 = first_tile(j), n = steps_of(j);
      float total = 0.0f;
      for (int s = 0; s < n; ++s, ++T) {
        const int db = T & 1;
        ok = mbar_wait(bar(Cfg::kBarDFull + db), (T / 2) & 1, abort_flag, args.err, kDevTimeoutMma) &&
             mbar_wait(bar(Cfg::kBarLFull + db), (T / 2) & 1, abort_flag, args.err, kDevTimeoutSlot);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // does some row of the step not see some key of the tile, or has a column no row?
        const int r0 = kPacked ? 0 : (t0 + s / kGroup) * kTileRows;
        const bool masked = pos0 + r0 < j * kTileKeys + kTileKeys - 1 || (!kPacked && r0 + kTileRows > rows);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const int pkey = j * kTileKeys + key;
        const uint32_t d = d_tmem + db * 128u + 64u * half;
        const float* off = col_off + db * 128 + 64 * half;
        const int* pos = col_pos + db * 128 + 64 * half;
        if constexpr (kPacked) {
#pragma unroll 1
          for (int c = 0; c < n_cols - 64 * half && c < 64; c += 16) {
            uint32_t x[16];
            tmem_ld16_wait(d + c, x);
            if (masked) sum16<true>(x, off + c, pos + c, pkey, sum);
            else sum16<false>(x, off + c, pos + c, pkey, sum);
          }
        } else {
          // the load of the next 16 columns is in flight while 16 are summed
          uint32_t x[16], y[16];
          tmem_ld16_issue(d, x);
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            tmem_ld16_wait_for(x);
            tmem_ld16_issue(d + c + 16, y);
            if (masked) sum16<true>(x, off + c, pos + c, pkey, sum);
            else sum16<false>(x, off + c, pos + c, pkey, sum);
            tmem_ld16_wait_for(y);
            if (c + 32 < 64) tmem_ld16_issue(d + c + 32, x);
            if (masked) sum16<true>(y, off + c + 16, pos + c + 16, pkey, sum);
            else sum16<false>(y, off + c + 16, pos + c + 16, pkey, sum);
          }
        }
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarDEmpty + db));
        total = __fadd_rn(total, __fadd_rn(__fadd_rn(sum[0].x, sum[0].y), __fadd_rn(sum[1].x, sum[1].y)));
      }
      if (half == 1) part[(K & 1) * 128 + key] = total;
      // one decision for the eight warps: all go on, or none does
      if (named_bar_or(1, Cfg::kSumThreads, !ok)) break;
      if (half == 0) {
        const int p = j * kTileKeys + key;
        bool known = true;                                // the tile's page is in the pool
        if (args.block_table != nullptr) {
          const int pg = __ldg(args.block_table + static_cast<size_t>(b) * args.pages_per_seq + j * kTileKeys / args.page_size);
          known = pg >= 0 && pg < args.num_pages;
        }
        if (known && p < seq_kv) {
          float* w = args.weights + static_cast<size_t>(bg) * args.kv_cap + p;
          *w = __fadd_rn(*w, __fadd_rn(total, part[(K & 1) * 128 + key]));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

template <bool kPacked>
static cudaError_t launch_weights_t(const CUtensorMap& tq, const CUtensorMap& tk, const WeightsArgs& a, cudaStream_t s) {
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kb_weights_kernel<kPacked>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(WeightsCfg::kSmemBytes));
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const long long grid = static_cast<long long>(a.splits) * a.B * a.Hkv;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  kb_weights_kernel<kPacked><<<static_cast<unsigned>(grid), WeightsCfg::kThreads, WeightsCfg::kSmemBytes, s>>>(tq, tk, a);
  return cudaGetLastError();
}

cudaError_t launch_weights(const CUtensorMap& tq, const CUtensorMap& tk, WeightsArgs a, int max_keys, int sm_count,
                           cudaStream_t s) {
  const int tiles = (max_keys + kTileKeys - 1) / kTileKeys;
  const int units = a.B * a.Hkv;
  if (a.L <= kMaxPackedRows) {
    // four key tiles a CTA at least, four waves of two CTAs per SM at most
    a.splits = std::max(1, std::min((tiles + 3) / 4, (8 * sm_count + units - 1) / units));
    return launch_weights_t<true>(tq, tk, a, s);
  }
  // at least 32 steps a CTA, so that its start is a small part of it
  const int steps = kGroup * ((a.L + kTileRows - 1) / kTileRows);
  const int per_cta = std::max(1, 32 / steps);
  a.splits = (tiles + per_cta - 1) / per_cta;
  return launch_weights_t<false>(tq, tk, a, s);
}

}  // namespace kb

// kb_weights.cu -- the attention weight that each cached key gets from a few
// query rows (at most 32; kb_weights_rows.cu: more): w_j += sum over rows i and
// heads h of 2^(s c - lse log2 e), s = q_i . k_j, c = log2(e) / sqrt(128), with
// the row's log-sum-exp given.
//
// A key tile is the A operand and the rows of a group's four heads, 16 .. 128
// of them, the B operand, which stays in shared memory while key tiles stream
// by: HBM bounds it.  S^T = K Q^T has a key per TMEM lane, so a thread sums its
// key's weights over the columns alone, without a shuffle.  Two warps share a
// key (columns 0..63 and 64..127); their sums meet once per key tile.
//   warp 0       TMA producer of the K ring
//   warp 1       TMEM allocator + MMA issuer (one lane)
//   warps 3..10  weights: warp w takes lanes 32 (w % 4) .. +31, column half (w - 3) / 4
// Three CTAs share an SM (two, with more than eight rows): one's tiles are on
// their way while another starts or sums.  More tiles in flight per CTA cost
// more than they gave (two CTAs with two slots 105 us, with three 110).
// Measured (one row of 16 conversations of 16K): 95 us, 5.8 TB/s, 86% of a
// plain copy's rate.
#include <algorithm>

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

struct WeightsCfg {
  static constexpr int kThreads = 11 * 32;
  static constexpr int kSumWarp0 = 3;
  static constexpr int kSumThreads = 256;
  static constexpr int kSlots = 2;                        // K tiles in flight
  static constexpr uint32_t kBarOff = kSlots * kTileBytes;
  static constexpr int kBarKFull = 0;                     // per K slot
  static constexpr int kBarKEmpty = kBarKFull + kSlots;
  static constexpr int kBarQFull = kBarKEmpty + kSlots;
  static constexpr int kBarDFull = kBarQFull + 1;         // per score buffer
  static constexpr int kBarDEmpty = kBarDFull + 2;        // ... read by all of the weight threads
  static constexpr int kBarDrain = kBarDEmpty + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr uint32_t kMiscOff = kBarOff + (kNumBars + 1) / 2 * 16;
  static constexpr uint32_t kColOff = kMiscOff + 16;      // float -lse log2 e x 128, then int position the same
  static constexpr uint32_t kPartOff = kColOff + 128 * 8;       // float x 128 x 2: the upper half's sums of a key tile
  static constexpr uint32_t kQOff = (kPartOff + 2 * 128 * 4 + 1023) / 1024 * 1024;      // the columns' queries, 256 bytes each
  // columns of a call's MMA (its TMEM allocation holds two score buffers of 64 or of 128)
  static constexpr int cols(int rows) { return (kGroup * rows + 15) / 16 * 16; }
  static constexpr uint32_t smem_bytes(int rows) { return kQOff + static_cast<uint32_t>(cols(rows)) * kHeadDim * 2; }
};
static_assert(WeightsCfg::kColOff % 16 == 0, "columns are read in 16-byte words");
static_assert(2 * (WeightsCfg::smem_bytes(kMaxPackedRows) + 1024) <= 228u * 1024u, "two CTAs share an SM");
static_assert(3 * (WeightsCfg::smem_bytes(8) + 1024) <= 228u * 1024u, "three, with up to eight rows");

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

__global__ void __launch_bounds__(WeightsCfg::kThreads, 3)
kb_weights_kernel(const __grid_constant__ CUtensorMap tmap_k, const WeightsArgs args) {
  using Cfg = WeightsCfg;
  extern __shared__ __align__(1024) uint8_t smem[];
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
  const int n_kv = rows == 0 ? 0 : (seq_kv - 1) / kTileKeys + 1;
  if (first >= n_kv) return;

  // columns m = head * rows + row of the MMA, in sixteens
  constexpr int slots = Cfg::kSlots;
  const int n_cols = Cfg::cols(rows);
  const uint32_t q_slab = n_cols * 128u;
  const uint32_t d_cols = args.L <= 16 ? 64u : 128u;      // of a score buffer

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kNumBars; ++i) {
      uint32_t count = 1u;
      if (i == Cfg::kBarQFull || (i >= Cfg::kBarDEmpty && i < Cfg::kBarDEmpty + 2)) count = Cfg::kSumThreads;
      mbar_init(bar(i), count);
    }
    if (sbase % 1024u != 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));    // (the swizzle's unit; never so)
    misc[1] = (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) ? 1u : 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + Cfg::kMiscOff, 2 * d_cols);
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
      int K = 0, st = 0;
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
        if (K >= slots) ok = mbar_wait(bar(Cfg::kBarKEmpty + st), (K / slots - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(Cfg::kBarKFull + st), kTileBytes);
        tma_load_tile(sbase + st * kTileBytes, &tmap_k, row, plane, bar(Cfg::kBarKFull + st));
        ++K;
        if (++st == slots) st = 0;
      }
      if (!ok)
        for (int x = max(K - slots, 0); x < K; ++x) weights_drain_wait(bar(Cfg::kBarKFull + x % slots), (x / slots) & 1);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0 && !skip) {
      const uint32_t idesc = idesc_bf16_f32(128, static_cast<uint32_t>(n_cols), 0);
      int K = 0;
      bool ok = mbar_wait(bar(Cfg::kBarQFull), 0, abort_flag, args.err, kDevTimeoutTma);
      for (int j = first; j < n_kv && ok; j += args.splits, ++K) {
        const int st = K % slots, db = K & 1;
        ok = mbar_wait(bar(Cfg::kBarKFull + st), (K / slots) & 1, abort_flag, args.err, kDevTimeoutTma);
        if (ok && K >= 2) ok = mbar_wait(bar(Cfg::kBarDEmpty + db), (K / 2 - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tmem_base + db * d_cols, desc_kmajor(sbase + st * kTileBytes, kk, 1024u, kSlabBytes),
                 desc_kmajor(sbase + Cfg::kQOff, kk, 1024u, q_slab), idesc, kk > 0 ? 1u : 0u);
        tc_commit(bar(Cfg::kBarDFull + db));
        tc_commit(bar(Cfg::kBarKEmpty + st));
      }
      if (!ok) {
        tc_commit(bar(Cfg::kBarDrain));
        weights_drain_wait(bar(Cfg::kBarDrain), 0);
      }
    }
  } else if (warp >= Cfg::kSumWarp0) {
    // ------------------------------------------------------------ weights
    const int st = static_cast<int>(threadIdx.x) - 32 * Cfg::kSumWarp0;
    bool some_off;                                        // some column's row gives nothing
    {
      // Q, zero behind its columns, in the swizzled layout; the columns' offsets and positions
      for (int idx = st; idx < n_cols * 16; idx += Cfg::kSumThreads) {
        const int m = idx >> 4, c = idx & 15;
        uint4 val = make_uint4(0u, 0u, 0u, 0u);
        if (m < kGroup * rows)
          val = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.q) +
                      ((static_cast<size_t>(b) * args.Hkv * kGroup + g * kGroup + m / rows) * args.L + m % rows) * kHeadDim) + c);
        *reinterpret_cast<uint4*>(smem + Cfg::kQOff + (c >> 3) * q_slab + (m >> 3) * 1024 + (m & 7) * 128 + (((c & 7) ^ (m & 7)) << 4)) = val;
      }
      constexpr float kLog2e = 1.44269504088896341f;
      bool off_row = false;
      if (st < 128) {
        const bool used = st < kGroup * rows;
        const float l = used ? __ldg(args.lse + (static_cast<size_t>(bg) * kGroup + st / rows) * args.L + st % rows) : INFINITY;
        // A row of an infinite log-sum-exp has no weights to give, whatever stands
        // in q: it sees no key (its scores times the scale, minus infinity, could
        // be NaN).
        off_row = used && isinf(l);
        reinterpret_cast<float*>(smem + Cfg::kColOff)[st] = isinf(l) ? -INFINITY : __fmul_rn(-l, kLog2e);
        reinterpret_cast<int*>(smem + Cfg::kColOff + 512)[st] = used && !off_row ? pos0 + st % rows : -1;
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(Cfg::kBarQFull));
      some_off = named_bar_or(1, Cfg::kSumThreads, off_row);
    }
    const int half = (warp - Cfg::kSumWarp0) >> 2;
    const int key = 32 * (warp & 3) + lane;               // TMEM lane = key of the tile
    const uint32_t d_tmem = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const float* off = reinterpret_cast<const float*>(smem + Cfg::kColOff) + 64 * half;
    const int* pos = reinterpret_cast<const int*>(smem + Cfg::kColOff + 512) + 64 * half;
    float* part = reinterpret_cast<float*>(smem + Cfg::kPartOff);
    int K = 0;
    bool ok = !skip;
    for (int j = first; j < n_kv && ok; j += args.splits, ++K) {
      const int db = K & 1;
      float total = 0.0f;
      ok = mbar_wait(bar(Cfg::kBarDFull + db), (K / 2) & 1, abort_flag, args.err, kDevTimeoutMma);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        // some row does not see some key of the tile, or a column has no row (its zeros times an infinite key are NaN)
        const bool masked = pos0 < j * kTileKeys + kTileKeys - 1 || n_cols > kGroup * rows || some_off;
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const int pkey = j * kTileKeys + key;
        const uint32_t d = d_tmem + db * d_cols + 64u * half;
#pragma unroll 1
        for (int c = 0; c < n_cols - 64 * half && c < 64; c += 16) {
          uint32_t x[16];
          tmem_ld16_wait(d + c, x);
          if (masked) sum16<true>(x, off + c, pos + c, pkey, sum);
          else sum16<false>(x, off + c, pos + c, pkey, sum);
        }
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarDEmpty + db));
        total = __fadd_rn(__fadd_rn(sum[0].x, sum[0].y), __fadd_rn(sum[1].x, sum[1].y));
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
    tmem_dealloc(tmem_base, 2 * d_cols);
  }
}

cudaError_t launch_weights(const CUtensorMap& tk, WeightsArgs a, int max_keys, int sm_count, cudaStream_t s) {
  using Cfg = WeightsCfg;
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kb_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(Cfg::smem_bytes(kMaxPackedRows)));
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  // four key tiles a CTA at least, four waves at most (one: 107 us in the case above)
  const int tiles = (max_keys - 1) / kTileKeys + 1;
  const int units = a.B * a.Hkv;
  const int resident = (a.L <= 8 ? 3 : 2) * sm_count;
  a.splits = std::max(1, std::min((tiles + 3) / 4, (4 * resident + units - 1) / units));
  const long long grid = static_cast<long long>(a.splits) * units;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  kb_weights_kernel<<<static_cast<unsigned>(grid), Cfg::kThreads, Cfg::smem_bytes(a.L), s>>>(tk, a);
  return cudaGetLastError();
}

}  // namespace kb

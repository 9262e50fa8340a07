// kb_decode8.cu -- new tokens (one or two query rows) over a KV cache held in 8
// bits (kb_cache8.cuh).
//
// The packed kernel (kb_decode.cu) spends a 128-row MMA on four query rows and
// reads every operand from shared memory, which an 8-bit cache makes the bound:
// bytes in, bytes out, bf16 values in and out again.  Here the two products are
// transposed: keys and channels take the MMA's 128 rows, the query rows its 16
// columns,
//   S^T = K Q^T,   O^T += V^T P^T,
// and K's values go from registers to tensor memory, not to shared memory.
// A tensor core sums the 16 products of a step, and the steps, in the same
// order whichever operand holds which rows, so S and O have the contract's
// bits (C2); the row math is the contract's (C3-C5) on S brought back to rows
// through shared memory.  Per pair of key tiles that leaves 136 KB through
// shared memory instead of 224, and an eighth of the tensor core's time.
//
//   warps 0..3    S^T from tensor memory to rows in shared memory; between
//                 tiles, as they fall due: scaling O where a row's maximum
//                 moved, folding a finished segment (C5), the epilogue.  A lane
//                 is a key of S^T and a channel of O^T
//   warps 4..7    K: bytes (staged by TMA) -> bf16 -> tensor memory
//   warps 8..11   V: bytes (staged by TMA) -> bf16 -> shared memory
//   warp 12       TMEM allocator + S^T issuer      warp 13   O^T issuer
//   warp 14       softmax, two tiles at a time
//   warp 15       producer: the tiles' pages and exponents, 32 tiles ahead, and
//                 TMA of the bytes
// Tensor memory: three K tiles of 64 columns, four S^T and O^T of 16.
//
// A CTA runs a contiguous block of the row's segments: all of them, folded
// here; or (args.cluster CTAs, a segment each) one, folded through the first
// CTA's shared memory; or (args.split CTAs) its share, whose partials go to the
// workspace; or
// (flat) a run of all KV heads' segments, piece by piece, so that every SM has
// as many as the others.
//
// Measured (B = 32, contexts of 16K): 244 us, 4.4 TB/s of bytes, against 332 in
// the packed kernel's shape and 258 with a CTA per KV head (256 of them); one
// conversation of 64K: 43 us with its segments over 128 CTAs.  What bounds it is the four schedulers: 1200 instructions
// each per pair of tiles, half of them the conversion's, on an ALU pipe that
// takes one every other cycle; HBM would allow 172 us.  Next come the
// instruction caches that sixteen warps of seven roles share: what is rare is
// out of line (timeouts, drains, odd tiles: 284 to 258 us with a CTA per head), and the conversion
// loops hold two chunks (one: 297 us; four: 261; eight: 309).  Eight warps for
// K and for V, one loop for both (279 us) and the shift on the FMA pipe were no
// better.
#include "kb_bytes.cuh"
#include "kb_cache8.cuh"
#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

struct Decode8Cfg {
  static constexpr int kRows = 8;                         // packed rows
  static constexpr int kN = 16;                           // columns of both products
  static constexpr int kConvWarps = 4;                    // of K, and of V
  static constexpr int kKWarp0 = 4, kVWarp0 = kKWarp0 + kConvWarps, kQkWarp = kVWarp0 + kConvWarps, kPvWarp = kQkWarp + 1;
  static constexpr int kSoftmaxWarp = kPvWarp + 1, kProdWarp = kSoftmaxWarp + 1;
  static constexpr int kThreads = (kProdWarp + 1) * 32;
  static constexpr int kKBytes = 3, kVBytes = 3;          // staged tiles of bytes
  static constexpr int kKBufs = 3;                        // K tiles in tensor memory
  static constexpr int kSBufs = 4;                        // S^T in tensor memory
  static constexpr int kXBufs = 4;                        // S in shared memory
  static constexpr int kPvBufs = 3;                       // V tiles and P in shared memory
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kKCol = 0, kSCol = kKBufs * 64, kOCol = kSCol + kSBufs * kN;
  static_assert(kOCol + kN <= kTmemCols, "tensor memory");
  static constexpr uint32_t kByteTile = kTileBytes / 2;
  static constexpr int kXStride = kTileKeys + 8;          // floats of a row of S: the lanes of a softmax warp fall on all banks
  static constexpr uint32_t kQSlab = kN * 128;            // one 64-column slab of Q or P
  static constexpr uint32_t kVOff = 0;
  static constexpr uint32_t kKByteOff = kVOff + kPvBufs * kTileBytes;
  static constexpr uint32_t kVByteOff = kKByteOff + kKBytes * kByteTile;
  static constexpr uint32_t kQOff = kVByteOff + kVBytes * kByteTile;
  static constexpr uint32_t kPOff = kQOff + 2 * kQSlab;
  static constexpr uint32_t kXOff = kPOff + kPvBufs * 2 * kQSlab;
  static constexpr uint32_t kStatsOff = kXOff + kXBufs * kRows * kXStride * 4;    // float2 (m, l) per row, two segments
  static constexpr uint32_t kAlphaOff = kStatsOff + 2 * kRows * 8;                // float per row
  static constexpr uint32_t kAskOff = kAlphaOff + kRows * 4;                      // int2: scalings asked for, the tile of the last
  static constexpr uint32_t kExpOff = kAskOff + 8;                // int per staged tile: its exponent
  static constexpr uint32_t kBarOff = (kExpOff + (kKBytes + kVBytes) * 4 + 15) & ~15u;
  static constexpr int kBarKByte = 0;
  static constexpr int kBarVByte = kBarKByte + kKBytes;
  static constexpr int kBarByteRead = kBarVByte + kVBytes;        // 4 warps: a staged tile has been read (K's, then V's)
  static constexpr int kBarKFull = kBarByteRead + kKBytes + kVBytes;   // 128: a K tile is in tensor memory
  static constexpr int kBarKEmpty = kBarKFull + kKBufs;   // its product is done
  static constexpr int kBarSFull = kBarKEmpty + kKBufs;
  static constexpr int kBarSEmpty = kBarSFull + kSBufs;   // 128
  static constexpr int kBarXFull = kBarSEmpty + kSBufs;   // 128
  static constexpr int kBarXEmpty = kBarXFull + kXBufs;   // softmax threads
  static constexpr int kBarVFull = kBarXEmpty + kXBufs;   // 128
  static constexpr int kBarPFull = kBarVFull + kPvBufs;   // softmax threads
  static constexpr int kBarPvDone = kBarPFull + kPvBufs;  // O^T holds the tile; its V and P may be replaced
  static constexpr int kBarORead = kBarPvDone + kPvBufs;  // 128: a finished segment's O^T has been read
  static constexpr int kBarStFull = kBarORead + 1;        // softmax threads, 2: a finished segment's (m, l) written ...
  static constexpr int kBarStEmpty = kBarStFull + 2;      // 128, 2: ... and read
  static constexpr int kBarScaled = kBarStEmpty + 2;      // 128: O^T scaled as asked
  static constexpr int kBarQReady = kBarScaled + 1;   // 128: Q (and zeros behind P's rows) written
  static constexpr int kBarDrain = kBarQReady + 1;        // 2: one per issuer
  static constexpr int kNumBars = kBarDrain + 2;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemUsed = kMiscOff + 16;
  static constexpr uint32_t kSmemBytes = kSmemUsed + 1024;
  static_assert(kSmemBytes <= 227u * 1024u, "shared memory budget");
};

constexpr int kPasses = 8;                                // 16-byte chunks of a tile's bytes per conversion thread
constexpr int kVStep = 16 * kHeadDim;                     // V, from a thread's row to its next: bytes staged, and of a slab

// A tile that ends the sequence (n of its rows lie in it; values past them are
// zero, whatever the block's mark) or whose values reach beyond 448 * 2^7, out
// of the way of the loops for whole ones.
__device__ __forceinline__ void odd16(const uint4& w, const Scale8& sc, bool live, uint4& lo, uint4& hi) {
  values8x16(w, sc.first, lo, hi);
  lo = scaled_again(lo, sc.second);
  hi = scaled_again(hi, sc.second);
  if (!live) lo = hi = make_uint4(0u, 0u, 0u, 0u);
}
__device__ __noinline__ void odd_values(const uint8_t* src, uint8_t* dst, int next_chunk, int row0, int n, Scale8 sc) {
#pragma unroll 1
  for (int i = 0; i < kPasses; ++i) {
    uint4 lo, hi;
    odd16(*reinterpret_cast<const uint4*>(src + i * kVStep), sc, row0 + kVStep / kHeadDim * i < n, lo, hi);
    *reinterpret_cast<uint4*>(dst + i * kVStep) = lo;
    *reinterpret_cast<uint4*>(dst + i * kVStep + next_chunk) = hi;
  }
}
__device__ __noinline__ void odd_keys(const uint8_t* src, uint32_t dst, int row, int n, Scale8 sc) {
#pragma unroll 1
  for (int i = 0; i < kPasses; ++i) {
    uint4 lo, hi;
    odd16(*reinterpret_cast<const uint4*>(src + ((i ^ (row & 7)) << 4)), sc, row < n, lo, hi);
    tmem_st8(dst + i * 8u, lo, hi);
  }
}

}  // namespace

// kFlat: the CTAs share all segments of the call; kCluster: a cluster shares a
// KV head's.  (Kernels of their own: either's code in the others' costs them 1 us.)
template <bool kFlat, bool kCluster>
__global__ void __launch_bounds__(Decode8Cfg::kThreads, 1)
kb_decode8_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const PackedArgs args) {
  using Cfg = Decode8Cfg;
  constexpr int kRows = Cfg::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return smem_addr(bars + i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = args.B * args.Hkv;
  const int split = kCluster ? args.cluster : args.part != nullptr && !kFlat ? args.split : 1;

  // Sequence b: the position of its query row 0 and its rows; false (reported
  // by the CTAs that it concerns) for a length out of range.
  auto rows_of = [&](int b, int& pos0, int& rows) {
    pos0 = args.start;
    rows = args.L;
    bool ok = true;
    if (args.ctx_lens != nullptr) {
      const int ctx = __ldg(args.ctx_lens + b);
      ok = ctx >= args.L && ctx <= args.max_ctx;
      pos0 = ctx - args.L;
    }
    if (args.starts != nullptr) {
      pos0 = __ldg(args.starts + b);
      rows = __ldg(args.lens + b);
      ok = pos0 >= 0 && rows >= 0 && rows <= args.L && pos0 <= args.max_ctx - rows;
    }
    if (!ok) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
    return ok;
  };
  // flat (one row a sequence): all segments of all KV heads in a row, cut into
  // as many runs as there are CTAs
  auto segments = [&](int b) {
    int pos0, rows;
    return b < args.B && rows_of(b, pos0, rows) && rows > 0 ? (pos0 / kTileKeys + kSegTiles) / kSegTiles : 0;
  };
  int f = 0, f_end = 1;                                   // this CTA's run (else: one piece)
  if constexpr (kFlat) {
    int total = 0;
    for (int b0 = 0; b0 < args.B; b0 += 32)
      total += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(segments(b0 + lane))));
    const long long all = static_cast<long long>(total) * args.Hkv;
    f = static_cast<int>(all * blockIdx.x / gridDim.x);
    f_end = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x);
  }
  bool begun = false;                                     // barriers and TMEM are there
  do {
    if (f >= f_end) break;
    int rank = 0, sub = 0, b = 0, g = 0, g0 = 0, g1 = 0;
    int pos0, rows;
    if constexpr (kFlat) {
      int before = 0;                                       // segments of a KV head in the sequences before
      for (int b0 = 0; b0 < args.B; b0 += 32) {
        const int ns = segments(b0 + lane);
        int incl = ns;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (before + incl) * args.Hkv > f);
        if (past != 0) {
          const int at = __ffs(static_cast<int>(past)) - 1;
          const int ns_b = __shfl_sync(0xffffffffu, ns, at);
          const int rest = f - (before + __shfl_sync(0xffffffffu, incl, at) - ns_b) * args.Hkv;
          b = b0 + at;
          g = rest / ns_b;
          g0 = rest % ns_b;
          g1 = min(ns_b, g0 + f_end - f);
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (g1 <= g0) break;                                // (lengths that changed meanwhile)
      rows_of(b, pos0, rows);
      f += g1 - g0;
    } else {
      // (sub-chunk 0 first; a cluster's CTAs are neighbours)
      const int cta = static_cast<int>(blockIdx.x) / (kCluster ? split : 1);
      rank = kCluster ? static_cast<int>(blockIdx.x) % split : cta / bh % split;
      sub = kCluster ? 0 : cta / (bh * split);
      b = cta % bh / args.Hkv;
      g = cta % args.Hkv;
      f = f_end;
      if (!rows_of(b, pos0, rows)) return;
    }
    const int seq_kv = pos0 + rows;
    // the sub-chunk's rows [r0, r1), as in the packed kernel
    const int cut = min(rows, (pos0 / kTileKeys + 1) * kTileKeys - pos0);   // rows before the first tile boundary
    const int r0 = sub == 0 ? 0 : cut, r1 = sub == 0 ? cut : rows;
    const int Lc = r1 - r0;
    if (Lc <= 0) return;                                    // no rows, or the chunk does not reach a second tile
    const int n_rows = kGroup * Lc;
    const int n_kv = (pos0 + r1 - 1) / kTileKeys + 1;       // C1
    if constexpr (!kFlat) {
      // this CTA's segments (ceil(rank ns / split) ..)
      const int ns = (n_kv + kSegTiles - 1) / kSegTiles;
      g0 = (rank * ns + split - 1) / split;
      g1 = ((rank + 1) * ns + split - 1) / split;
      if (g0 >= g1 && !kCluster) return;                    // (a cluster's CTA stays for its barriers)
    }
    const int j0 = g0 * kSegTiles, nt = max(min(n_kv, g1 * kSegTiles) - j0, 0);

    if (threadIdx.x == 0) {
      for (int i = 0; i < Cfg::kNumBars; ++i) {
        uint32_t count = 1u;
        if ((i >= Cfg::kBarSEmpty && i < Cfg::kBarXEmpty) || i == Cfg::kBarORead || (i >= Cfg::kBarStEmpty && i <= Cfg::kBarQReady))
          count = 128u;
        if ((i >= Cfg::kBarKFull && i < Cfg::kBarKEmpty) || (i >= Cfg::kBarVFull && i < Cfg::kBarPFull)) count = 32u * Cfg::kConvWarps;
        if (i >= Cfg::kBarByteRead && i < Cfg::kBarKFull) count = static_cast<uint32_t>(Cfg::kConvWarps);
        if ((i >= Cfg::kBarXEmpty && i < Cfg::kBarVFull) || (i >= Cfg::kBarPFull && i < Cfg::kBarPvDone) ||
            (i >= Cfg::kBarStFull && i < Cfg::kBarStEmpty))
          count = 32u;
        if (begun) mbar_inval(bar(i));
        mbar_init(bar(i), count);
      }
      if (!begun) misc[1] = (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) ? 1u : 0u;
      reinterpret_cast<volatile int2*>(smem + Cfg::kAskOff)->x = 0;
      fence_mbar_init();
    }
    if (warp == Cfg::kQkWarp && !begun) {
      tmem_alloc(sbase + Cfg::kMiscOff, Cfg::kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    begun = true;
    const uint32_t tmem_base = misc[0];
    const bool skip = *abort_flag != 0;

    if (warp < 4) {
      // ------------------------------------------- S to rows, O^T's upkeep
      {
        // Q: packed row m = head * Lc + row, zeros behind, in the swizzled layout; zeros behind P's rows
        for (int idx = threadIdx.x; idx < Cfg::kN * 16; idx += 128) {
          const int m = idx >> 4, c = idx & 15;
          uint4 val = make_uint4(0u, 0u, 0u, 0u);
          if (m < n_rows)
            val = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.q) +
                        ((static_cast<size_t>(b) * args.Hq + g * kGroup + m / Lc) * args.L + r0 + m % Lc) * kHeadDim) + c);
          const uint32_t at = (c >> 3) * Cfg::kQSlab + (m >> 3) * 1024 + (m & 7) * 128 + (((c & 7) ^ (m & 7)) << 4);
          *reinterpret_cast<uint4*>(smem + Cfg::kQOff + at) = val;
          if (m >= kRows)
            for (int i = 0; i < Cfg::kPvBufs; ++i)
              *reinterpret_cast<uint4*>(smem + Cfg::kPOff + i * 2 * Cfg::kQSlab + at) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(Cfg::kBarQReady));
      }
      const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
      const int me = 32 * warp + lane;                      // key of a tile, channel of O
      const uint32_t o_tmem = tmem_base + Cfg::kOCol + lane_off;
      const float c_log2 = score_scale_log2();
      const volatile int2* ask = reinterpret_cast<const volatile int2*>(smem + Cfg::kAskOff);
      const float* alphas = reinterpret_cast<const float*>(smem + Cfg::kAlphaOff);
      int answered = 0;
      RowState acc = row_state_init();                      // lane r: row r of the folded segments
      float acc_o[kRows];                                   // channel `me` of every row
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc_o[i] = 0.0f;
      int G = 0;                                            // segments folded
      const int n_seg = g1 - g0;
      // One loop looks at everything that can fall due, in turn, and waits for
      // nothing by itself, so no two of them can hold each other up.  (One copy of
      // each step, too: with the steps repeated at every wait the warps' code no
      // longer fitted the instruction cache, 2.4 us a tile.)
      int j = 0;                                            // next tile
      bool ok = !skip;
      uint64_t t0 = global_timer_ns();
#pragma unroll 1
      while (ok && (j < nt || G < n_seg)) {
        bool moved = false;
        if (j < nt) {
          const int sb = j % Cfg::kSBufs, xb = j % Cfg::kXBufs;
          const bool due = mbar_try_wait_hint(bar(Cfg::kBarSFull + sb), (j / Cfg::kSBufs) & 1, 20u) &&
                           (j < Cfg::kXBufs || mbar_test_wait(bar(Cfg::kBarXEmpty + xb), (j / Cfg::kXBufs - 1) & 1));
          if (__all_sync(0xffffffffu, due)) {
            tc_fence_after();
            uint32_t s[Cfg::kN];
            tmem_ld16_wait(tmem_base + Cfg::kSCol + sb * Cfg::kN + lane_off, s);
            tc_fence_before();
            mbar_arrive(bar(Cfg::kBarSEmpty + sb));
            uint32_t* x = reinterpret_cast<uint32_t*>(smem + Cfg::kXOff) + xb * kRows * Cfg::kXStride + me;
#pragma unroll
            for (int i = 0; i < kRows; ++i) x[i * Cfg::kXStride] = s[i];
            mbar_arrive(bar(Cfg::kBarXFull + xb));
            ++j;
            moved = true;
          }
        }
        if (G < n_seg && j > min(nt, (G + 1) * kSegTiles) - 1) {
          const int t_last = min(nt, (G + 1) * kSegTiles) - 1;
          // (the phase of t_last's barrier stays until this segment is read: the next product waits for that)
          const bool due = mbar_test_wait(bar(Cfg::kBarStFull + (G & 1)), (G >> 1) & 1) &&
                           mbar_test_wait(bar(Cfg::kBarPvDone + t_last % Cfg::kPvBufs), (t_last / Cfg::kPvBufs) & 1);
          if (__all_sync(0xffffffffu, due)) {
            tc_fence_after();
            uint32_t o[Cfg::kN];
            tmem_ld16_wait(o_tmem, o);
            tc_fence_before();
            mbar_arrive(bar(Cfg::kBarORead));
            const float2 sv = lane < kRows ? reinterpret_cast<const float2*>(smem + Cfg::kStatsOff)[(G & 1) * kRows + lane]
                                           : make_float2(-INFINITY, 0.0f);
            mbar_arrive(bar(Cfg::kBarStEmpty + (G & 1)));
            const RowState sg{sv.x, __fmul_rn(sv.x, c_log2), sv.y};
            if (args.part != nullptr) {
              // the segment's partial, for the fold of all CTAs' segments
#pragma unroll
              for (int i = 0; i < kRows; ++i)
                if (i < n_rows)
                  args.part[(((static_cast<size_t>(b) * args.Hq + g * kGroup + i / Lc) * args.L + r0 + i % Lc) * args.n_seg + g0 + G) *
                                kPartFloats + me] = __uint_as_float(o[i]);
              if (warp == 0 && lane < n_rows)
                *reinterpret_cast<float4*>(
                    args.part + (((static_cast<size_t>(b) * args.Hq + g * kGroup + lane / Lc) * args.L + r0 + lane % Lc) * args.n_seg +
                                 g0 + G) * kPartFloats + kHeadDim) = make_float4(sg.m, sg.mc, sg.l, 0.0f);
            } else if (G == 0) {
              acc = sg;
#pragma unroll
              for (int i = 0; i < kRows; ++i) acc_o[i] = __uint_as_float(o[i]);
            } else {
              const FoldScale f = fold_state(acc, sg);
#pragma unroll
              for (int i = 0; i < kRows; ++i)
                acc_o[i] = fold_o(acc_o[i], __uint_as_float(o[i]),
                                  FoldScale{__shfl_sync(0xffffffffu, f.a, i), __shfl_sync(0xffffffffu, f.b, i)});
            }
            ++G;
            moved = true;
          }
        }
        const int asked = __shfl_sync(0xffffffffu, lane == 0 ? ask->x : 0, 0);
        if (asked != answered) {
          __threadfence_block();
          const int tile = __shfl_sync(0xffffffffu, lane == 0 ? ask->y : 0, 0);
          // O^T must hold every tile before `tile`
          const bool due = mbar_test_wait(bar(Cfg::kBarPvDone + (tile - 1) % Cfg::kPvBufs), ((tile - 1) / Cfg::kPvBufs) & 1);
          if (__all_sync(0xffffffffu, due)) {
            tc_fence_after();
            uint32_t o[Cfg::kN];
            tmem_ld16_wait(o_tmem, o);
#pragma unroll
            for (int i = 0; i < kRows; ++i) o[i] = __float_as_uint(__fmul_rn(__uint_as_float(o[i]), alphas[i]));
            tmem_st16(o_tmem, o);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar(Cfg::kBarScaled));
            ++answered;
            moved = true;
          }
        }
        if (moved) {
          t0 = global_timer_ns();
        } else {
          // bounded as mbar_wait
          bool stop = *abort_flag != 0;
          if (global_timer_ns() - t0 > KB_WAIT_LIMIT_NS) {
            atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevTimeoutSoftmax));
            stop = true;
          }
          if (__any_sync(0xffffffffu, stop)) {
            *abort_flag = 1;
            ok = false;
          }
        }
      }
      if constexpr (kCluster) {
        // A segment a CTA (one row a sequence): once every CTA is done with its
        // rings, the partials go to the first CTA's, which folds them in order.
        // (A CTA that gave up has set the error word; then nothing is written.)
        constexpr uint32_t kSlot = 128 * 16 + 64;           // four rows of each channel, then the rows' states
        cluster_sync();
        if (ok && rank > 0 && nt > 0) {
          const uint32_t slot = smem_addr_in_cta(sbase + Cfg::kVOff + (g0 - 1) * kSlot, 0u);
          st_cluster_f32x4(slot + me * 16u, make_float4(acc_o[0], acc_o[1], acc_o[2], acc_o[3]));
          if (warp == 0 && lane < kGroup) st_cluster_f32x4(slot + 2048u + lane * 16u, make_float4(acc.m, acc.mc, acc.l, 0.0f));
        }
        cluster_sync();
        ok = ok && rank == 0 && *reinterpret_cast<volatile uint32_t*>(args.err) == 0;
        const int ns = (n_kv + kSegTiles - 1) / kSegTiles;
#pragma unroll 1
        for (int sg = 1; sg < ns && rank == 0; ++sg) {
          const uint8_t* slot = smem + Cfg::kVOff + (sg - 1) * kSlot;
          const float4 v = reinterpret_cast<const float4*>(slot)[me];
          const float4 x = lane < kGroup ? reinterpret_cast<const float4*>(slot + 2048)[lane] : make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
          const FoldScale f = fold_state(acc, RowState{x.x, x.y, x.z});
          const float o[kGroup] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            acc_o[i] = fold_o(acc_o[i], o[i], FoldScale{__shfl_sync(0xffffffffu, f.a, i), __shfl_sync(0xffffffffu, f.b, i)});
        }
      }
      if (ok && args.part == nullptr) {
        const float inv = row_inv_l(acc);                   // C4, lane r: row r
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float inv_l = __shfl_sync(0xffffffffu, inv, i);
          if (i < n_rows)
            static_cast<__nv_bfloat16*>(args.o)[((static_cast<size_t>(b) * args.Hq + g * kGroup + i / Lc) * args.L + r0 + i % Lc) * kHeadDim + me] =
                __float2bfloat16_rn(__fmul_rn(acc_o[i], inv_l));
        }
      }
    } else if (warp < Cfg::kQkWarp) {
      // ------------------------------------------------ bytes to bf16 values
      if (!skip) {
        const bool is_v = warp >= Cfg::kVWarp0;
        const int t = static_cast<int>(threadIdx.x) - 32 * (is_v ? Cfg::kVWarp0 : Cfg::kKWarp0);
        constexpr int kStages = Cfg::kKBytes;
        static_assert(Cfg::kKBytes == Cfg::kVBytes, "one walk for both");
        const uint32_t bytes0 = bar(is_v ? Cfg::kBarVByte : Cfg::kBarKByte), read0 = bar(Cfg::kBarByteRead + (is_v ? kStages : 0));
        const uint8_t* staged = smem + (is_v ? Cfg::kVByteOff : Cfg::kKByteOff);
        const int* held = reinterpret_cast<const int*>(smem + Cfg::kExpOff) + (is_v ? kStages : 0);
        // V: a thread's column of eight rows, as in the packed kernel's rings; K:
        // the thread's own row
        const int col = (t & 3) | ((t >> 1) & 4), low = is_v ? ((t >> 4) & 3) ^ ((t & 4) ? 5 : 0) : (t & 7);
        const int row0 = is_v ? low + 8 * (t >> 6) : t;
        const int next_chunk = (low & 1) ? -16 : 16;
        uint8_t* dst0 = smem + Cfg::kVOff + (col >> 2) * kSlabBytes + (row0 >> 3) * 1024 + low * 128 + (((2 * (col & 3)) ^ low) << 4);
        const uint32_t k_tmem = tmem_base + Cfg::kKCol + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const int bufs = is_v ? Cfg::kPvBufs : Cfg::kKBufs;
        const uint32_t empty0 = bar(is_v ? Cfg::kBarPvDone : Cfg::kBarKEmpty), full0 = bar(is_v ? Cfg::kBarVFull : Cfg::kBarKFull);
        bool ok = true;
#pragma unroll 1
        for (int jj = 0; jj < nt; ++jj) {
          const int st = jj % kStages, buf = jj % bufs;
          ok = wait_near(bytes0 + 8u * st, (jj / kStages) & 1, abort_flag, args.err, kDevTimeoutTma);
          if (ok && jj >= bufs) ok = wait_near(empty0 + 8u * buf, (jj / bufs - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const Scale8 sc = scale8(held[st]);
          const int n = seq_kv - (j0 + jj) * kTileKeys;     // rows of the sequence in the tile
          const bool whole = n >= kTileKeys && !sc.two;     // else: the sequence's last tile, or values beyond 448 * 2^7
          const uint8_t* src = staged + st * Cfg::kByteTile + row0 * 128;
          // (small loops stay in the schedulers' instruction caches, which the kernel's many roles share)
          if (is_v) {
            constexpr int kStep = kVStep;                    // from a thread's row to its next: bytes staged, and of a slab
            uint8_t* dst = dst0 + buf * kTileBytes;
            src += (col ^ low) << 4;
            if (!whole) odd_values(src, dst, next_chunk, row0, n, sc);
#pragma unroll 1
            for (int i = 0; i < kPasses && whole; i += 2) {
              uint4 w[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) w[q] = *reinterpret_cast<const uint4*>(src + (i + q) * kStep);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint4 lo, hi;
                values8x16(w[q], sc.first, lo, hi);
                *reinterpret_cast<uint4*>(dst + (i + q) * kStep) = lo;
                *reinterpret_cast<uint4*>(dst + (i + q) * kStep + next_chunk) = hi;
              }
            }
            fence_proxy_async_smem();
            mbar_arrive(full0 + 8u * buf);
          } else {
            tc_fence_after();
            if (!whole) odd_keys(src, k_tmem + buf * 64u, row0, n, sc);
#pragma unroll 1
            for (int i = 0; i < kPasses && whole; i += 2) {
              uint4 w[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) w[q] = *reinterpret_cast<const uint4*>(src + (((i + q) ^ low) << 4));
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint4 lo, hi;
                values8x16(w[q], sc.first, lo, hi);
                tmem_st8(k_tmem + buf * 64u + (i + q) * 8u, lo, hi);
              }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(full0 + 8u * buf);
          }
          __syncwarp();                                     // (the stage is read)
          if (lane == 0) mbar_arrive(read0 + 8u * st);
        }
      }
    } else if (warp == Cfg::kQkWarp) {
      // -------------------------------------------------------- S^T issuer
      if (lane == 0 && !skip) {
        const uint32_t idesc = idesc_bf16_f32(128, Cfg::kN, 0);
        const uint32_t q = sbase + Cfg::kQOff;
        bool ok = wait_near(bar(Cfg::kBarQReady), 0, abort_flag, args.err, kDevTimeoutTma);
        for (int j = 0; j < nt && ok; ++j) {
          const int kb = j % Cfg::kKBufs, sb = j % Cfg::kSBufs;
          ok = wait_near(bar(Cfg::kBarKFull + kb), (j / Cfg::kKBufs) & 1, abort_flag, args.err, kDevTimeoutTma);
          if (ok && j >= Cfg::kSBufs)
            ok = wait_near(bar(Cfg::kBarSEmpty + sb), (j / Cfg::kSBufs - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem_base + Cfg::kSCol + sb * Cfg::kN, tmem_base + Cfg::kKCol + kb * 64u + kk * 8u,
                   desc_kmajor(q, kk, 1024u, Cfg::kQSlab), idesc, kk > 0 ? 1u : 0u);
          tc_commit(bar(Cfg::kBarSFull + sb));
          tc_commit(bar(Cfg::kBarKEmpty + kb));
        }
        if (!ok || kFlat) {                                  // (flat: no arrival comes late for the next piece's barriers)
          tc_commit(bar(Cfg::kBarDrain));
          drain_far(bar(Cfg::kBarDrain), 0);
        }
      }
    } else if (warp == Cfg::kPvWarp) {
      // -------------------------------------------------------- O^T issuer
      // The first product of a segment clears O^T, once the segment before it
      // has been read.
      if (lane == 0 && !skip) {
        const uint32_t idesc = idesc_bf16_f32(128, Cfg::kN, 0) | (1u << 15);     // A: channels are contiguous
        bool ok = true;
        for (int j = 0; j < nt && ok; ++j) {
          const int pb = j % Cfg::kPvBufs;
          const bool first = j % kSegTiles == 0;
          ok = wait_near(bar(Cfg::kBarVFull + pb), (j / Cfg::kPvBufs) & 1, abort_flag, args.err, kDevTimeoutTma);
          if (ok && first && j > 0) ok = wait_near(bar(Cfg::kBarORead), (j / kSegTiles - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
          if (ok) ok = wait_near(bar(Cfg::kBarPFull + pb), (j / Cfg::kPvBufs) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem_base + Cfg::kOCol, desc_v(sbase + Cfg::kVOff + pb * kTileBytes, kk),
                   desc_kmajor(sbase + Cfg::kPOff + pb * 2 * Cfg::kQSlab, kk, 1024u, Cfg::kQSlab), idesc, (first && kk == 0) ? 0u : 1u);
          tc_commit(bar(Cfg::kBarPvDone + pb));
        }
        if (!ok || kFlat) {
          tc_commit(bar(Cfg::kBarDrain + 1));
          drain_far(bar(Cfg::kBarDrain + 1), 0);
        }
      }
    } else if (warp == Cfg::kProdWarp) {
      // ----------------------------------------------------------- producer
      if (!skip)
        produce_bytes<Cfg::kKBytes, true>(tmap_k, tmap_v, args, b, g, j0, nt, sbase + Cfg::kKByteOff, sbase + Cfg::kVByteOff,
                                    reinterpret_cast<int*>(smem + Cfg::kExpOff), bar(Cfg::kBarKByte), bar(Cfg::kBarByteRead), abort_flag);
    } else if (warp == Cfg::kSoftmaxWarp) {
      // --- softmax: eight lanes per row and two tiles at a time, or (more than
      // four rows) four lanes per row and a tile at a time
      const bool oct = n_rows <= 4;
      const int m = oct ? lane >> 3 : lane >> 2, u = oct ? lane & 7 : lane & 3;       // packed row
      const int pos = pos0 + (m < n_rows ? r0 + m % Lc : r0);         // unused rows take the sub-chunk's first position
      const float* x_row = reinterpret_cast<const float*>(smem + Cfg::kXOff) + m * Cfg::kXStride;
      uint8_t* p_row = smem + Cfg::kPOff + m * 128;
      volatile int2* ask = reinterpret_cast<volatile int2*>(smem + Cfg::kAskOff);
      float* alphas = reinterpret_cast<float*>(smem + Cfg::kAlphaOff);
      float2* stats = reinterpret_cast<float2*>(smem + Cfg::kStatsOff);
      RowState st = row_state_init();
      int asked = 0;
      bool ok = !skip;
      // tile j's P may go to its product; O^T is scaled before it where a row's
      // reference maximum moved (rare)
      auto publish = [&](int j, float alpha) {
        if (j % kSegTiles != 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          if (u == 0) alphas[m] = alpha;
          __threadfence_block();
          __syncwarp();
          if (lane == 0) {
            ask->y = j;
            __threadfence_block();
            ask->x = asked + 1;
          }
          ok = wait_near(bar(Cfg::kBarScaled), asked & 1, abort_flag, args.err, kDevTimeoutSoftmax);
          ok = __all_sync(0xffffffffu, ok);
          ++asked;
        }
        mbar_arrive(bar(Cfg::kBarPFull + j % Cfg::kPvBufs));
      };
      for (int j = 0; j < nt && ok;) {
        const bool two = oct && j + 1 < nt;                 // (a segment has an even number of tiles, but for the last)
        const int jl = two ? j + 1 : j;
        // waiting for the later of two covers both: they come in order
        ok = wait_near(bar(Cfg::kBarXFull + jl % Cfg::kXBufs), (jl / Cfg::kXBufs) & 1, abort_flag, args.err, kDevTimeoutMma);
        if (ok && jl >= Cfg::kPvBufs)                       // P's buffers are free once the products that read them are done
          ok = wait_near(bar(Cfg::kBarPvDone + jl % Cfg::kPvBufs), (jl / Cfg::kPvBufs - 1) & 1, abort_flag, args.err, kDevTimeoutMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (j % kSegTiles == 0) st = row_state_init();
        const int n_valid = j0 + jl == n_kv - 1 ? pos - (j0 + jl) * kTileKeys + 1 : kTileKeys;   // of tile jl
        if (oct) {
          float x[2][16], alpha[2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[t][r] = x_row[(j + (two ? t : 0)) % Cfg::kXBufs * (kRows * Cfg::kXStride) + 8 * r + u];
          if (n_valid < kTileKeys) {                        // the contract's mask; then one copy of its row math
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const bool off = 8 * r + u >= n_valid;
              x[0][r] = off && !two ? -INFINITY : x[0][r];
              x[1][r] = off && two ? -INFINITY : x[1][r];
            }
          }
          mbar_arrive(bar(Cfg::kBarXEmpty + j % Cfg::kXBufs));
          if (two) {
            mbar_arrive(bar(Cfg::kBarXEmpty + jl % Cfg::kXBufs));
            row_softmax_tiles_oct<true>(x, st, alpha);
          } else {
            row_softmax_tiles_oct<false>(x, st, alpha);
          }
          // key 8r + u of row m: half word u of chunk r
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (t == 0 || two) {
              uint8_t* pd = p_row + (j + t) % Cfg::kPvBufs * 2 * Cfg::kQSlab + 2 * u;
#pragma unroll
              for (int r = 0; r < 16; ++r)
                *reinterpret_cast<__nv_bfloat16*>(pd + (r >> 3) * Cfg::kQSlab + (((r & 7) ^ m) << 4)) = __float2bfloat16_rn(x[t][r]);
            }
          fence_proxy_async_smem();
          publish(j, alpha[0]);
          if (two && ok) publish(jl, alpha[1]);
        } else {
          float x[32];
          const float* xr = x_row + j % Cfg::kXBufs * (kRows * Cfg::kXStride);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float2 v = reinterpret_cast<const float2*>(xr)[4 * r + u];
            x[2 * r] = v.x;
            x[2 * r + 1] = v.y;
          }
          mbar_arrive(bar(Cfg::kBarXEmpty + j % Cfg::kXBufs));
          if (n_valid < kTileKeys) {
#pragma unroll
            for (int r = 0; r < 32; ++r) x[r] = 8 * (r >> 1) + 2 * u + (r & 1) < n_valid ? x[r] : -INFINITY;
          }
          uint32_t p[16];
          const float alpha = row_softmax_tile_quad<false>(x, u, kTileKeys, st, p);
          // the pair of keys 8r + 2u of row m: word u of chunk r
          uint8_t* pd = p_row + j % Cfg::kPvBufs * 2 * Cfg::kQSlab + 4 * u;
#pragma unroll
          for (int r = 0; r < 16; ++r) *reinterpret_cast<uint32_t*>(pd + (r >> 3) * Cfg::kQSlab + (((r & 7) ^ m) << 4)) = p[r];
          fence_proxy_async_smem();
          publish(j, alpha);
        }
        if (!ok) break;
        if (jl % kSegTiles == kSegTiles - 1 || jl == nt - 1) {
          const int G = jl / kSegTiles;
          if (G >= 2) {
            ok = wait_near(bar(Cfg::kBarStEmpty + (G & 1)), (G / 2 - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          if (u == 0) stats[(G & 1) * kRows + m] = make_float2(st.m, st.l);
          mbar_arrive(bar(Cfg::kBarStFull + (G & 1)));
        }
        j = jl + 1;
      }
    }

    if (kCluster && warp >= 4) {                              // the other warps' part in the cluster's barriers
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag != 0) break;
  } while (kFlat);                                        // pieces
  if (begun && warp == Cfg::kQkWarp) {
    __syncwarp();
    tmem_dealloc(misc[0], Cfg::kTmemCols);
  }
}

template <bool kFlat, bool kCluster>
static cudaError_t launch_decode8_t(const CUtensorMap& tk, const CUtensorMap& tv, const PackedArgs& a, long long grid, cudaStream_t s) {
  using Cfg = Decode8Cfg;
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kb_decode8_kernel<kFlat, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(Cfg::kSmemBytes));
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(kCluster ? a.cluster : 1);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kb_decode8_kernel<kFlat, kCluster>, tk, tv, a);
}

cudaError_t launch_decode8(const CUtensorMap& tk, const CUtensorMap& tv, const PackedArgs& a, int n_sub, cudaStream_t s) {
  const long long units = static_cast<long long>(n_sub) * a.B * a.Hkv;
  if (a.part != nullptr) {
    if (a.split == 0) return launch_decode8_t<true, false>(tk, tv, a, a.ctas, s);
    return launch_decode8_t<false, false>(tk, tv, a, a.split * units, s);
  }
  if (a.cluster > 1) return launch_decode8_t<false, true>(tk, tv, a, a.cluster * units, s);
  return launch_decode8_t<false, false>(tk, tv, a, units, s);
}

}  // namespace kb

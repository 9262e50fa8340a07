// kb_sparse.cu -- attention of query rows over listed key blocks (chunks and
// whole sequences), under the numerical contract of kb_contract.cuh.
//
// A row's keys are those of its listed blocks, up to its position.  Its
// result is that of the contract's walk over the listed blocks alone: tiles
// in ascending order (C1), the same products and row function (C2, C3), the
// same segments of eight tiles anchored at tile 0 (C5; a segment of which the
// row lists nothing is left out), the same normalisation (C4).  So a row has
// the same bits here, in a chunk of any split and alone as a new token, and a
// row that lists every block has the dense entry points' bits.  A row that
// lists nothing is zero, with a log-sum-exp of -inf.
//
// Layout.  Lists differ from row to row but little between neighbours, so a
// unit of 32 positions times the four heads of a KV head (128 rows: the MMA's
// M) walks the union of its rows' lists (kb_sparse_plan.cu).  A row that did
// not list a tile has its scores masked there: P = 0 adds exactly nothing to
// O, and the row's state stays as it was.  Work beyond the lists is what the
// union adds; K and V are read once for four heads.
//
// Roles and pipeline are those of the dense tile kernel (kb_prefill2.cu):
//   warps 0..7   softmax (quads of threads per row)
//   warp 8       TMA producer of Q and the K ring
//   warp 9       TMEM allocator + Q K^T issuer
//   warp 10      TMA producer of the V ring (zeroes a V tail)
//   warp 11      P V issuer
//   warps 12..15 fold and epilogue: warp 12+h owns head h, lane r row r
// TMEM: S, P0, P1 (64 columns each), O0, O1.  Scattered lists give segments of
// one or two tiles, so a segment's fold must not hold up the next one's P V:
// segments alternate between two O buffers and two sets of row statistics.
// One S buffer is enough beside them, because P has columns of its own: the
// softmax warps read a tile's scores at once and release them before they
// compute, so Q K^T of the next tile runs under the softmax of this one.
//
// Measured: 2048 rows at the end of 64K keys, 16 blocks a row (47 a unit) 235
// us; 8192 rows, 16 a row (21 a unit) 337 us.  That is about 2,300 cycles a tile
// and SM, against 1,750 of the dense kernel, whose segments are eight tiles
// long: the softmax warps' chain is the bound (two warps per SM quarter, 47 %
// of issue slots, tensor pipe 44 to 50 % busy).  Of the chunk with its plan (248
// us): one O buffer 289, and a select per masked key besides 307.
// Tried and slower, in the chunk above: both products issued by one thread 283;
// rows A and B of a thread skipped one by one where they did not list the tile
// 396 (their chains no longer overlap); a warp's tile skipped where none of its
// sixteen positions listed it 249 (neighbours' lists overlap too much); units
// dealt one at a time through a ring in shared memory, 1.9 us a unit more than a
// fixed deal.
#include "kb_sparse.cuh"

namespace kb {

struct SparseCfg {
  static constexpr int kThreads = 512;
  static constexpr int kLoadWarpK = 8;
  static constexpr int kMmaWarp = 9;
  static constexpr int kLoadWarpV = 10;
  static constexpr int kPvWarp = 11;
  static constexpr int kFoldWarp0 = 12;
  static constexpr int kStages = 3;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kPCol = 128u;                  // S in columns 0..127, then P(T) in P buffer T%2, 64 columns
  static constexpr uint32_t kOCol = 256u;                  // two of them: segment G in O buffer G%2
  // 256 softmax, 128 producer/issuer and 128 fold threads share the launch's 512 x 128 registers
  static constexpr uint32_t kSoftmaxRegs = 136;
  static constexpr uint32_t kOtherRegs = 64;
  static constexpr uint32_t kFoldRegs = 176;
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kKOff = kTileBytes;
  static constexpr uint32_t kVOff = kKOff + kStages * kTileBytes;
  static constexpr uint32_t kBarOff = kVOff + kStages * kTileBytes;
  static constexpr int kBarQFull = 0;
  static constexpr int kBarKFull = 1;
  static constexpr int kBarVFull = kBarKFull + kStages;
  static constexpr int kBarKEmpty = kBarVFull + kStages;   // Q K^T(T) done, K slot T%3 free
  static constexpr int kBarVEmpty = kBarKEmpty + kStages;  // P V(T) done, V slot T%3 free
  static constexpr int kBarSFull = kBarVEmpty + kStages;   // S(T) written
  static constexpr int kBarSRead = kBarSFull + 1;          // S(T) read (256 arrivals)
  static constexpr int kBarPFull = kBarSRead + 1;          // 2: P(T) written (256 arrivals)
  static constexpr int kBarPDone = kBarPFull + 2;          // 2: P V(T) done, P buffer T%2 free
  static constexpr int kBarVReady = kBarPDone + 2;         // a unit's last V tile with its tail zeroed
  static constexpr int kBarQEmpty = kBarVReady + kStages;  // a unit's last Q K^T done
  static constexpr int kBarSegDone = kBarQEmpty + 1;       // 2: segment G's last P V done
  static constexpr int kBarORead = kBarSegDone + 2;        // 2: segment G's O was read (128 fold threads)
  static constexpr int kBarStFull = kBarORead + 2;         // 2: segment G's (m, l) written (256 softmax)
  static constexpr int kBarStEmpty = kBarStFull + 2;       // 2: ... and read (128 fold threads)
  static constexpr int kBarDrain = kBarStEmpty + 2;        // 2: one per MMA issuer
  static constexpr int kNumBars = kBarDrain + 2;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kStatsOff = (kMiscOff + 16u + 15u) & ~15u;   // 2: float2 (m, l) per row
  static constexpr uint32_t kSmemUsed = kStatsOff + 2u * kTileRows * 8;
  static constexpr uint32_t kSmemBytes = kSmemUsed;        // the array is declared 1 KB aligned: no room is left to round up
};
static_assert(8 * 32 * SparseCfg::kSoftmaxRegs + 4 * 32 * SparseCfg::kOtherRegs + 4 * 32 * SparseCfg::kFoldRegs <=
                  512 * 128,
              "register split above the launch's registers");

namespace {

__device__ __forceinline__ void drain_wait_s(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 50000000ull) break;
}

// The last entry's V tile holds rows past the sequence (only a paged or
// ragged cache maps them; a contiguous uniform one reads zeros there).
__device__ __forceinline__ bool has_v_tail(const SparseArgs& a, const SparseUnit& w, uint32_t last_entry) {
  return (a.block_table != nullptr || a.starts != nullptr) && static_cast<int>(last_entry & kEntryBlock) == w.own &&
         w.kv_len < (w.own + 1) * kTileKeys;
}

}  // namespace

__global__ void __launch_bounds__(SparseCfg::kThreads, 1)
kb_sparse_tile_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const SparseArgs args) {
  using Cfg = SparseCfg;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return smem_addr(bars + i); };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kNumBars; ++i) {
      uint32_t count = 1u;
      if (i == Cfg::kBarSRead || (i >= Cfg::kBarPFull && i < Cfg::kBarPFull + 2) ||
          (i >= Cfg::kBarStFull && i < Cfg::kBarStFull + 2))
        count = 256u;
      if ((i >= Cfg::kBarORead && i < Cfg::kBarORead + 2) || (i >= Cfg::kBarStEmpty && i < Cfg::kBarStEmpty + 2)) count = 128u;
      mbar_init(bar(i), count);
    }
    if ((sbase & 1023u) != 0u) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));   // never expected
    misc[1] = (*reinterpret_cast<volatile uint32_t*>(args.err) != 0) ? 1u : 0u;
    fence_mbar_init();
  }
  if (warp == Cfg::kMmaWarp) {
    tmem_alloc(sbase + Cfg::kMiscOff, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];
  const bool skip = (*abort_flag != 0);
  // Every role counts the tiles it has handled (T); ring slots, S buffers and
  // barrier parities follow from that count.

  if (warp >= Cfg::kFoldWarp0) {
    // ------------------------------------------------- fold and epilogue
    regs_increase<Cfg::kFoldRegs>();
    const int head = warp - Cfg::kFoldWarp0;
    const int row = 32 * head + lane;                                // TMEM lane
    const uint32_t o_tmem0 = tmem_base + Cfg::kOCol + (static_cast<uint32_t>(32 * head) << 16);
    const float2* stats = reinterpret_cast<const float2*>(smem + Cfg::kStatsOff);
    const float c = score_scale_log2();
    int G = 0;                                                       // segments
    bool ok = !skip;
    KB_FOR_EACH_SPARSE_UNIT(args, u, w, n, walk) {
      if (!ok) break;
      RowState acc = row_state_init();
      bool none = true;                                              // the row has folded no segment yet
      uint32_t oacc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) oacc[i] = 0u;
      for (int j = 0; j < n && ok; ++j) {
        if (!(__ldg(&walk[j].x) & kEntrySegEnd)) continue;
        const int buf = G & 1;                                       // segment G's O and stats buffers
        const uint32_t turn = (G >> 1) & 1;
        const uint32_t o_tmem = o_tmem0 + 128u * buf;
        ok = mbar_wait_idle(bar(Cfg::kBarStFull + buf), turn, abort_flag, args.err, kDevTimeoutSoftmax, 64);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float2 st = stats[kTileRows * buf + row];
        const RowState sg{st.x, __fmul_rn(st.x, c), st.y};
        mbar_arrive(bar(Cfg::kBarStEmpty + buf));
        ok = mbar_wait_idle(bar(Cfg::kBarSegDone + buf), turn, abort_flag, args.err, kDevTimeoutMma, 32);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // C5, per row: a segment without listed blocks is left out, the first
        // one is taken as it is (a NaN sum is no empty segment)
        const bool has = st.x != -INFINITY || !(st.y == 0.0f);
        const bool take = has && none;
        const bool fold = has && !none;
        FoldScale f{1.0f, 1.0f};
        if (fold) f = fold_state(acc, sg);
        if (take) acc = sg;
        none = none && !has;
        uint32_t oa[16], ob[16];
        auto chunk = [&](int base, const uint32_t (&o)[16]) {
          if (fold) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 r = fold_o2(make_float2(__uint_as_float(oacc[base + i]), __uint_as_float(oacc[base + i + 1])),
                                       make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f);
              oacc[base + i] = __float_as_uint(r.x);
              oacc[base + i + 1] = __float_as_uint(r.y);
            }
          } else if (take) {
#pragma unroll
            for (int i = 0; i < 16; ++i) oacc[base + i] = o[i];
          }
          __syncwarp();                                              // rows differ; the next TMEM load is the whole warp's
        };
        tmem_ld16_issue(o_tmem, oa);
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
          tmem_ld16_wait_for(oa);
          tmem_ld16_issue(o_tmem + 16u * (q + 1), ob);
          chunk(16 * q, oa);
          tmem_ld16_wait_for(ob);
          if (q + 2 < 8) tmem_ld16_issue(o_tmem + 16u * (q + 2), oa);
          chunk(16 * (q + 1), ob);
        }
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarORead + buf));
        ++G;
      }
      if (!ok) break;
      const int i = w.t * kUnitRows + lane - w.start;                // query row index in q / o
      if (i >= 0 && i < w.L) {
        const float inv_l = none ? 0.0f : row_inv_l(acc);
        const size_t plane_row = (static_cast<size_t>(w.b) * args.Hq + w.g * kGroup + head) * static_cast<size_t>(args.L) + i;
        if (args.lse != nullptr) {
          constexpr float kLn2 = 0.69314718055994531f;
          args.lse[plane_row] = none ? -INFINITY : __fmul_rn(__fadd_rn(acc.mc, log2f(acc.l)), kLn2);
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.o) + plane_row * kHeadDim);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          uint32_t wv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            wv[e] = pack_bf16x2(__fmul_rn(__uint_as_float(oacc[8 * q + 2 * e]), inv_l),
                                __fmul_rn(__uint_as_float(oacc[8 * q + 2 * e + 1]), inv_l));
          dst[q] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
        }
      }
    }
  } else if (warp >= Cfg::kLoadWarpK) {
    regs_decrease<Cfg::kOtherRegs>();
    if (warp == Cfg::kLoadWarpK || warp == Cfg::kLoadWarpV) {
      // --------------------------------------------------------- producers
      const bool is_v = (warp == Cfg::kLoadWarpV);
      if (!skip) {
        const uint64_t keep = l2_policy_evict_last();
        const CUtensorMap* tmap = is_v ? &tmap_v : &tmap_k;
        const int full0 = is_v ? Cfg::kBarVFull : Cfg::kBarKFull;
        const int empty0 = is_v ? Cfg::kBarVEmpty : Cfg::kBarKEmpty;
        const uint32_t ring = sbase + (is_v ? Cfg::kVOff : Cfg::kKOff);
        if (lane == 0) {
          tma_prefetch_desc(tmap);
          if (!is_v) tma_prefetch_desc(&tmap_q);
        }
        int T = 0, U = 0;                                            // tiles; units with tiles
        bool ok = true;
        KB_FOR_EACH_SPARSE_UNIT(args, u, w, n, walk) {
          if (!ok) break;
          if (n == 0) continue;
          if (!is_v) {
            if (U > 0) ok = mbar_wait(bar(Cfg::kBarQEmpty), (U - 1) & 1, abort_flag, args.err, kDevTimeoutSlot);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(Cfg::kBarQFull), kTileBytes);
              tma_load_group(sbase + Cfg::kQOff, &tmap_q, w.t * kUnitRows - w.start, w.b * args.Hkv + w.g,
                             bar(Cfg::kBarQFull));
            }
          }
          ++U;
          uint32_t next = __ldg(&walk[0].x), entry = next;
          for (int j = 0; j < n; ++j, ++T) {
            entry = next;
            if (j + 1 < n) next = __ldg(&walk[j + 1].x);
            const int slot = T % Cfg::kStages;
            int row = static_cast<int>(entry & kEntryBlock) * kTileKeys, plane = w.b * args.Hkv + w.g;
            if (args.block_table != nullptr && lane == 0) {
              int pg = args.block_table[static_cast<size_t>(w.b) * args.pages_per_seq + row / args.page_size];
              if (pg < 0 || pg >= args.num_pages) {
                atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
                pg = args.num_pages;       // beyond the map: the TMA unit reads zeros
              }
              row = row % args.page_size;
              plane = pg * args.Hkv + w.g;
            }
            if (T >= Cfg::kStages)
              ok = mbar_wait(bar(empty0 + slot), ((T / Cfg::kStages) - 1) & 1, abort_flag, args.err,
                             kDevTimeoutSlot);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(full0 + slot), kTileBytes);
              tma_load_tile_hint(ring + slot * kTileBytes, tmap, row, plane, bar(full0 + slot), keep);
            }
          }
          if (ok && is_v && has_v_tail(args, w, entry)) {
            // V rows past kv_len in the unit's last tile may hold anything: zero them
            const int TL = T - 1;
            const int slot = TL % Cfg::kStages;
            ok = mbar_wait(bar(Cfg::kBarVFull + slot), (TL / Cfg::kStages) & 1, abort_flag, args.err,
                           kDevTimeoutTma);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              uint8_t* vt = smem + Cfg::kVOff + slot * kTileBytes;
              for (int idx = (w.kv_len - w.own * kTileKeys) * 16 + lane; idx < kTileKeys * 16; idx += 32) {
                const int vr = idx >> 4;
                const int ch = idx & 15;
                *reinterpret_cast<uint4*>(vt + (ch >> 3) * kSlabBytes + (vr >> 3) * 1024 + (vr & 7) * 128 +
                                          (((ch & 7) ^ (vr & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(Cfg::kBarVReady + slot));
            }
          }
        }
        if (!ok && lane == 0) {
          if (!is_v && U > 0) drain_wait_s(bar(Cfg::kBarQFull), (U - 1) & 1);
          for (int x = (T > Cfg::kStages ? T - Cfg::kStages : 0); x < T; ++x)
            drain_wait_s(bar(full0 + x % Cfg::kStages), (x / Cfg::kStages) & 1);
        }
      }
    } else if (warp == Cfg::kMmaWarp) {
      // ------------------------------------------------------ Q K^T issuer
      if (lane == 0 && !skip) {
        const uint32_t q_saddr = sbase + Cfg::kQOff;
        int T = 0, U = 0;
        bool ok = true;
        KB_FOR_EACH_SPARSE_UNIT(args, u, w, n, walk) {
          if (!ok) break;
          if (n == 0) continue;
          ok = mbar_wait(bar(Cfg::kBarQFull), U & 1, abort_flag, args.err, kDevTimeoutTma);
          for (int j = 0; j < n && ok; ++j, ++T) {
            const int slot = T % Cfg::kStages;
            ok = mbar_wait(bar(Cfg::kBarKFull + slot), (T / Cfg::kStages) & 1, abort_flag, args.err, kDevTimeoutTma);
            if (ok && T > 0) ok = mbar_wait_hint(bar(Cfg::kBarSRead), (T - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            if (!ok) break;
            tc_fence_after();
            issue_qk(tmem_base, q_saddr, 1024u, kSlabBytes, sbase + Cfg::kKOff + slot * kTileBytes);
            tc_commit(bar(Cfg::kBarSFull));
            tc_commit(bar(Cfg::kBarKEmpty + slot));
          }
          if (ok) tc_commit(bar(Cfg::kBarQEmpty));
          ++U;
        }
        if (!ok) {
          tc_commit(bar(Cfg::kBarDrain));
          drain_wait_s(bar(Cfg::kBarDrain), 0);
        }
      }
    } else {
      // -------------------------------------------------------- P V issuer
      if (lane == 0 && !skip) {
        int T = 0, F = 0;                                           // F: segments finished
        uint32_t zero_parity = 0;                                   // bit s: zero-tail phases of V slot s, mod 2
        bool ok = true;
        KB_FOR_EACH_SPARSE_UNIT(args, u, w, n, walk) {
          if (!ok) break;
          if (n == 0) continue;
          uint32_t next = __ldg(&walk[0].x);
          for (int j = 0; j < n && ok; ++j, ++T) {
            const uint32_t entry = next;
            if (j + 1 < n) next = __ldg(&walk[j + 1].x);
            const int pb = T & 1, slot = T % Cfg::kStages;
            ok = mbar_wait_hint(bar(Cfg::kBarPFull + pb), (T >> 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            if (ok) {
              if (j == n - 1 && has_v_tail(args, w, entry)) {
                ok = mbar_wait(bar(Cfg::kBarVReady + slot), (zero_parity >> slot) & 1u, abort_flag, args.err,
                               kDevTimeoutTma);
                zero_parity ^= 1u << slot;
              } else {
                ok = mbar_wait(bar(Cfg::kBarVFull + slot), (T / Cfg::kStages) & 1, abort_flag, args.err, kDevTimeoutTma);
              }
            }
            const bool first = (entry & kEntrySegStart) != 0u;
            const int buf = F & 1;                                  // the segment's O buffer
            if (ok && first && F >= 2)
              ok = mbar_wait(bar(Cfg::kBarORead + buf), ((F >> 1) - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            if (!ok) break;
            tc_fence_after();
            issue_pv(tmem_base + Cfg::kOCol + 128u * buf, tmem_base + Cfg::kPCol + 64u * pb,
                     sbase + Cfg::kVOff + slot * kTileBytes, first);
            tc_commit(bar(Cfg::kBarPDone + pb));
            tc_commit(bar(Cfg::kBarVEmpty + slot));
            if (entry & kEntrySegEnd) {
              tc_commit(bar(Cfg::kBarSegDone + buf));
              ++F;
            }
          }
        }
        if (!ok) {
          tc_commit(bar(Cfg::kBarDrain + 1));
          drain_wait_s(bar(Cfg::kBarDrain + 1), 0);
        }
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    regs_increase<Cfg::kSoftmaxRegs>();
    const int q4 = warp & 3;                                        // head = TMEM lane quarter of this warp
    const int r0 = 16 * (warp >> 2) + (lane >> 2);                  // the thread's rows of the unit: r0 and r0 + 8
    const uint32_t lane_off = static_cast<uint32_t>(32 * q4 + 16 * (warp >> 2)) << 16;
    const int u4 = lane & 3;
    float2* stats = reinterpret_cast<float2*>(smem + Cfg::kStatsOff);
    int T = 0, G = 0;                                               // tiles, segments
    bool ok = !skip;
    KB_FOR_EACH_SPARSE_UNIT(args, u, w, n, walk) {
      if (!ok) break;
      if (n == 0) continue;
      RowState sA = row_state_init(), sB = row_state_init();
      uint2 next = __ldg(&walk[0]);
      const int p0 = w.t * kUnitRows - w.own * kTileKeys;           // the unit's first row within its own block
      for (int j = 0; j < n && ok; ++j, ++T) {
        const uint2 entry = next;
        if (j + 1 < n) next = __ldg(&walk[j + 1]);
        ok = mbar_wait_hint(bar(Cfg::kBarSFull), T & 1, abort_flag, args.err, kDevTimeoutMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_tmem = tmem_base + lane_off;
        float xA[32], xB[32];
        {
          uint32_t v0[32], v1[32];
          tmem_ld_16x256b_x8_pair_wait(s_tmem, s_tmem + 64u, v0, v1);   // keys 0..63, 64..127
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            xA[2 * r] = __uint_as_float(v0[4 * r]);
            xA[2 * r + 1] = __uint_as_float(v0[4 * r + 1]);
            xB[2 * r] = __uint_as_float(v0[4 * r + 2]);
            xB[2 * r + 1] = __uint_as_float(v0[4 * r + 3]);
            xA[16 + 2 * r] = __uint_as_float(v1[4 * r]);
            xA[16 + 2 * r + 1] = __uint_as_float(v1[4 * r + 1]);
            xB[16 + 2 * r] = __uint_as_float(v1[4 * r + 2]);
            xB[16 + 2 * r + 1] = __uint_as_float(v1[4 * r + 3]);
          }
        }
        // S is in registers: the next tile's Q K^T may overwrite it
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarSRead));
        const bool seg_start = (entry.x & kEntrySegStart) != 0u;
        if (seg_start) {                                            // C5: each segment starts fresh
          sA = row_state_init();
          sB = row_state_init();
        }
        // rows without keys so far hold O = 0: nothing to rescale when their
        // reference max first moves
        const bool freshA = sA.m == -INFINITY, freshB = sB.m == -INFINITY;
        const bool diag = static_cast<int>(entry.x & kEntryBlock) == w.own;
        uint32_t pkA[16], pkB[16];
        float aA, aB;
        const bool onA = (entry.y >> r0) & 1u, onB = (entry.y >> (r0 + 8)) & 1u;
        const float lA = sA.l, lB = sB.l;
        if (!diag) {
          aA = row_softmax_tile_quad<false, true>(xA, u4, kTileKeys, sA, pkA, onA);
          aB = row_softmax_tile_quad<false, true>(xB, u4, kTileKeys, sB, pkB, onB);
        } else {
          aA = row_softmax_tile_quad<true, true>(xA, u4, onA ? p0 + r0 + 1 : 0, sA, pkA);
          aB = row_softmax_tile_quad<true, true>(xB, u4, onB ? p0 + r0 + 9 : 0, sB, pkB);
        }
        if (freshA) aA = 1.0f;
        if (freshB) aB = 1.0f;
        // a row that did not list the tile, but whose sum moved: its scores were
        // not finite, and its weights are zero all the same
        const bool moved_off = (!onA && !(sA.l == lA)) || (!onB && !(sB.l == lB));
        if (__any_sync(0xffffffffu, moved_off)) {
          if (!onA) sA.l = lA;
          if (!onB) sB.l = lB;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            pkA[r] = onA ? pkA[r] : 0u;
            pkB[r] = onB ? pkB[r] : 0u;
          }
        }
        if (!seg_start && __any_sync(0xffffffffu, aA != 1.0f || aB != 1.0f)) {
          ok = mbar_wait(bar(Cfg::kBarPDone + ((T - 1) & 1)), ((T - 1) >> 1) & 1, abort_flag, args.err, kDevTimeoutMma);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t o_tmem = tmem_base + Cfg::kOCol + 128u * (G & 1) + lane_off;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t o[32];
            tmem_ld_16x256b_x8_wait(o_tmem + 64u * half, o);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const float2 ra = __fmul2_rn(make_float2(__uint_as_float(o[4 * r]), __uint_as_float(o[4 * r + 1])),
                                           make_float2(aA, aA));
              const float2 rb = __fmul2_rn(make_float2(__uint_as_float(o[4 * r + 2]), __uint_as_float(o[4 * r + 3])),
                                           make_float2(aB, aB));
              o[4 * r] = __float_as_uint(ra.x);
              o[4 * r + 1] = __float_as_uint(ra.y);
              o[4 * r + 2] = __float_as_uint(rb.x);
              o[4 * r + 3] = __float_as_uint(rb.y);
            }
            tmem_st_16x256b_x8(o_tmem + 64u * half, o);
          }
        }
        const int pb = T & 1;
        if (T >= 2) {                                               // P V(T-2) has read this P buffer
          ok = mbar_wait(bar(Cfg::kBarPDone + pb), ((T >> 1) - 1) & 1, abort_flag, args.err, kDevTimeoutMma);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        {
          uint32_t pv[32];
#pragma unroll
          for (int r = 0; r < 16; ++r) { pv[2 * r] = pkA[r]; pv[2 * r + 1] = pkB[r]; }
          tmem_st_16x128b_x16(tmem_base + Cfg::kPCol + 64u * pb + lane_off, pv);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarPFull + pb));
        if (entry.x & kEntrySegEnd) {
          // hand the finished segment's (m, l) to the fold warps, once they
          // have read those of the segment two before
          const int buf = G & 1;
          if (G >= 2) {
            ok = mbar_wait(bar(Cfg::kBarStEmpty + buf), ((G >> 1) - 1) & 1, abort_flag, args.err, kDevTimeoutSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          if (u4 == 0) {
            stats[kTileRows * buf + 32 * q4 + r0] = make_float2(sA.m, sA.l);
            stats[kTileRows * buf + 32 * q4 + r0 + 8] = make_float2(sB.m, sB.l);
          }
          mbar_arrive(bar(Cfg::kBarStFull + buf));
          ++G;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

cudaError_t launch_sparse_tile(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const SparseArgs& a, int device, int sm_count, cudaStream_t s) {
  using Cfg = SparseCfg;
  static_assert(Cfg::kSmemBytes <= 227u * 1024u, "shared memory budget");
  static bool configured[64] = {};
  if (!configured[device]) {
    const cudaError_t e = cudaFuncSetAttribute(kb_sparse_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Cfg::kSmemBytes));
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  kb_sparse_tile_kernel<<<static_cast<unsigned>(unit_grid(a, sm_count, 16)), Cfg::kThreads, Cfg::kSmemBytes, s>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

}  // namespace kb

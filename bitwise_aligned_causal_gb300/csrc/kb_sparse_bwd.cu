// kb_sparse_bwd.cu -- gradient of block-sparse attention over a whole
// sequence (row i at position i): the dense backward's formulas
// (kb_backward.cu) over the listed keys alone,
//   dS_ij = P_ij (dP_ij - delta_i),  dq_i = sum_j dS_ij k_j / sqrt(128),
//   dk_j = sum_i dS_ij q_i / sqrt(128),  dv_j = sum_i P_ij dO_i,
// j over row i's listed keys, i over the rows (of the four heads) that listed
// key j's block.  A row that lists nothing and a block nobody lists have zero
// gradients.
//
// Rows come in the units of the forward (32 positions times four heads, 128
// rows).  The dq kernel runs one CTA per unit over the unit's walk; the dk/dv
// kernel one CTA per (b, KV head, key block) over the rows that listed it,
// found in the plan's row masks and packed 32 positions to a step.  A row of a
// unit that did not list the dq kernel's block at hand has P = 0 there.
// Every gradient element is summed in one order, by one CTA, or by two of which
// the second adds both halves; atomics count rows and draw tickets, no more.
//
// Roundings: P and dS go to the tensor core as bf16, with fp32 sums, but for dq
// dS goes as two bf16 parts, for 7 % of the kernel's time.  Relative errors
// against the 64-bit formulas, root mean square, of 1999 rows with 7 blocks;
// rounding the result to bf16 alone is 0.0017:
//   dq 0.0023 (replayed in 64 bits with one part 0.0031).  What is left is
//     delta's, which comes from the forward's bf16 o and whose error is common to
//     a row's keys: 0.0020 with o in two bf16 parts (another tensor between
//     forward and backward, not made), 0.0017 with an exact delta.
//   dk 0.0024 to 0.0029.  What is left is the one rounding of its dS: replayed
//     0.0024 to 0.0027, with an exact delta 0.0024 to 0.0025, with dS in two parts
//     0.0018 (a second product a step, not made).
//   dv 0.0023, the one rounding of P, as in the forward, whose bits are the
//     dense contract's.
//
// Measured for 8192 rows of 32 heads, 16 blocks a row, in the launch list of
// one pass: delta 23 us, dq 502 us (42,700 tiles: about 3,400 cycles a tile and
// SM; the dense kernel 3,200), dk/dv 452 us (201 steps an SM: 4,400 cycles a
// step, the dense kernel's pace), plan and order 17 us.
#include <type_traits>

#include "kb_bwd.cuh"
#include "kb_sparse.cuh"

namespace kb {

// -------------------------------------------------------------- dq kernel

struct SparseBwdQCfg {
  static constexpr int kThreads = 384;        // 8 elementwise warps, two producers, two MMA issuers
  static constexpr int kLoadWarp = 8;         // Q, dO and the K ring
  static constexpr int kMmaWarp = 9;          // TMEM allocator + S, dP issuer
  static constexpr int kDqWarp = 10;          // dQ issuer
  static constexpr int kLoadWarpV = 11;       // the V ring
  // K(j) is read by S(j) and by dQ(j), V(j) only by dP(j): the K ring frees
  // a slot after dQ(j), the V ring after S(j), dP(j), so V needs fewer slots
  static constexpr int kKStages = 3;
  static constexpr int kVStages = 2;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColDP = 128, kColDQ = 256;
  static constexpr uint32_t kColDS = 384, kColDSLow = 448;      // dS as the sum of two bf16 parts, 64 columns each
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kDOOff = kTileBytes;
  static constexpr uint32_t kKOff = 2 * kTileBytes;
  static constexpr uint32_t kVOff = kKOff + kKStages * kTileBytes;
  static constexpr uint32_t kBarOff = kVOff + kVStages * kTileBytes;
  static constexpr int kBarQD = 0;                         // Q and dO landed
  static constexpr int kBarKFull = 1;                      // 3: K(j) landed in slot j%3
  static constexpr int kBarKEmpty = kBarKFull + kKStages;  // 3: dQ(j) done, K slot j%3 free
  static constexpr int kBarVFull = kBarKEmpty + kKStages;  // 2: V(j) landed in slot j%2
  static constexpr int kBarVEmpty = kBarVFull + kVStages;  // 2: S(j), dP(j) done, V slot j%2 free
  static constexpr int kBarSFull = kBarVEmpty + kVStages;  // S(j), dP(j) in TMEM
  static constexpr int kBarSFree = kBarSFull + 1;          // S(j) read (256 arrivals)
  static constexpr int kBarDSFull = kBarSFree + 1;         // dS(j) in TMEM (256 arrivals)
  static constexpr int kBarDQDone = kBarDSFull + 1;        // dQ += dS(j) K(j) finished
  static constexpr int kBarDrain = kBarDQDone + 1;          // 2: one per issuer
  static constexpr int kBarDPFree = kBarDrain + 2;         // dP(j) read (256 arrivals)
  static constexpr int kBarSDone = kBarDPFree + 1;         // S(j) in TMEM (kBarSFull: dP(j) too)
  static constexpr int kBarQDEmpty = kBarSDone + 1;        // a unit's last S, dP done
  static constexpr int kNumBars = kBarQDEmpty + 1;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16 + 1024;
};

// Every role of a CTA walks the same units in the same order; T counts tiles
// (ring slots and parities follow from it), U units with tiles.
__global__ void __launch_bounds__(SparseBwdQCfg::kThreads, 1)
kb_sparse_bwd_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                 const SparseBwdArgs args) {
  using Cfg = SparseBwdQCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return smem_addr(bars + i); };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  uint32_t* const err = args.plan.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kNumBars; ++i)
      mbar_init(bar(i), (i == Cfg::kBarSFree || i == Cfg::kBarDSFull || i == Cfg::kBarDPFree) ? 256u : 1u);
    misc[1] = (*reinterpret_cast<volatile uint32_t*>(err) != 0) ? 1u : 0u;
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

  if (warp == Cfg::kLoadWarp || warp == Cfg::kLoadWarpV) {
    // ----------------------------------------------------------- producers
    // One warp per ring: Q, dO and K; V.
    const bool is_v = (warp == Cfg::kLoadWarpV);
    if (!skip) {
      const uint64_t keep = l2_policy_evict_last();
      const int stages = is_v ? Cfg::kVStages : Cfg::kKStages;
      const int full0 = is_v ? Cfg::kBarVFull : Cfg::kBarKFull;
      const int empty0 = is_v ? Cfg::kBarVEmpty : Cfg::kBarKEmpty;
      const uint32_t ring = sbase + (is_v ? Cfg::kVOff : Cfg::kKOff);
      const CUtensorMap* tmap = is_v ? &tmap_v : &tmap_k;
      if (lane == 0) {
        tma_prefetch_desc(tmap);
        if (!is_v) {
          tma_prefetch_desc(&tmap_q);
          tma_prefetch_desc(&tmap_do);
        }
      }
      int T = 0, U = 0;
      bool ok = true;
      KB_FOR_EACH_SPARSE_UNIT(args.plan, u, w, n, walk) {
        if (!ok) break;
        if (n == 0) continue;
        const int group = w.b * args.plan.Hkv + w.g;
        if (!is_v) {
          if (U > 0) ok = mbar_wait(bar(Cfg::kBarQDEmpty), (U - 1) & 1, abort_flag, err, kDevTimeoutSlot);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(Cfg::kBarQD), 2 * kTileBytes);
            tma_load_group(sbase + Cfg::kQOff, &tmap_q, w.t * kUnitRows, group, bar(Cfg::kBarQD));
            tma_load_group(sbase + Cfg::kDOOff, &tmap_do, w.t * kUnitRows, group, bar(Cfg::kBarQD));
          }
        }
        ++U;
        uint32_t next = __ldg(&walk[0].x);
        for (int j = 0; j < n; ++j, ++T) {
          const int slot = T % stages;
          const int block = static_cast<int>(next & kEntryBlock);
          if (j + 1 < n) next = __ldg(&walk[j + 1].x);
          if (T >= stages)
            ok = mbar_wait(bar(empty0 + slot), ((T / stages) - 1) & 1, abort_flag, err, kDevTimeoutSlot);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(full0 + slot), kTileBytes);
            tma_load_tile_hint(ring + slot * kTileBytes, tmap, block * kTileKeys, group, bar(full0 + slot), keep);
          }
        }
      }
      if (!ok && lane == 0) {
        if (!is_v && U > 0) drain_wait_b(bar(Cfg::kBarQD), (U - 1) & 1);
        for (int x = (T > stages ? T - stages : 0); x < T; ++x)
          drain_wait_b(bar(full0 + x % stages), (x / stages) & 1);
      }
    }
  } else if (warp == Cfg::kMmaWarp) {
    // ------------------------------------------------------ S, dP issuer
    // S(j+1), dP(j+1) go out as soon as the elementwise warps have read S(j),
    // dP(j); a second thread issues the dQ products, so neither stream's
    // barrier waits leave the tensor pipe idle.
    if (lane == 0 && !skip) {
      const uint32_t q_s = sbase + Cfg::kQOff, do_s = sbase + Cfg::kDOOff;
      int T = 0, U = 0;
      bool ok = true;
      KB_FOR_EACH_SPARSE_UNIT(args.plan, u, w, n, walk) {
        if (!ok) break;
        if (n == 0) continue;
        ok = mbar_wait(bar(Cfg::kBarQD), U & 1, abort_flag, err, kDevTimeoutTma);
        for (int j = 0; j < n && ok; ++j, ++T) {
          const int ks = T % Cfg::kKStages, vs = T % Cfg::kVStages;
          ok = mbar_wait_hint(bar(Cfg::kBarKFull + ks), (T / Cfg::kKStages) & 1, abort_flag, err, kDevTimeoutTma);
          if (ok) ok = mbar_wait_hint(bar(Cfg::kBarVFull + vs), (T / Cfg::kVStages) & 1, abort_flag, err, kDevTimeoutTma);
          if (ok && T > 0) ok = mbar_wait_hint(bar(Cfg::kBarSFree), (T - 1) & 1, abort_flag, err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
          // S's first K step goes out once S(j-1) has been read, the rest, with
          // dP's steps interleaved, once dP(j-1) has been read too
          const uint32_t k_s = sbase + Cfg::kKOff + ks * kTileBytes, v_s = sbase + Cfg::kVOff + vs * kTileBytes;
          mma_ss(tmem_base + Cfg::kColS, desc_kmajor(q_s, 0, 1024u, kSlabBytes), desc_kmajor(k_s, 0, 1024u, kSlabBytes),
                 kIdescQK, 0u);
          if (T > 0) ok = mbar_wait_hint(bar(Cfg::kBarDPFree), (T - 1) & 1, abort_flag, err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            mma_ss(tmem_base + Cfg::kColDP, desc_kmajor(do_s, kk, 1024u, kSlabBytes), desc_kmajor(v_s, kk, 1024u, kSlabBytes),
                   kIdescQK, kk > 0 ? 1u : 0u);
            if (kk < 7)
              mma_ss(tmem_base + Cfg::kColS, desc_kmajor(q_s, kk + 1, 1024u, kSlabBytes),
                     desc_kmajor(k_s, kk + 1, 1024u, kSlabBytes), kIdescQK, 1u);
            if (kk == 6) tc_commit(bar(Cfg::kBarSDone));             // S is complete before dP's last step
          }
          tc_commit(bar(Cfg::kBarSFull));
          tc_commit(bar(Cfg::kBarVEmpty + vs));
        }
        if (ok) tc_commit(bar(Cfg::kBarQDEmpty));
        ++U;
      }
      if (!ok) {
        tc_commit(bar(Cfg::kBarDrain));
        drain_wait_b(bar(Cfg::kBarDrain), 0);
      }
    }
  } else if (warp == Cfg::kDqWarp) {
    // ---------------------------------------------------------- dQ issuer
    // dQ(j) reads dS(j) and K(j); the K slot is released after it (S(j)
    // finished before dS(j) existed).
    if (lane == 0 && !skip) {
      int T = 0;
      bool ok = true;
      KB_FOR_EACH_SPARSE_UNIT(args.plan, u, w, n, walk) {
        if (!ok) break;
        // a unit's first dS comes after the same warps have read the last unit's dQ
        for (int j = 0; j < n && ok; ++j, ++T) {
          ok = mbar_wait_hint(bar(Cfg::kBarDSFull), T & 1, abort_flag, err, kDevTimeoutSoftmax);
          if (!ok) break;
          tc_fence_after();
          const int ks = T % Cfg::kKStages;
          issue_pv(tmem_base + Cfg::kColDQ, tmem_base + Cfg::kColDS, sbase + Cfg::kKOff + ks * kTileBytes, j == 0);
          issue_pv(tmem_base + Cfg::kColDQ, tmem_base + Cfg::kColDSLow, sbase + Cfg::kKOff + ks * kTileBytes, false);
          tc_commit(bar(Cfg::kBarDQDone));
          tc_commit(bar(Cfg::kBarKEmpty + ks));
        }
      }
      if (!ok) {
        tc_commit(bar(Cfg::kBarDrain + 1));
        drain_wait_b(bar(Cfg::kBarDrain + 1), 0);
      }
    }
  } else {
    // ------------------------------------------------------- elementwise
    // Warp w owns TMEM lanes 32(w%4) + 16(w/4) .. +15: rows r0 .. of head
    // w%4.  A thread holds the unit's rows r0 and r0 + 8 and, of each group of
    // 8 keys, keys 2u and 2u+1 (u = lane % 4), as the 16x256b load lays them out.
    const int head = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(32 * head + 16 * (warp >> 2)) << 16;
    const int u = lane & 3;
    const int r0 = 16 * (warp >> 2) + (lane >> 2);
    const uint32_t warp_rows = 0xFFFFu << (16 * (warp >> 2));
    const int S = args.plan.L;
    const float2 c2 = make_float2(score_scale_log2(), score_scale_log2());
    int T = 0;
    bool ok = !skip;
    KB_FOR_EACH_SPARSE_UNIT(args.plan, unit, w, n, walk) {
      if (!ok) break;
      const int p0 = w.t * kUnitRows - w.own * kTileKeys;               // the unit's first row within its own block
      const int iA = w.t * kUnitRows + r0, iB = iA + 8;                 // query positions
      const bool vA = iA < S, vB = iB < S;
      const size_t row0 = (static_cast<size_t>(w.b) * args.plan.Hq + w.g * kGroup + head) * static_cast<size_t>(S);
      // rows past the sequence list nothing, as do rows with lse = -inf: every
      // key of theirs is masked
      const float lseA = vA ? __fmul_rn(args.lse[row0 + iA], kLog2e) : 0.0f;
      const float lseB = vB ? __fmul_rn(args.lse[row0 + iB], kLog2e) : 0.0f;
      const float dlA = vA ? args.delta[row0 + iA] : 0.0f;
      const float dlB = vB ? args.delta[row0 + iB] : 0.0f;
      const float2 nlA = make_float2(-lseA, -lseA), nlB = make_float2(-lseB, -lseB);
      const float2 ndA = make_float2(-dlA, -dlA), ndB = make_float2(-dlB, -dlB);
      // a tile that some row of the warp did not list, and the own one, masks
      // keys from nA, nB on; the others take no select
      auto tile_ds = [&](auto mask_tag, const uint32_t (&sv)[32], const uint32_t (&pv)[32], int half, int nA, int nB,
                         uint32_t (&ds)[32], uint32_t (&low)[32]) {
        constexpr bool kMask = decltype(mask_tag)::value;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int key = 64 * half + 8 * r + 2 * u;                   // keys key, key + 1 within the tile
          const int at = 2 * (8 * half + r);
          ds_split_pair<kMask>(sv[4 * r], sv[4 * r + 1], pv[4 * r], pv[4 * r + 1], c2, nlA, ndA, key >= nA, key + 1 >= nA,
                               ds[at], low[at]);
          ds_split_pair<kMask>(sv[4 * r + 2], sv[4 * r + 3], pv[4 * r + 2], pv[4 * r + 3], c2, nlB, ndB, key >= nB,
                               key + 1 >= nB, ds[at + 1], low[at + 1]);
        }
      };
      uint2 next = n > 0 ? __ldg(&walk[0]) : make_uint2(0u, 0u);
      for (int j = 0; j < n && ok; ++j, ++T) {
        const uint2 entry = next;
        if (j + 1 < n) next = __ldg(&walk[j + 1]);
        ok = mbar_wait_hint(bar(Cfg::kBarSDone), T & 1, abort_flag, err, kDevTimeoutMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const bool diag = static_cast<int>(entry.x & kEntryBlock) == w.own;
        const int nA = (entry.y >> r0) & 1u ? (diag ? p0 + r0 + 1 : kTileKeys) : 0;
        const int nB = (entry.y >> (r0 + 8)) & 1u ? (diag ? p0 + r0 + 9 : kTileKeys) : 0;
        uint32_t ds[32], low[32];
        // all of S(j) and dP(j) into registers first, so S(j+1), dP(j+1) can be
        // issued while this tile's dS is computed: S as soon as it is complete
        // (before dP's last step), released on its own barrier so S(j+1) can
        // start while dP is still being read
        uint32_t sv0[32], pv0[32], sv1[32], pv1[32];
        tmem_ld_16x256b_x8_pair_wait(tmem_base + Cfg::kColS + lane_off, tmem_base + Cfg::kColS + lane_off + 64u, sv0,
                                     sv1);
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarSFree));                              // S(j) fully read
        ok = mbar_wait_hint(bar(Cfg::kBarSFull), T & 1, abort_flag, err, kDevTimeoutMma);   // dP(j) too
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_16x256b_x8_pair_wait(tmem_base + Cfg::kColDP + lane_off, tmem_base + Cfg::kColDP + lane_off + 64u, pv0,
                                     pv1);
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarDPFree));                             // dP(j) fully read
        if (diag || (entry.y & warp_rows) != warp_rows) {
          tile_ds(std::true_type{}, sv0, pv0, 0, nA, nB, ds, low);
          tile_ds(std::true_type{}, sv1, pv1, 1, nA, nB, ds, low);
        } else {
          tile_ds(std::false_type{}, sv0, pv0, 0, nA, nB, ds, low);
          tile_ds(std::false_type{}, sv1, pv1, 1, nA, nB, ds, low);
        }
        if (T > 0) {                                                   // dQ(j-1) has read dS(j-1)
          ok = mbar_wait(bar(Cfg::kBarDQDone), (T - 1) & 1, abort_flag, err, kDevTimeoutMma);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st_16x128b_x16(tmem_base + Cfg::kColDS + lane_off, ds);
        tmem_st_16x128b_x16(tmem_base + Cfg::kColDSLow + lane_off, low);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarDSFull));
      }
      if (ok && n > 0) ok = mbar_wait(bar(Cfg::kBarDQDone), (T - 1) & 1, abort_flag, err, kDevTimeoutMma);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        __nv_bfloat16* base = static_cast<__nv_bfloat16*>(args.dq) + row0 * kHeadDim;
        uint32_t* dA = reinterpret_cast<uint32_t*>(base + static_cast<size_t>(vA ? iA : 0) * kHeadDim);
        uint32_t* dB = reinterpret_cast<uint32_t*>(base + static_cast<size_t>(vB ? iB : 0) * kHeadDim);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t v[32];
          tmem_ld_16x256b_x8_wait(tmem_base + Cfg::kColDQ + lane_off + 64u * half, v);
          if (n == 0) {                                              // nothing listed: the gradient is zero
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int col = 64 * half + 8 * r + 2 * u;
            const uint32_t wa = pack_bf16x2(__fmul_rn(__uint_as_float(v[4 * r]), kInvSqrtD),
                                            __fmul_rn(__uint_as_float(v[4 * r + 1]), kInvSqrtD));
            const uint32_t wb = pack_bf16x2(__fmul_rn(__uint_as_float(v[4 * r + 2]), kInvSqrtD),
                                            __fmul_rn(__uint_as_float(v[4 * r + 3]), kInvSqrtD));
            if (vA) dA[col >> 1] = wa;
            if (vB) dB[col >> 1] = wb;
          }
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

// ----------------------------------------------------------- dk/dv kernel
//
// A step takes 32 positions that listed the key block, whichever units they
// come from, with their four heads: row 4r + h of the step's Q and dO tiles is
// head h of its r-th position, so no row of a step is idle but in the last
// one.  Four producer warps find the positions in the plan's row masks and
// copy their rows with 16-byte asynchronous copies into the swizzled tiles: a
// TMA box per position (four heads, 512 bytes) took 11,000 cycles a step, and
// whole units (all 32 rows of a unit of which some listed the block) 1.5 times
// the steps.  At S = 8192 with 16 blocks per row, without shared blocks and in
// order of the blocks: 565 us, against 1127 and 688 us; with both 452 us.
//
// Blocks differ in how many rows list them (the first block is kept by all),
// and one CTA for the longest would hold up the launch.  So a block of
// kSparseSplitSteps steps or more is shared by two CTAs, half of its steps each:
// both leave their fp32 sums in the workspace, and whichever is done last adds
// the other's to its own.  Neither waits, and a sum of two terms has one value
// in either order.  What is summed how depends on the block's rows alone, not
// on the batch or the width of the lists.  The shares are dealt longest first
// (kb_sparse_order_kernel).  Clusters of two CTAs per block, the second leaving
// at once where there is nothing to share, took 579 us against 565 without: a
// cluster needs two free SMs at a time.

// A job: x the (b, KV head), y the key block, whether it is shared, and which
// half this is.
constexpr uint32_t kJobSplit = 1u << 31, kJobSecond = 1u << 30, kJobBlock = kJobSecond - 1u;

// The launch's jobs, longest first, by one CTA: a counting sort on the number
// of steps (capped at 1023).  The order within one length is that of atomics;
// it decides only which SM runs what.  A few microseconds; blocks taken as they
// come left the last CTAs with 240 steps where 201 are the even share.
constexpr int kOrderThreads = 1024;
__global__ void __launch_bounds__(kOrderThreads, 1) kb_sparse_order_kernel(const SparseBwdArgs args) {
  __shared__ int first[kOrderThreads];                // per length (1023 - steps): jobs, then where they start
  __shared__ int warp_sum[kOrderThreads / 32];
  const int t = static_cast<int>(threadIdx.x), warp = t >> 5, lane = t & 31;
  const int groups = args.plan.B * args.plan.Hkv, blocks = args.plan.max_blocks;
  first[t] = 0;
  __syncthreads();
  auto each_job = [&](auto fn) {
    for (long long i = t; i < static_cast<long long>(groups) * blocks; i += kOrderThreads) {
      const int group = static_cast<int>(i / blocks), jt = static_cast<int>(i % blocks);
      const int steps = (__ldg(args.plan.row_counts + i) + kUnitRows - 1) / kUnitRows;
      const bool split = jt < args.n_split && steps >= kSparseSplitSteps;
      const int y = jt | (split ? static_cast<int>(kJobSplit) : 0);
      fn(split ? steps / 2 : steps, group, y);
      if (split) fn(steps - steps / 2, group, y | static_cast<int>(kJobSecond));
    }
  };
  each_job([&](int steps, int, int) { atomicAdd(&first[kOrderThreads - 1 - min(steps, kOrderThreads - 1)], 1); });
  __syncthreads();
  // exclusive sums over the lengths
  const int mine = first[t];
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  first[t] = before + upto - mine;
  if (t == kOrderThreads - 1) *args.n_jobs = before + upto;
  __syncthreads();
  each_job([&](int steps, int group, int y) {
    args.jobs[atomicAdd(&first[kOrderThreads - 1 - min(steps, kOrderThreads - 1)], 1)] = make_int2(group, y);
  });
}

struct SparseBwdKVCfg {
  static constexpr int kThreads = 416;        // 8 elementwise warps, 4 producers, the MMA issuer
  static constexpr int kLoadWarp0 = 8;
  static constexpr int kLoadWarps = 4;
  static constexpr int kMmaWarp = 12;
  static constexpr int kStages = 2;           // Q/dO ring
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColST = 0, kColDPT = 128, kColDV = 256, kColDK = 384;
  static constexpr uint32_t kKOff = 0;
  static constexpr uint32_t kVOff = kTileBytes;
  static constexpr uint32_t kQOff = 2 * kTileBytes;                   // slot s: Q at kQOff + s*2*tile,
  static constexpr uint32_t kSlotBytes = 2 * kTileBytes;              //         dO right after it
  static constexpr uint32_t kVecOff = kQOff + kStages * kSlotBytes;   // slot s: -lse2[128], -delta[128]
  static constexpr uint32_t kVecBytes = (2 * 128 + 32 + 4) * 4;       // ... the positions' places, "own block" flag
  static constexpr int kQueue = 32 + 1024;                            // positions found and not yet used, per producer warp
  static constexpr uint32_t kQueueOff = kVecOff + kStages * kVecBytes;
  static constexpr uint32_t kBarOff = kQueueOff + kLoadWarps * kQueue * 4;
  static constexpr int kBarKV = 0;                                    // K(jt), V(jt) landed
  static constexpr int kBarQDFull = 1;                                // 2: Q, dO of step s landed
  static constexpr int kBarQDEmpty = kBarQDFull + kStages;            // 2: dV, dK of step s done
  static constexpr int kBarVecFull = kBarQDEmpty + kStages;           // 2: lse2, delta of step s (32 arrivals)
  static constexpr int kBarSTFull = kBarVecFull + kStages;            // S^T, dP^T of step s in TMEM
  static constexpr int kBarPDSFull = kBarSTFull + 1;                  // 4: P^T, dS^T of query quarter 0..3
                                                                      //    stored (256 arrivals each)
  static constexpr int kBarDone = kBarPDSFull + 4;                    // every dV, dK product finished
  static constexpr int kBarDrain = kBarDone + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16 + 1024;
};

__global__ void __launch_bounds__(SparseBwdKVCfg::kThreads, 1)
kb_sparse_bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const SparseBwdArgs args) {
  using Cfg = SparseBwdKVCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kMiscOff);
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return smem_addr(bars + i); };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // this CTA's job: (b, KV head), key block and share of its steps
  if (static_cast<int>(blockIdx.x) >= __ldg(args.n_jobs)) return;
  const int2 job = __ldg(args.jobs + blockIdx.x);
  const int group = job.x;
  const int jt = job.y & static_cast<int>(kJobBlock);
  const int share = (job.y & static_cast<int>(kJobSecond)) ? 1 : 0;
  const int S = args.plan.L;
  const int n_tiles = args.plan.n_tiles;
  uint32_t* const err = args.plan.err;
  // rows that listed this block, as masks of the position tiles from the block's own on
  const uint32_t* const masks =
      args.plan.masks + (static_cast<size_t>(group) * args.plan.max_blocks + jt) * n_tiles;
  const int t0 = jt * (kTileKeys / kUnitRows);

  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kNumBars; ++i) {
      uint32_t count = 1u;
      if (i >= Cfg::kBarPDSFull && i < Cfg::kBarPDSFull + 4) count = 256u;
      if (i >= Cfg::kBarVecFull && i < Cfg::kBarVecFull + Cfg::kStages) count = 32u;
      if (i >= Cfg::kBarQDFull && i < Cfg::kBarQDFull + Cfg::kStages) count = 32u * Cfg::kLoadWarps;
      mbar_init(bar(i), count);
    }
    misc[1] = (*reinterpret_cast<volatile uint32_t*>(err) != 0) ? 1u : 0u;
    fence_mbar_init();
  }
  const int n_rows = __ldg(args.plan.row_counts + static_cast<size_t>(group) * args.plan.max_blocks + jt);
  const int block_steps = (n_rows + kUnitRows - 1) / kUnitRows;
  const bool split = job.y < 0;                       // kJobSplit
  const int step0 = share ? (split ? block_steps / 2 : block_steps) : 0;
  const int n_steps = (split && !share ? block_steps / 2 : block_steps) - step0;

  if (warp == Cfg::kMmaWarp) {
    __syncwarp();
    tmem_alloc(sbase + Cfg::kMiscOff, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];
  const bool skip = (*abort_flag != 0);

  if (warp >= Cfg::kLoadWarp0 && warp < Cfg::kLoadWarp0 + Cfg::kLoadWarps) {
    // ----------------------------------------------------------- producers
    // Every warp finds the step's positions for itself and copies the rows of
    // eight of them.
    if (!skip) {
      const int lw = warp - Cfg::kLoadWarp0;
      if (lw == 0 && lane == 0) {
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        if (n_steps > 0) {
          mbar_arrive_expect_tx(bar(Cfg::kBarKV), 2 * kTileBytes);
          tma_load_tile(sbase + Cfg::kKOff, &tmap_k, jt * kTileKeys, group, bar(Cfg::kBarKV));
          tma_load_tile(sbase + Cfg::kVOff, &tmap_v, jt * kTileKeys, group, bar(Cfg::kBarKV));
        }
      }
      bool ok = true;
      int* queue = reinterpret_cast<int*>(smem + Cfg::kQueueOff) + lw * Cfg::kQueue;
      int tb = t0, queued = 0, used = 0;                               // next masks; the queue holds used .. queued-1
      int skip_rows = step0 * kUnitRows;                               // positions of the share before this one
      for (int s = 0; s < n_steps; ++s) {
        const int slot = s % Cfg::kStages;
        // the next 32 positions: what is left moves to the front, then the
        // set bits of 32 masks at a time join it
        while (queued - used < kUnitRows && tb < n_tiles) {
          const int rest = queued - used;
          const int keep_pos = lane < rest ? queue[used + lane] : 0;
          __syncwarp();
          if (lane < rest) queue[lane] = keep_pos;
          // at once, not only when the window adds positions: a window without any
          // would let the next one move from where this move has written
          used = 0;
          queued = rest;
          uint32_t m = tb + lane < n_tiles ? __ldg(masks + tb + lane) : 0u;
          int at = __popc(m);
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += v;
          }
          const int total = __shfl_sync(0xffffffffu, at, 31);
          tb += 32;
          if (total <= skip_rows) {                                    // all of the other share's, or an empty window
            skip_rows -= total;
            continue;
          }
          at += rest - __popc(m);
          for (; m != 0u; m &= m - 1u) queue[at++] = (tb - 32 + lane) * kUnitRows + __ffs(m) - 1;
          __syncwarp();
          used = skip_rows;                                            // > 0 only where the share begins: rest is 0 there
          skip_rows = 0;
          queued = rest + total;
        }
        // a step short of positions is filled up with rows past the sequence,
        // which read as zeros; a position there was not listed by this call
        int pos = lane < queued - used ? queue[used + lane] : S;
        const bool listed = pos < S;
        if (!listed) pos = S;
        used = min(queued, used + kUnitRows);
        if (s >= Cfg::kStages)
          ok = mbar_wait(bar(Cfg::kBarQDEmpty + slot), ((s / Cfg::kStages) - 1) & 1, abort_flag, err,
                         kDevTimeoutSlot);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // 16 lanes a row, two rows a copy: rows 32 lw .. 32 lw + 31 of both tiles
        const int c = lane & 15;
        const uint32_t dst = sbase + Cfg::kQOff + slot * Cfg::kSlotBytes + static_cast<uint32_t>(c >> 3) * kSlabBytes;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int row = 32 * lw + 2 * k + (lane >> 4);
          const int p = __shfl_sync(0xffffffffu, pos, 8 * lw + (k >> 1));
          const uint32_t size = p < S ? 16u : 0u;                      // a filler row is written as zeros
          const size_t from = ((static_cast<size_t>(group) * kGroup + (row & 3)) * static_cast<size_t>(S) + (p < S ? p : 0)) *
                                  kHeadDim + 8 * c;
          const uint32_t at = dst + static_cast<uint32_t>((row >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4));
          cp_async16(at, static_cast<const __nv_bfloat16*>(args.q) + from, size);
          cp_async16(at + kTileBytes, static_cast<const __nv_bfloat16*>(args.dout) + from, size);
        }
        // -lse (base 2) and -delta of the step's 128 query rows; a filler gets
        // -lse2 = -inf, so its P (and dS) is exactly zero
        if (lw == 0) {
          float* vec = reinterpret_cast<float*>(smem + Cfg::kVecOff + slot * Cfg::kVecBytes);
          float nl[kGroup], nd[kGroup];
  #pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            const size_t at = (static_cast<size_t>(group) * kGroup + h) * static_cast<size_t>(S) + pos;
            nl[h] = listed ? -__fmul_rn(args.lse[at], kLog2e) : __int_as_float(0xFF800000);
            nd[h] = listed ? -args.delta[at] : -0.0f;
          }
          reinterpret_cast<float4*>(vec)[lane] = make_float4(nl[0], nl[1], nl[2], nl[3]);
          reinterpret_cast<float4*>(vec + 128)[lane] = make_float4(nd[0], nd[1], nd[2], nd[3]);
          // the position's place in the key block, if the block is its own
          const int place = pos - jt * kTileKeys;
          reinterpret_cast<int*>(vec)[256 + lane] = place;
          const uint32_t own = __ballot_sync(0xffffffffu, place < kTileKeys);
          if (lane == 0) reinterpret_cast<uint32_t*>(vec)[288] = own;
          mbar_arrive(bar(Cfg::kBarVecFull + slot));
        }
        cp_async_wait();
        fence_proxy_async_smem();                                      // the copies -> visible to the tensor core
        mbar_arrive(bar(Cfg::kBarQDFull + slot));
      }
      if (!ok && lw == 0 && lane == 0) drain_wait_b(bar(Cfg::kBarKV), 0);
    }
  } else if (warp == Cfg::kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    // per step: S^T = K Q^T, dP^T = V dO^T, then for each quarter of the
    // query columns (32 queries), once its P^T and dS^T are stored, K steps
    // 2q and 2q+1 of dV += P^T dO and dK += dS^T Q.  A quarter's steps read
    // only the columns that quarter wrote, so they run while the next quarter
    // is computed.  P^T and dS^T overwrite S^T and dP^T, whose next values are
    // issued after these products (in issue order).
    if (lane == 0 && !skip) {
      bool ok = n_steps == 0 || mbar_wait(bar(Cfg::kBarKV), 0, abort_flag, err, kDevTimeoutTma);
      for (int s = 0; s < n_steps && ok; ++s) {
        const int slot = s % Cfg::kStages;
        const uint32_t q_s = sbase + Cfg::kQOff + slot * Cfg::kSlotBytes;
        const uint32_t do_s = q_s + kTileBytes;
        ok = mbar_wait_hint(bar(Cfg::kBarQDFull + slot), (s / Cfg::kStages) & 1, abort_flag, err, kDevTimeoutTma);
        if (!ok) break;
        tc_fence_after();
        issue_qk_pair(tmem_base + Cfg::kColST, sbase + Cfg::kKOff, q_s, tmem_base + Cfg::kColDPT, sbase + Cfg::kVOff,
                      do_s);
        tc_commit(bar(Cfg::kBarSTFull));
        ok = mbar_wait_hint(bar(Cfg::kBarPDSFull), s & 1, abort_flag, err, kDevTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        issue_pv_pair<0, 2>(tmem_base + Cfg::kColDV, tmem_base + Cfg::kColST, do_s, tmem_base + Cfg::kColDK,
                            tmem_base + Cfg::kColDPT, q_s, s == 0);
        ok = mbar_wait_hint(bar(Cfg::kBarPDSFull + 1), s & 1, abort_flag, err, kDevTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        issue_pv_pair<2, 4>(tmem_base + Cfg::kColDV, tmem_base + Cfg::kColST, do_s, tmem_base + Cfg::kColDK,
                            tmem_base + Cfg::kColDPT, q_s, false);
        ok = mbar_wait_hint(bar(Cfg::kBarPDSFull + 2), s & 1, abort_flag, err, kDevTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        issue_pv_pair<4, 6>(tmem_base + Cfg::kColDV, tmem_base + Cfg::kColST, do_s, tmem_base + Cfg::kColDK,
                            tmem_base + Cfg::kColDPT, q_s, false);
        ok = mbar_wait_hint(bar(Cfg::kBarPDSFull + 3), s & 1, abort_flag, err, kDevTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        issue_pv_pair<6, 8>(tmem_base + Cfg::kColDV, tmem_base + Cfg::kColST, do_s, tmem_base + Cfg::kColDK,
                            tmem_base + Cfg::kColDPT, q_s, false);
        tc_commit(bar(Cfg::kBarQDEmpty + slot));
      }
      if (ok) tc_commit(bar(Cfg::kBarDone));
      if (!ok) {
        tc_commit(bar(Cfg::kBarDrain));
        drain_wait_b(bar(Cfg::kBarDrain), 0);
      }
    }
  } else {
    // ------------------------------------------------------- elementwise
    // rows are keys (lanes as in the dq kernel), columns are query rows
    const int lane_base = 32 * (warp & 3) + 16 * (warp >> 2);
    const uint32_t lane_off = static_cast<uint32_t>(lane_base) << 16;
    const int u = lane & 3;
    const int rA = lane_base + (lane >> 2);
    const int rB = rA + 8;
    const float2 c2 = make_float2(score_scale_log2(), score_scale_log2());
    // one query quarter (eight positions): a step with positions of the block
    // itself masks keys past them, the others take no select
    auto quarter = [&](auto diag_tag, const uint32_t (&sv)[16], const uint32_t (&pv)[16], const float* vnl,
                       const float* vnd, int qt, const int* place, uint32_t (&pp)[8], uint32_t (&dd)[8]) {
      constexpr bool kDiag = decltype(diag_tag)::value;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int qc = 32 * qt + 8 * r + 2 * u;                      // query rows qc, qc + 1 within their tile
        const float2 nl = *reinterpret_cast<const float2*>(vnl + qc);
        const float2 nd = *reinterpret_cast<const float2*>(vnd + qc);
        const int at = kDiag ? place[qc >> 2] : 0;                   // both columns are heads of one position
        p_ds_pair<kDiag>(sv[4 * r], sv[4 * r + 1], pv[4 * r], pv[4 * r + 1], c2, nl, nd, rA > at, rA > at,
                         pp[2 * r], dd[2 * r]);
        p_ds_pair<kDiag>(sv[4 * r + 2], sv[4 * r + 3], pv[4 * r + 2], pv[4 * r + 3], c2, nl, nd, rB > at,
                         rB > at, pp[2 * r + 1], dd[2 * r + 1]);
      }
    };
    bool ok = !skip;
    for (int s = 0; s < n_steps && ok; ++s) {
      const int slot = s % Cfg::kStages;
      ok = mbar_wait_hint(bar(Cfg::kBarSTFull), s & 1, abort_flag, err, kDevTimeoutMma);
      if (ok) ok = mbar_wait_hint(bar(Cfg::kBarVecFull + slot), (s / Cfg::kStages) & 1, abort_flag, err,
                             kDevTimeoutTma);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float* vnl = reinterpret_cast<const float*>(smem + Cfg::kVecOff + slot * Cfg::kVecBytes);
      const float* vnd = vnl + 128;
      const int* place = reinterpret_cast<const int*>(vnl) + 256;
      const bool diag = reinterpret_cast<const uint32_t*>(vnl)[288] != 0u;
#pragma unroll
      for (int qt = 0; qt < 4; ++qt) {                                 // query quarter: 32 query columns
        uint32_t sv[16], pv[16];
        tmem_ld_16x256b_x4_pair_wait(tmem_base + Cfg::kColST + lane_off + 32u * qt,
                                     tmem_base + Cfg::kColDPT + lane_off + 32u * qt, sv, pv);
        uint32_t pp[8], dd[8];
        if (diag) quarter(std::true_type{}, sv, pv, vnl, vnd, qt, place, pp, dd);
        else quarter(std::false_type{}, sv, pv, vnl, vnd, qt, place, pp, dd);
        // bf16 pairs of query columns 32*qt.. go to columns 16*qt.. of the
        // same buffers; those fp32 columns were read in this quarter or an
        // earlier one
        tmem_st_16x128b_x4(tmem_base + Cfg::kColST + lane_off + 16u * qt, pp);
        tmem_st_16x128b_x4(tmem_base + Cfg::kColDPT + lane_off + 16u * qt, dd);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(Cfg::kBarPDSFull + qt));
      }
    }
    if (ok) ok = mbar_wait(bar(Cfg::kBarDone), 0, abort_flag, err, kDevTimeoutMma);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    // A shared block: this thread's sums, part by part (dv's halves, then
    // dk's), as a float4 of registers 4r .. 4r+3 per r
    float4* const sums = args.sums + ((static_cast<size_t>(group) * args.n_split + jt) * 2) * (32 * 256);
    bool writes = ok && (share == 0 || split);
    if (split) {                                                     // every elementwise warp meets the barriers
      float4* const mine = sums + share * (32 * 256);
#pragma unroll 1
      for (int part = 0; part < 4 && ok; ++part) {
        uint32_t v[32];
        tmem_ld_16x256b_x8_wait(tmem_base + (part < 2 ? Cfg::kColDV : Cfg::kColDK) + lane_off + 64u * (part & 1), v);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          mine[(8 * part + r) * 256 + threadIdx.x] =
              make_float4(__uint_as_float(v[4 * r]), __uint_as_float(v[4 * r + 1]), __uint_as_float(v[4 * r + 2]),
                          __uint_as_float(v[4 * r + 3]));
      }
      // all 256 threads' sums, then one ticket: the second to draw finds the
      // other CTA's sums complete
      __threadfence();
      named_bar_sync(1u, 256u);
      if (threadIdx.x == 0) {
        misc[3] = *abort_flag != 0 ? 0u
                                   : static_cast<uint32_t>(
                                         atomicAdd(args.tickets + static_cast<size_t>(group) * args.n_split + jt, 1));
        __threadfence();
      }
      named_bar_sync(1u, 256u);
      writes = writes && misc[3] == 1u;
    }
    if (writes) {
      const int jA = jt * kTileKeys + rA, jB = jt * kTileKeys + rB;
      const bool vA = jA < S, vB = jB < S;
      const size_t kv0 = static_cast<size_t>(group) * static_cast<size_t>(S);
      const float4* const theirs = sums + (1 - share) * (32 * 256);
#pragma unroll 1
      for (int part = 0; part < 4; ++part) {                         // dk is scaled by 1/sqrt(128)
        const int which = part >> 1, half = part & 1;
        __nv_bfloat16* base = static_cast<__nv_bfloat16*>(which ? args.dk : args.dv) + kv0 * kHeadDim;
        uint32_t* oA = reinterpret_cast<uint32_t*>(base + static_cast<size_t>(vA ? jA : 0) * kHeadDim);
        uint32_t* oB = reinterpret_cast<uint32_t*>(base + static_cast<size_t>(vB ? jB : 0) * kHeadDim);
        const float sc = which ? kInvSqrtD : 1.0f;
        uint32_t v[32];
        tmem_ld_16x256b_x8_wait(tmem_base + (which ? Cfg::kColDK : Cfg::kColDV) + lane_off + 64u * half, v);
        if (n_steps == 0) {                                          // listed by nobody: the gradient is zero
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (split) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float4 x = __ldcg(theirs + (8 * part + r) * 256 + threadIdx.x);
            v[4 * r] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * r]), x.x));
            v[4 * r + 1] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * r + 1]), x.y));
            v[4 * r + 2] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * r + 2]), x.z));
            v[4 * r + 3] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * r + 3]), x.w));
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int col = 64 * half + 8 * r + 2 * u;
          const uint32_t wa = pack_bf16x2(__fmul_rn(__uint_as_float(v[4 * r]), sc),
                                          __fmul_rn(__uint_as_float(v[4 * r + 1]), sc));
          const uint32_t wb = pack_bf16x2(__fmul_rn(__uint_as_float(v[4 * r + 2]), sc),
                                          __fmul_rn(__uint_as_float(v[4 * r + 3]), sc));
          if (vA) oA[col >> 1] = wa;
          if (vB) oB[col >> 1] = wb;
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

// --------------------------------------------------------------- launcher

cudaError_t launch_sparse_backward(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CUtensorMap& tdo, const SparseBwdArgs& a, int device, int sm_count,
                                   cudaStream_t s) {
  static_assert(SparseBwdQCfg::kSmemBytes <= 227u * 1024u, "shared memory budget (dq)");
  static_assert(SparseBwdKVCfg::kSmemBytes <= 227u * 1024u, "shared memory budget (dk, dv)");
  static bool configured[64] = {};
  cudaError_t e;
  if (!configured[device]) {
    e = cudaFuncSetAttribute(kb_sparse_bwd_dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(SparseBwdQCfg::kSmemBytes));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kb_sparse_bwd_dkdv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(SparseBwdKVCfg::kSmemBytes));
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  kb_sparse_bwd_dq_kernel<<<static_cast<unsigned>(unit_grid(a.plan, sm_count, 32)), SparseBwdQCfg::kThreads,
                            SparseBwdQCfg::kSmemBytes, s>>>(tq, tk, tv, tdo, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kb_sparse_order_kernel<<<1, kOrderThreads, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid_kv = static_cast<unsigned>((a.plan.max_blocks + a.n_split) * a.plan.B * a.plan.Hkv);
  kb_sparse_bwd_dkdv_kernel<<<grid_kv, SparseBwdKVCfg::kThreads, SparseBwdKVCfg::kSmemBytes, s>>>(tk, tv, a);
  return cudaGetLastError();
}

}  // namespace kb

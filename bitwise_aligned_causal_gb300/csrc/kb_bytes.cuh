// kb_bytes.cuh -- bringing the tiles of a KV cache held in 8 bits to shared
// memory, for the kernels that attend over it (kb_decode.cu, kb_decode8.cu).
#pragma once

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

// mbar_wait with one test in line and the rest out of line: the kernel's
// twenty waits would otherwise spread its warps' loops over more code than the
// instruction cache holds.
static __device__ __noinline__ bool wait_far(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* err, uint32_t code) {
  return mbar_wait(bar, parity, abort_flag, err, code);
}
__device__ __forceinline__ bool wait_near(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* err, uint32_t code) {
  return mbar_try_wait_hint(bar, parity, 200u) || wait_far(bar, parity, abort_flag, err, code);
}

__device__ __forceinline__ void drain_bytes(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 50000000ull) break;
}

static __device__ __noinline__ void drain_far(uint32_t bar, uint32_t parity) { drain_bytes(bar, parity); }

// Rows 128 j .. of sequence b, KV head g: the row of the byte map and its
// plane, and the place of the block's exponent.  False for a page index out of
// range (reported; the map reads zeros there).
__device__ __forceinline__ bool byte_tile(const PackedArgs& a, int b, int g, int j, int& row, int& plane, size_t& e_at) {
  const int key = j * kTileKeys;
  const int blocks = (a.plane_rows + kTileKeys - 1) / kTileKeys;
  bool ok = true;
  if (a.block_table == nullptr) {
    row = key;
    plane = b * a.Hkv + g;
  } else {
    int pg = __ldg(a.block_table + static_cast<size_t>(b) * a.pages_per_seq + key / a.page_size);
    if (pg < 0 || pg >= a.num_pages) {
      atomicCAS(a.err, 0u, static_cast<uint32_t>(kDevBadInput));
      pg = a.num_pages;
      ok = false;
    }
    row = key % a.page_size;
    plane = pg * a.Hkv + g;
  }
  e_at = ok ? static_cast<size_t>(plane) * blocks + row / kTileKeys : 0;
  return ok;
}

// One warp: tiles j0 .. j0 + nt - 1 of sequence b, KV head g, K's and V's bytes
// by turns, each into its ring of kStages staged tiles (16 KB, 128-byte
// swizzle), their exponents beside them (`held`: K's stages, then V's).
// full0: barriers of landed tiles, K's stages, then V's; read0: the same for
// tiles that have been read.  Lane l looks up the page and the exponents of
// tile l of the next 32, so that no load's latency is waited for.  kFar: waits
// out of line (not in a kernel that moves registers between its warps).
template <int kStages, bool kFar>
__device__ __forceinline__ void produce_bytes(const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, const PackedArgs& args,
                                              int b, int g, int j0, int nt, uint32_t k_staged, uint32_t v_staged, int* held,
                                              uint32_t full0, uint32_t read0, volatile uint32_t* abort_flag) {
  constexpr uint32_t kBytes = kTileBytes / 2;
  const int lane = static_cast<int>(threadIdx.x & 31u);
  if (lane == 0) {
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  const uint64_t stream_once = l2_policy_evict_first();
  struct Place {
    int row, plane, ke, ve;
  };
  auto look_up = [&](int jj) {
    Place p{0, 0, 0, 0};
    size_t e_at = 0;
    if (jj < nt && byte_tile(args, b, g, j0 + jj, p.row, p.plane, e_at)) {
      p.ke = args.k_exp[e_at];
      p.ve = args.v_exp[e_at];
    }
    return p;
  };
  Place cur{}, next = look_up(lane);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return kFar ? wait_near(bar, parity, abort_flag, args.err, kDevTimeoutSlot) : mbar_wait(bar, parity, abort_flag, args.err, kDevTimeoutSlot);
  };
  int k_issued = 0, v_issued = 0;
  bool ok = true;
  for (int jj = 0; jj < nt && ok; ++jj) {
    if ((jj & 31) == 0) {
      cur = next;
      next = look_up(jj + 32 + lane);
    }
    const int from = jj & 31, st = jj % kStages;
    const int row = __shfl_sync(0xffffffffu, cur.row, from), plane = __shfl_sync(0xffffffffu, cur.plane, from);
    const int ke = __shfl_sync(0xffffffffu, cur.ke, from), ve = __shfl_sync(0xffffffffu, cur.ve, from);
    if (lane == 0) {
      if (jj >= kStages) ok = wait(read0 + 8u * st, (jj / kStages - 1) & 1);
      if (ok) {
        held[st] = ke;
        mbar_arrive_expect_tx(full0 + 8u * st, kBytes);
        tma_load_3d_hint(k_staged + st * kBytes, &tmap_k, 0, row, plane, full0 + 8u * st, stream_once);
        k_issued = jj + 1;
        if (jj >= kStages) ok = wait(read0 + 8u * (kStages + st), (jj / kStages - 1) & 1);
      }
      if (ok) {
        held[kStages + st] = ve;
        mbar_arrive_expect_tx(full0 + 8u * (kStages + st), kBytes);
        tma_load_3d_hint(v_staged + st * kBytes, &tmap_v, 0, row, plane, full0 + 8u * (kStages + st), stream_once);
        v_issued = jj + 1;
      }
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  }
  // no copy is in flight when the CTA leaves, whoever gave up
  auto drain = [](uint32_t bar, uint32_t parity) { kFar ? drain_far(bar, parity) : drain_bytes(bar, parity); };
  if (lane == 0) {
    for (int x = max(0, k_issued - kStages); x < k_issued; ++x) drain(full0 + 8u * (x % kStages), (x / kStages) & 1);
    for (int x = max(0, v_issued - kStages); x < v_issued; ++x) drain(full0 + 8u * (kStages + x % kStages), (x / kStages) & 1);
  }
}

}  // namespace kb

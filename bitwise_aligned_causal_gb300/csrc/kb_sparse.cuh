// kb_sparse.cuh -- what the block-sparse kernels share: the plan that turns
// per-row block lists into per-tile walks, and the units.
//
// A unit is 32 query positions (aligned to absolute multiples of 32) of one
// KV head with its four query heads: 128 rows of one MMA tile, row
// 32 * head + r.  The 32 positions lie in one key block, the unit's own.  The
// unit walks the union of its rows' lists in ascending order; entry e of the
// walk is a key block and a mask whose bit r says that row r listed it.
#pragma once

#include <cstdint>

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

constexpr int kUnitRows = 32;
constexpr uint32_t kEntrySegStart = 1u << 30;   // first entry of its C5 segment in this walk
constexpr uint32_t kEntrySegEnd = 1u << 31;     // last entry of its C5 segment in this walk
constexpr uint32_t kEntryBlock = kEntrySegStart - 1u;

struct SparseUnit {
  int b, g;              // batch, KV head
  int t;                 // absolute position tile: positions 32t .. 32t+31
  int own;               // the key block they lie in
  int start, L;          // the sequence's first query position and row count
  int kv_len;            // start + L
  bool live;
};

// Unit `u` of the launch: (b, KV head) slowest, so the units that run at one
// time share a group's K and V in L2; the last positions first (they can
// have the longest walks).
__device__ __forceinline__ SparseUnit sparse_unit(const SparseArgs& a, int u) {
  SparseUnit w;
  const int bg = u / a.n_tiles;
  const int rank = u % a.n_tiles;
  w.b = bg / a.Hkv;
  w.g = bg % a.Hkv;
  w.start = a.starts != nullptr ? a.starts[w.b] : a.start;
  w.L = a.lens != nullptr ? a.lens[w.b] : a.L;
  w.live = w.start >= 0 && w.L >= 1 && w.L <= a.L && w.start <= a.kv_cap - w.L;
  const int first = w.live ? w.start / kUnitRows : 0;
  const int n = w.live ? (w.start + w.L - 1) / kUnitRows - first + 1 : 0;
  w.live = w.live && rank < n;
  w.t = first + n - 1 - rank;
  w.own = w.t * kUnitRows / kTileKeys;
  w.kv_len = w.start + w.L;
  return w;
}

// Units of a CTA: one of every gridDim.x, in alternating direction, so that
// CTAs with late units of one round have early ones of the next.
__device__ __forceinline__ int unit_of_turn(int turn) {
  const int grid = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  return turn * grid + ((turn & 1) ? grid - 1 - c : c);
}

__device__ __forceinline__ const uint2* unit_walk(const SparseArgs& a, int u) {
  return a.walks + static_cast<size_t>(u) * a.walk_cap;
}

// Every role of a CTA walks the same units in the same order: unit u, its
// SparseUnit w, its walk and the walk's length n (>= 0; absent units are passed
// over).
#define KB_FOR_EACH_SPARSE_UNIT(plan, u, w, n, walk)                                                       \
  for (int turn = 0, u = unit_of_turn(0); turn * static_cast<int>(gridDim.x) < (plan).n_units;             \
       u = unit_of_turn(++turn))                                                                           \
    if (const int n = u < (plan).n_units ? __ldg((plan).walk_len + u) : -1; n >= 0)                        \
      if (const SparseUnit w = sparse_unit(plan, u); true)                                                 \
        if (const uint2* const walk = unit_walk(plan, u); true)

// CTAs for a plan's units: one per SM that goes from unit to unit, its rings
// and TMEM already set up, where that leaves SMs idle for at most 1/`part` of the
// units' time; else one per unit, as SMs come free.  Forward (part 16): 13.5
// units per SM 338 us against 352 with a CTA per unit, 9.9 117 against 135, 3.4
// 250 against 234.  dq (part 32), whose start costs less, by the whole gradient:
// 13.5 units per SM (8192 rows) 1304 us against 1222, 9.9 (3 x 1999) 358 against
// 379, 8.0 (4864) 582 against 579.
inline int unit_grid(const SparseArgs& a, int sm_count, int part) {
  const long long idle = (static_cast<long long>(a.n_units) + sm_count - 1) / sm_count * sm_count - a.n_units;
  return a.n_units > sm_count && idle * part <= a.n_units ? sm_count : a.n_units;
}

// TMA box of query rows packed by GQA group (host_group_map): 32 rows of the
// four heads of group `group`.
__device__ __forceinline__ void tma_load_group(uint32_t dst, const void* tmap, int row, int group, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(row), "r"(0), "r"(0), "r"(group), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_group_hint(uint32_t dst, const void* tmap, int row, int group, uint32_t bar,
                                                    uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(row), "r"(0), "r"(0), "r"(group), "r"(bar),
        "l"(policy)
      : "memory");
}

// Asynchronous copy of 16 bytes into shared memory, `size` (0 or 16) of them
// from global memory and zeros after that.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
// Wait for every such copy of this thread.
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace kb

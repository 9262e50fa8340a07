// kb_sparse_plan.cu -- the plan of a block-sparse call: for every unit (32
// positions of one KV head, kb_sparse.cuh) the union of its rows' block lists
// in ascending order, each with the mask of the rows that listed it.
//
// One CTA per unit keeps a row mask per key block in shared memory, so lists
// may come in any order and name a block twice; blocks past a row's own are
// dropped, since none of their keys is visible to it.  The lists are read
// once (4 bytes an entry) and the walk written once (8 bytes): 6.6 us for 512
// units and 512 blocks, 10.8 us for 2048 units and 64, beside 235 and 337 us of
// attention; bound by the latency of its steps.
#include "kb_sparse.cuh"

namespace kb {

constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) kb_sparse_plan_kernel(const SparseArgs args) {
  extern __shared__ uint32_t row_mask[];              // per key block 0..own
  __shared__ int warp_count[kPlanThreads / 32];
  const int u = static_cast<int>(blockIdx.x);
  // one decision for the CTA: the word may change while its threads read it
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(args.err) != 0)) {
    // the attention kernel must not walk what an earlier call left here, even
    // if the error word is cleared before it starts
    if (threadIdx.x == 0) args.walk_len[u] = -1;
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SparseUnit w = sparse_unit(args, u);
  if (!w.live) {
    // a start or length out of range (an absent unit of a shorter sequence is none)
    if (threadIdx.x == 0) {
      if (w.L < 0 || w.L > args.L || w.start < 0 || w.start > args.kv_cap - w.L)
        atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
      args.walk_len[u] = -1;
    }
    return;
  }
  const int nb = w.own + 1;
  for (int j = threadIdx.x; j < nb; j += kPlanThreads) row_mask[j] = 0u;
  __syncthreads();
  const int i0 = w.t * kUnitRows - w.start;           // row index of the unit's first position (may be negative)
  const int* lists = args.blocks + ((static_cast<size_t>(w.b) * args.Hkv + w.g) * args.L + max(i0, 0)) * args.n_select;
  const int n_cap = (args.kv_cap + kTileKeys - 1) / kTileKeys;
  // the unit's rows lie one after another; entry e of them is of row `r`
  const int r0 = max(0, -i0), rows = min(kUnitRows - r0, w.L - max(i0, 0));
  int r = r0 + static_cast<int>(threadIdx.x) / args.n_select, k = static_cast<int>(threadIdx.x) % args.n_select;
  const int r_step = kPlanThreads / args.n_select, k_step = kPlanThreads % args.n_select;
  for (int e = threadIdx.x; e < rows * args.n_select; e += kPlanThreads) {
    const int j = __ldg(lists + e);
    if (j < -1 || j >= n_cap) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
    else if (j >= 0 && j <= w.own) atomicOr(&row_mask[j], 1u << r);
    r += r_step;
    k += k_step;
    if (k >= args.n_select) {
      k -= args.n_select;
      ++r;
    }
  }
  __syncthreads();
  if (args.masks != nullptr) {
    int* counts = args.row_counts + (static_cast<size_t>(w.b) * args.Hkv + w.g) * args.max_blocks;
    uint32_t* m = args.masks + (static_cast<size_t>(w.b) * args.Hkv + w.g) * args.max_blocks * args.n_tiles + w.t;
    for (int j = threadIdx.x; j < nb; j += kPlanThreads) {
      m[static_cast<size_t>(j) * args.n_tiles] = row_mask[j];
      if (row_mask[j] != 0u) atomicAdd(counts + j, __popc(row_mask[j]));     // whole numbers: any order
    }
  }
  uint2* walk = args.walks + static_cast<size_t>(u) * args.walk_cap;
  int n = 0;                                          // entries of the blocks before j0
  for (int j0 = 0; j0 < nb; j0 += kPlanThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t m = j < nb ? row_mask[j] : 0u;
    const uint32_t any = __ballot_sync(0xffffffffu, m != 0u);
    if (lane == 0) warp_count[warp] = __popc(any);
    __syncthreads();
    int at = n;
#pragma unroll
    for (int k = 0; k < kPlanThreads / 32; ++k) {
      const int c = warp_count[k];
      if (k < warp) at += c;
      n += c;
    }
    if (m != 0u) {
      // the warp's 32 blocks are four whole segments
      const uint32_t seg = (any >> (lane & ~(kSegTiles - 1))) & ((1u << kSegTiles) - 1u), place = lane % kSegTiles;
      const bool first = (seg & ((1u << place) - 1u)) == 0u, last = (seg >> place) == 1u;
      walk[at + __popc(any & ((1u << lane) - 1u))] =
          make_uint2(static_cast<uint32_t>(j) | (first ? kEntrySegStart : 0u) | (last ? kEntrySegEnd : 0u), m);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) args.walk_len[u] = n;
}

cudaError_t launch_sparse_plan(const SparseArgs& a, int device, cudaStream_t s) {
  static bool configured[64] = {};
  if (!configured[device]) {
    const cudaError_t e = cudaFuncSetAttribute(kb_sparse_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  const int blocks = a.max_blocks;
  kb_sparse_plan_kernel<<<static_cast<unsigned>(a.n_units), kPlanThreads, static_cast<size_t>(blocks) * 4, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kb

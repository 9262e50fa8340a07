// kb_evict.cu -- cutting a cache to its heaviest keys, in place.
//
// Choice.  A cluster of CTAs per (batch, KV head), as many (1 to 8) as find
// SMs.  Weights become whole numbers in the order of their values (a NaN above
// all), the threshold is found digit by digit (11, 11 and 10 bits, a histogram
// each, summed over the cluster through distributed shared memory), and of the
// keys that equal it the lowest rows are kept.  A CTA reads its run of rows
// from memory once, into shared memory; its warps own contiguous runs of it:
// each counts its keys above and at the threshold, a scan over warps and CTAs
// gives every run its place, and a second walk writes the kept rows and their
// weights in order.  Runs that do not fit (caches of more than 40960 keys a
// CTA) are read again for each step.
//
// Move.  A kept row never moves to a higher one, so the rows of a plane can be
// copied in ascending order in place: tile by tile, a tile's rows are loaded
// by all threads before the first is stored, and later tiles' sources lie
// behind every store made before them, so the loads of the next tiles are in
// flight meanwhile.  That is one chain per plane; a row's 256 bytes split into
// slices of their own chains, and as many slices are taken as fill the SMs (32
// bytes, a DRAM sector, at the least).
#include <algorithm>

#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

namespace {

constexpr int kChoiceThreads = 1024;
constexpr int kChoiceWarps = kChoiceThreads / 32;
constexpr int kBins = 2048;

// Whole numbers in the order of the values; -0 is 0, a NaN is above all.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.0f));
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kMaxHeld = 40960;                           // weights a CTA can hold in shared memory

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Sum of the first `warp` of 32 numbers in shared memory (all lanes call it).
__device__ __forceinline__ int sum_below(const int* x, int warp) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(lane < warp ? x[lane] : 0)));
}

// The bin that holds the m-th largest (m >= 1) of the cluster's histograms,
// and how many lie above that bin.  All threads of the cluster call it.
__device__ __forceinline__ int2 find_bin(const uint32_t* hist, int m, int2* found, int* warp_sum, int ctas) {
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5;
  // thread t holds bins 2047 - 2t and 2046 - 2t: descending order
  int h0 = 0, h1 = 0;
  if (ctas == 1) {
    h0 = static_cast<int>(hist[kBins - 1 - 2 * t]);
    h1 = static_cast<int>(hist[kBins - 2 - 2 * t]);
  } else {
    // all loads leave before the first is used (one by one they took 5 us)
    const uint32_t at = smem_addr(hist + kBins - 2 - 2 * t);
    float2 v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = c < ctas ? ld_cluster_f32x2(smem_addr_in_cta(at, static_cast<uint32_t>(c))) : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      h0 += __float_as_int(v[c].y);
      h1 += __float_as_int(v[c].x);
    }
  }
  int incl = h0 + h1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  const int before = incl - h0 - h1 + sum_below(warp_sum, warp);
  if (before < m && m <= before + h0) *found = make_int2(kBins - 1 - 2 * t, before);
  else if (before + h0 < m && m <= before + h0 + h1) *found = make_int2(kBins - 2 - 2 * t, before + h0);
  __syncthreads();
  return *found;
}

}  // namespace

// held: weights of a CTA's run that fit in its dynamic shared memory.
__global__ void __launch_bounds__(kChoiceThreads) kb_evict_choose_kernel(const EvictArgs args, int held) {
  extern __shared__ float own[];
  __shared__ uint32_t hist[kBins];
  __shared__ int warp_sum[kChoiceWarps], warp_eq[kChoiceWarps];
  __shared__ int totals[2], skip_word;                    // this CTA's keys above and at the threshold; nothing to do
  __shared__ int2 found;
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5;
  const int ctas = static_cast<int>(gridDim.x) / (args.B * args.Hkv), rank = static_cast<int>(blockIdx.x) % ctas;
  const int bg = static_cast<int>(blockIdx.x) / ctas, b = bg / args.Hkv;
  const int n = args.lens[b];
  const float* w = args.weights + static_cast<size_t>(bg) * args.kv_cap;
  float* w_out = args.weights_out + static_cast<size_t>(bg) * args.kv_cap;
  int* kept = args.kept + static_cast<size_t>(bg) * args.keep;
  // the cluster decides together whether to go on: every CTA looks at the same words
  // (the error word may change meanwhile, so only the first CTA reads it)
  bool bad = n < 0 || n > args.kv_cap, skip = false;
  if (rank == 0) skip = *reinterpret_cast<volatile uint32_t*>(args.err) != 0;
  if (!bad && args.block_table != nullptr)
    for (int i = t; i < (n + args.page_size - 1) / args.page_size; i += kChoiceThreads) {
      const int pg = args.block_table[static_cast<size_t>(b) * args.pages_per_seq + i];
      bad = bad || pg < 0 || pg >= args.num_pages;
    }
  bad = __syncthreads_or(bad);
  skip = __syncthreads_or(skip);
  if (ctas > 1) {
    if (t == 0) skip_word = skip ? 1 : 0;
    cluster_sync();
    skip = ld_cluster_u32(smem_addr_in_cta(smem_addr(&skip_word), 0u)) != 0;
    if (skip) cluster_sync();                             // all have read the first CTA's word (else later barriers say so)
  }
  if (skip) return;
  const int gt = rank * kChoiceThreads + t, g_threads = ctas * kChoiceThreads;    // this thread in the cluster
  if (bad) {
    if (gt == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
    for (int i = gt; i < args.keep; i += g_threads) kept[i] = -1;     // nothing moves
    if (ctas > 1) cluster_sync();
    return;
  }
  if (n <= args.keep) {
    for (int i = gt; i < args.keep; i += g_threads) kept[i] = i < n ? i : -1;
    for (int i = gt; i < args.kv_cap; i += g_threads) {
      const float x = i < n ? w[i] : 0.0f;
      w_out[i] = x;
    }
    if (ctas > 1) cluster_sync();
    return;
  }
  // rows lo .. hi-1 compete for m places
  const int lo = args.keep_first, hi = n - args.keep_last, m = args.keep - args.keep_first - args.keep_last;
  // this CTA's rows c0 .. c1-1, this warp's r0 .. r1-1
  const int run = ((n + ctas * kChoiceWarps - 1) / (ctas * kChoiceWarps) + 31) / 32 * 32;
  const int c0 = min(rank * kChoiceWarps * run, n), c1 = min(c0 + kChoiceWarps * run, n);
  const int r0 = min(c0 + warp * run, c1), r1 = min(r0 + run, c1);
  const bool holds = kChoiceWarps * run <= held;          // the same in every CTA
  if (holds) {
    // eight loads in flight per thread
    for (int i0 = c0 + t; i0 < c1; i0 += 8 * kChoiceThreads) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = i0 + k * kChoiceThreads < c1 ? w[i0 + k * kChoiceThreads] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i0 + k * kChoiceThreads < c1) own[i0 + k * kChoiceThreads - c0] = x[k];
    }
  }
  auto weight = [&](int i) { return holds ? own[i - c0] : w[i]; };
  uint32_t threshold = 0xFFFFFFFFu;                       // of the keys at it, `ties` are kept
  int ties = 0;
  if (m > 0) {
    uint32_t prefix = 0;
    int left = m;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      for (int i = t; i < kBins; i += kChoiceThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = max(lo, c0) + t; i < min(hi, c1); i += kChoiceThreads) {
        const uint32_t u = order_of(weight(i));
        if (pass == 0 || (u >> (shift + width)) == prefix) atomicAdd(&hist[(u >> shift) & ((1u << width) - 1u)], 1u);
      }
      if (ctas > 1) cluster_sync();
      else __syncthreads();
      const int2 f = find_bin(hist, left, &found, warp_sum, ctas);
      prefix = (prefix << width) | static_cast<uint32_t>(f.x);
      left -= f.y;
      if (ctas > 1) cluster_sync();                       // every CTA has read the histograms
      else __syncthreads();
    }
    threshold = prefix;
    ties = left;
  } else if (ctas > 1) {
    cluster_sync();                                       // every CTA holds its weights before one writes
  } else {
    __syncthreads();
  }
  // 2: kept whatever the ties, 1: at the threshold, 0: dropped
  auto rank_of = [&](int i) {
    if (i < lo || i >= hi) return 2;
    if (m == 0) return 0;
    const uint32_t u = order_of(weight(i));
    return u > threshold ? 2 : u == threshold ? 1 : 0;
  };
  int over = 0, at = 0;
  for (int i = r0; i < r1; i += 32) {
    const int k = i + lane < r1 ? rank_of(i + lane) : 0;
    over += __popc(__ballot_sync(0xffffffffu, k == 2));
    at += __popc(__ballot_sync(0xffffffffu, k == 1));
  }
  if (lane == 0) {
    warp_sum[warp] = over;
    warp_eq[warp] = at;
  }
  __syncthreads();
  int over_before = sum_below(warp_sum, warp), eq_before = sum_below(warp_eq, warp);
  if (ctas > 1) {
    if (t == kChoiceThreads - 1) {
      totals[0] = over_before + over;
      totals[1] = eq_before + at;
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      over_before += static_cast<int>(ld_cluster_u32(smem_addr_in_cta(smem_addr(&totals[0]), static_cast<uint32_t>(c))));
      eq_before += static_cast<int>(ld_cluster_u32(smem_addr_in_cta(smem_addr(&totals[1]), static_cast<uint32_t>(c))));
    }
  }
  for (int i = r0; i < r1; i += 32) {
    const int k = i + lane < r1 ? rank_of(i + lane) : 0;
    const uint32_t b2 = __ballot_sync(0xffffffffu, k == 2), b1 = __ballot_sync(0xffffffffu, k == 1);
    const uint32_t below = (1u << lane) - 1u;
    const int eq = eq_before + __popc(b1 & below);        // keys at the threshold on lower rows
    if (k == 2 || (k == 1 && eq < ties)) {
      const int to = over_before + __popc(b2 & below) + min(eq, ties);
      kept[to] = i + lane;
      if (holds) w_out[to] = own[i + lane - c0];          // (weights_out may be weights: all were read before)
    }
    over_before += __popc(b2);
    eq_before += __popc(b1);
  }
  // all kept rows are written, and no CTA reads another's shared memory any more
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  if (!holds) {
    // the first CTA gathers the kept weights, in place: a tile's are all read before one is written
    if (rank != 0) return;
    for (int i0 = 0; i0 < args.keep; i0 += kChoiceThreads) {
      const int i = i0 + t;
      const float x = i < args.keep ? w[__ldcg(kept + i)] : 0.0f;
      __syncthreads();
      if (i < args.keep) w_out[i] = x;
    }
    __syncthreads();
    for (int i = args.keep + t; i < args.kv_cap; i += kChoiceThreads) w_out[i] = 0.0f;
    return;
  }
  for (int i = args.keep + gt; i < args.kv_cap; i += g_threads) w_out[i] = 0.0f;
}

constexpr int kMoveThreads = 512;
constexpr int kMoveAhead = 4;                             // tiles whose loads are in flight

__global__ void __launch_bounds__(kMoveThreads) kb_evict_move_kernel(const EvictArgs args, int slices) {
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(args.err) != 0)) return;
  const int chunks = 16 / slices;                         // 16-byte chunks of a row in a slice
  const int slice = static_cast<int>(blockIdx.x) % slices;
  const int bg = static_cast<int>(blockIdx.x) / slices;
  const int b = bg / args.Hkv, g = bg % args.Hkv;
  const int n = args.lens[b];
  if (n <= args.keep || n > args.kv_cap) return;          // nothing moves (or the choice reported it)
  uint4* base = static_cast<uint4*>(blockIdx.y != 0 ? args.v : args.k);
  const int* kept = args.kept + static_cast<size_t>(bg) * args.keep;
  const int t = static_cast<int>(threadIdx.x);
  const int col = slice * chunks + t % chunks, row_t = t / chunks;
  const int tile = kMoveThreads / chunks;                 // rows of a tile
  auto place = [&](int row) {
    size_t r = static_cast<size_t>(bg) * args.kv_cap + row;
    if (args.block_table != nullptr) {
      const int pg = __ldg(args.block_table + static_cast<size_t>(b) * args.pages_per_seq + row / args.page_size);
      r = (static_cast<size_t>(pg) * args.Hkv + g) * args.page_size + row % args.page_size;
    }
    return base + r * 16 + col;
  };
  // rows of kMoveAhead tiles in registers, the old rows of the next ones looked up
  uint4 v[kMoveAhead];
  bool moves[kMoveAhead];
  int from[kMoveAhead];
  auto look_up = [&](int i0) { return i0 + row_t < args.keep ? __ldg(kept + i0 + row_t) : -1; };
  auto load = [&](int i0, int src, uint4& x, bool& mv) {
    mv = src > i0 + row_t;
    if (mv) x = *place(src);
  };
#pragma unroll
  for (int a = 0; a < kMoveAhead; ++a) from[a] = look_up(a * tile);
#pragma unroll
  for (int a = 0; a < kMoveAhead; ++a) {
    load(a * tile, from[a], v[a], moves[a]);
    from[a] = look_up((a + kMoveAhead) * tile);
  }
  for (int i0 = 0; i0 < args.keep; i0 += kMoveAhead * tile) {
#pragma unroll
    for (int a = 0; a < kMoveAhead; ++a) {
      const int i = i0 + a * tile;
      __syncthreads();                                    // the tile is loaded in every thread
      if (moves[a]) *place(i + row_t) = v[a];
      load(i + kMoveAhead * tile, from[a], v[a], moves[a]);
      from[a] = look_up(i + 2 * kMoveAhead * tile);
    }
  }
}

cudaError_t launch_evict(const EvictArgs& a, int sm_count, cudaStream_t s) {
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kb_evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld * 4);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  // CTAs of a (batch, KV head)'s choice: no more than find SMs together, at least 4096 keys each
  int ctas = 8;
  while (ctas > 1 && (static_cast<long long>(a.B) * a.Hkv * ctas > sm_count || a.kv_cap < 4096 * ctas)) ctas /= 2;
  // a run is a multiple of 32 rows per warp
  const long long run = (static_cast<long long>(a.kv_cap) / ctas + 2LL * kChoiceThreads) / kChoiceThreads * kChoiceThreads;
  const int held = static_cast<int>(std::min<long long>(run, kMaxHeld));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.Hkv * ctas), 1, 1);
  cfg.blockDim = dim3(kChoiceThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(held) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  if ((e = cudaLaunchKernelEx(&cfg, kb_evict_choose_kernel, a, held)) != cudaSuccess) return e;
  int slices = 1;
  while (slices < 8 && 2LL * a.B * a.Hkv * slices < 2LL * sm_count) slices *= 2;
  kb_evict_move_kernel<<<dim3(static_cast<unsigned>(a.B * a.Hkv * slices), 2), kMoveThreads, 0, s>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace kb

// kb_evict.cu -- cutting a cache to its heaviest keys, in place.
//
// Choice.  One CTA per (batch, KV head).  Weights become whole numbers in the
// order of their values (a NaN above all), the threshold is found digit by
// digit (11, 11 and 10 bits, a histogram each), and of the keys that equal it
// the lowest rows are kept.  Warps own contiguous runs of rows: each counts
// its keys above and at the threshold, one scan over the warps gives every
// run its place, and a second walk writes the kept rows in order.
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

// The bin that holds the m-th largest (m >= 1) of a histogram, and how many
// lie above that bin.  All threads call it.
__device__ __forceinline__ int2 find_bin(const uint32_t* hist, int m, int2* found, int* warp_sum) {
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5;
  // thread t holds bins 2047 - 2t and 2046 - 2t: descending order
  const int h0 = static_cast<int>(hist[kBins - 1 - 2 * t]), h1 = static_cast<int>(hist[kBins - 2 - 2 * t]);
  int incl = h0 + h1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = incl - h0 - h1;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  if (before < m && m <= before + h0) *found = make_int2(kBins - 1 - 2 * t, before);
  else if (before + h0 < m && m <= before + h0 + h1) *found = make_int2(kBins - 2 - 2 * t, before + h0);
  __syncthreads();
  return *found;
}

}  // namespace

__global__ void __launch_bounds__(kChoiceThreads) kb_evict_choose_kernel(const EvictArgs args) {
  __shared__ uint32_t hist[kBins];
  __shared__ int warp_sum[kChoiceWarps], warp_eq[kChoiceWarps];
  __shared__ int2 found;
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(args.err) != 0)) return;
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5;
  const int bg = static_cast<int>(blockIdx.x), b = bg / args.Hkv;
  const int n = args.lens[b];
  const float* w = args.weights + static_cast<size_t>(bg) * args.kv_cap;
  float* w_out = args.weights_out + static_cast<size_t>(bg) * args.kv_cap;
  int* kept = args.kept + static_cast<size_t>(bg) * args.keep;
  bool bad = n < 0 || n > args.kv_cap;
  if (!bad && args.block_table != nullptr)
    for (int i = t; i < (n + args.page_size - 1) / args.page_size; i += kChoiceThreads) {
      const int pg = args.block_table[static_cast<size_t>(b) * args.pages_per_seq + i];
      bad = bad || pg < 0 || pg >= args.num_pages;
    }
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
    for (int i = t; i < args.keep; i += kChoiceThreads) kept[i] = -1;     // nothing moves
    return;
  }
  if (n <= args.keep) {
    for (int i = t; i < args.keep; i += kChoiceThreads) kept[i] = i < n ? i : -1;
    for (int i = t; i < args.kv_cap; i += kChoiceThreads) {
      const float x = i < n ? w[i] : 0.0f;
      w_out[i] = x;
    }
    return;
  }
  // rows lo .. hi-1 compete for m places
  const int lo = args.keep_first, hi = n - args.keep_last, m = args.keep - args.keep_first - args.keep_last;
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
      for (int i = lo + t; i < hi; i += kChoiceThreads) {
        const uint32_t u = order_of(w[i]);
        if (pass == 0 || (u >> (shift + width)) == prefix) atomicAdd(&hist[(u >> shift) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      const int2 f = find_bin(hist, left, &found, warp_sum);
      prefix = (prefix << width) | static_cast<uint32_t>(f.x);
      left -= f.y;
      __syncthreads();
    }
    threshold = prefix;
    ties = left;
  }
  // every warp counts its run of rows
  const int run = ((n + kChoiceWarps - 1) / kChoiceWarps + 31) / 32 * 32;
  const int r0 = min(warp * run, n), r1 = min(r0 + run, n);
  // 2: kept whatever the ties, 1: at the threshold, 0: dropped
  auto rank = [&](int i) {
    if (i < lo || i >= hi) return 2;
    if (m == 0) return 0;
    const uint32_t u = order_of(w[i]);
    return u > threshold ? 2 : u == threshold ? 1 : 0;
  };
  int over = 0, at = 0;
  for (int i = r0; i < r1; i += 32) {
    const int k = i + lane < r1 ? rank(i + lane) : 0;
    over += __popc(__ballot_sync(0xffffffffu, k == 2));
    at += __popc(__ballot_sync(0xffffffffu, k == 1));
  }
  if (lane == 0) {
    warp_sum[warp] = over;
    warp_eq[warp] = at;
  }
  __syncthreads();
  int over_before = 0, eq_before = 0;
  for (int x = 0; x < warp; ++x) {
    over_before += warp_sum[x];
    eq_before += warp_eq[x];
  }
  for (int i = r0; i < r1; i += 32) {
    const int k = i + lane < r1 ? rank(i + lane) : 0;
    const uint32_t b2 = __ballot_sync(0xffffffffu, k == 2), b1 = __ballot_sync(0xffffffffu, k == 1);
    const uint32_t below = (1u << lane) - 1u;
    const int eq = eq_before + __popc(b1 & below);        // keys at the threshold on lower rows
    if (k == 2 || (k == 1 && eq < ties)) kept[over_before + __popc(b2 & below) + min(eq, ties)] = i + lane;
    over_before += __popc(b2);
    eq_before += __popc(b1);
  }
  __syncthreads();
  // the kept weights, in place: a tile's are all read before one is written
  for (int i0 = 0; i0 < args.keep; i0 += kChoiceThreads) {
    const int i = i0 + t;
    const float x = i < args.keep ? w[kept[i]] : 0.0f;
    __syncthreads();
    if (i < args.keep) w_out[i] = x;
  }
  __syncthreads();
  for (int i = args.keep + t; i < args.kv_cap; i += kChoiceThreads) w_out[i] = 0.0f;
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
  uint4 v[kMoveAhead];
  bool moves[kMoveAhead];
  auto load = [&](int i0, uint4& x, bool& mv) {
    const int i = i0 + row_t;
    const int src = i < args.keep ? kept[i] : -1;
    mv = src > i;
    if (mv) x = *place(src);
  };
#pragma unroll
  for (int a = 0; a < kMoveAhead; ++a) load(a * tile, v[a], moves[a]);
  for (int i0 = 0; i0 < args.keep; i0 += kMoveAhead * tile) {
#pragma unroll
    for (int a = 0; a < kMoveAhead; ++a) {
      const int i = i0 + a * tile + row_t;
      __syncthreads();                                    // the tile is loaded in every thread
      if (moves[a]) *place(i) = v[a];
      load(i0 + (a + kMoveAhead) * tile, v[a], moves[a]);
    }
  }
}

cudaError_t launch_evict(const EvictArgs& a, int sm_count, cudaStream_t s) {
  kb_evict_choose_kernel<<<static_cast<unsigned>(a.B * a.Hkv), kChoiceThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int slices = 1;
  while (slices < 8 && 2LL * a.B * a.Hkv * slices < 2LL * sm_count) slices *= 2;
  kb_evict_move_kernel<<<dim3(static_cast<unsigned>(a.B * a.Hkv * slices), 2), kMoveThreads, 0, s>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace kb

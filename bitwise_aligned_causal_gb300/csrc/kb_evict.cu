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
// copied in ascending order in place: a tile's rows are in registers before the
// first is stored, and later tiles' sources lie behind every store made before
// them, so the loads of the next tile are in flight meanwhile.  A tile is shared
// by a cluster of CTAs, as many (1 to 8) as find SMs; its mbarriers put all loads
// of a tile before its stores.  A warp looks up the old
// and new places of its 16 rows in its lanes and hands them round, so a 16-byte
// piece costs four shuffles and no address arithmetic.
//
// Measured, in a replayed graph: 16 paged sequences of 4.5K cut to 2000, a CTA a
// plane, 52 us, of which the choice takes 13 (in slices of rows, with a look-up
// per piece, the move took 65, not 38), the move at a plain copy's rate; a paged
// 28K cache of 18K kept keys, clusters of eight, 62; 64K cut to 8K 41, of which
// the choice takes 25: three digits' rounds of the cluster, a few us each.  A
// third tile in registers cost 15 us in the second case.
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
  __shared__ __align__(16) uint32_t hist[kBins];         // (read in pairs of bins)
  __shared__ int warp_sum[kChoiceWarps], warp_eq[kChoiceWarps];
  __shared__ int totals[2], skip_word;                    // this CTA's keys above and at the threshold; nothing to do
  __shared__ int2 found;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");    // (the move's CTAs may come and wait)
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
  }
  const int gt = rank * kChoiceThreads + t, g_threads = ctas * kChoiceThreads;    // this thread in the cluster
  if (skip || bad) {
    if (bad && gt == 0) atomicCAS(args.err, 0u, static_cast<uint32_t>(kDevBadInput));
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

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = kMoveThreads / 2;               // of a CTA's part of a tile: 16 a warp

// All CTAs of the cluster have read their part of a tile: tell_read, after the
// CTA's threads have met, arrives on every CTA's mbarrier (bar: this CTA's) with
// release, and wait_read waits for this CTA's with acquire.  That puts every load
// of the tile before any store of it.
__device__ __forceinline__ void tell_read(uint32_t bar, int ctas) {
  if (static_cast<int>(threadIdx.x) < ctas) mbar_arrive_cluster(smem_addr_in_cta(bar, threadIdx.x));
}
// Bounded as mbar_wait; false: gave up, after which no thread of the CTA waits
// any more (all go on through their tiles, so no barrier of the CTA is missed; a
// vote on it in __syncthreads_and cost a quarter of the time).
__device__ __forceinline__ bool wait_read(uint32_t bar, uint32_t parity, volatile int* gave_up, uint32_t* err) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*gave_up != 0) return false;
    if (global_timer_ns() - t0 > KB_WAIT_LIMIT_NS) {
      atomicCAS(err, 0u, static_cast<uint32_t>(kDevTimeoutSlot));
      *gave_up = 1;
      return false;
    }
  }
}

// kShared: a plane's CTAs are a cluster.  page_magic: 2^32 / page_size, rounded down.
template <bool kShared>
__global__ void __launch_bounds__(kMoveThreads, 2) kb_evict_move_kernel(const EvictArgs args, int ctas, uint32_t page_magic) {
  asm volatile("griddepcontrol.wait;" ::: "memory");      // (the choice is made)
  const int rank = static_cast<int>(blockIdx.x) % ctas;
  const int plane = static_cast<int>(blockIdx.x) / ctas;  // of B * Hkv key planes, then of the value planes
  const int bg = plane % (args.B * args.Hkv);
  const int b = bg / args.Hkv, g = bg % args.Hkv;
  const int n = args.lens[b];
  if (n <= args.keep || n > args.kv_cap) return;          // nothing moves (or the choice reported it): the whole cluster
  __shared__ uint64_t met;
  __shared__ int gave_up;
  const uint32_t bar = smem_addr(&met);
  if (kShared) {
    if (threadIdx.x == 0) {
      gave_up = 0;
      mbar_init(bar, static_cast<uint32_t>(ctas));
      fence_mbar_init();
    }
    cluster_sync();                                       // every CTA's barrier is there
  }
  char* base = static_cast<char*>(plane != bg ? args.v : args.k);
  const int* kept = args.kept + static_cast<size_t>(bg) * args.keep;
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
  const int mine = rank * kMoveRows + 16 * warp + (lane & 15);      // the row of a tile that this lane looks up
  const int tile = ctas * kMoveRows;
  auto place = [&](int row) {
    size_t r = static_cast<size_t>(bg) * args.kv_cap + row;
    if (args.block_table != nullptr) {
      int at = static_cast<int>(__umulhi(static_cast<uint32_t>(row), page_magic));      // row / page_size, or one less
      int in = row - at * args.page_size;
      if (in >= args.page_size) {
        ++at;
        in -= args.page_size;
      }
      const int pg = __ldg(args.block_table + static_cast<size_t>(b) * args.pages_per_seq + at);
      r = (static_cast<size_t>(pg) * args.Hkv + g) * args.page_size + in;
    }
    return static_cast<unsigned long long>(r * (kHeadDim * 2u));
  };
  auto old_row = [&](int i) { return i < args.keep ? __ldcg(kept + i) : -1; };
  constexpr unsigned long long kNone = ~0ull;
  struct Rows {                                           // this warp's 16 of a tile: 8 loads of two rows
    uint4 v[8];
    unsigned long long to;                                // where the row that this lane looked up goes
  };
  auto load = [&](Rows& x, int i, int src) {
    const bool moves = src > i;                           // (-1: no such row)
    unsigned long long from = kNone;
    x.to = kNone;
    if (moves) {
      from = place(src);
      x.to = place(i);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const unsigned long long at = __shfl_sync(0xffffffffu, from, 2 * k + (lane >> 4));
      if (at != kNone) x.v[k] = *reinterpret_cast<const uint4*>(base + at + (lane & 15) * 16);
    }
  };
  auto store = [&](const Rows& x) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const unsigned long long at = __shfl_sync(0xffffffffu, x.to, 2 * k + (lane >> 4));
      if (at != kNone) *reinterpret_cast<uint4*>(base + at + (lane & 15) * 16) = x.v[k];
    }
  };
  // The values of a tile are there once they have been used.
  auto wait_loaded = [](const Rows& x) {
    uint32_t all = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) all |= x.v[k].x | x.v[k].y | x.v[k].z | x.v[k].w;
    if (all == 0x9E3779B9u) __nanosleep(0);
  };
  Rows set[2] = {};
  load(set[0], mine, old_row(mine));
  int ahead = old_row(tile + mine);                       // old rows are looked up a tile before their rows are read
  for (int i0 = 0; i0 < args.keep; i0 += 2 * tile) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int i = i0 + a * tile;                        // (past the last row nothing is read or written)
      // A release waits for all loads on their way, so a cluster's next tile leaves
      // behind it (three caches of 32K 104 us; before it 120); a CTA alone has none
      // and gains by an earlier start (16 caches of 4.5K 52 us; behind it 55).
      auto load_next = [&]() {
        load(set[a ^ 1], i + tile + mine, ahead);
        ahead = old_row(i + 2 * tile + mine);
      };
      if (!kShared) load_next();
      wait_loaded(set[a]);                                // the tile is loaded, here ...
      __syncthreads();                                    // ... in the CTA ...
      if (kShared) {
        tell_read(bar, ctas);
        load_next();
      }
      if (!kShared || wait_read(bar, static_cast<uint32_t>(a), &gave_up, args.err)) store(set[a]);    // ... and in the cluster
    }
  }
  if (kShared) cluster_sync();                            // (no CTA leaves while another may arrive on its barrier)
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
  // CTAs of a plane's move: as many as find a place together (clusters fill four
  // fifths of the two places on an SM), at most one per part of a tile
  const long long planes = 2LL * a.B * a.Hkv;
  const int movers = static_cast<int>(std::max(1LL, std::min({8LL, 8LL * sm_count / (5 * planes), (a.keep + kMoveRows - 1LL) / kMoveRows})));
  cudaLaunchConfig_t mv{};
  mv.gridDim = dim3(static_cast<unsigned>(planes * movers), 1, 1);
  mv.blockDim = dim3(kMoveThreads, 1, 1);
  mv.stream = s;
  cudaLaunchAttribute mattr[2];
  mattr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;      // its launch is hidden by the choice
  mattr[0].val.programmaticStreamSerializationAllowed = 1;
  mattr[1].id = cudaLaunchAttributeClusterDimension;
  mattr[1].val.clusterDim.x = static_cast<unsigned>(movers);
  mattr[1].val.clusterDim.y = 1;
  mattr[1].val.clusterDim.z = 1;
  mv.attrs = mattr;
  mv.numAttrs = movers > 1 ? 2 : 1;
  const uint32_t magic = a.block_table != nullptr ? static_cast<uint32_t>((1ull << 32) / static_cast<uint32_t>(a.page_size)) : 0u;
  return cudaLaunchKernelEx(&mv, movers > 1 ? kb_evict_move_kernel<true> : kb_evict_move_kernel<false>, a, movers, magic);
}

}  // namespace kb

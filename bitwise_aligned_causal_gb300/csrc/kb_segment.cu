// kb_segment.cu -- the fold of the C5 segmented mode for the packed kernel.
//
// In segmented mode the packed kernel (decode and chunks of at most 32 rows)
// runs one CTA per (segment, sub-chunk, b, kv head) and leaves each row's
// per-segment partial (O unnormalised, m, mc, l) in the caller's workspace.
// This kernel folds a row's segments left to right with fold_state / fold_o
// (the functions the segmented tile kernel applies in TMEM at its segment
// ends) and normalises (C4), so every entry point of the mode gives the same
// bits (KernelBraid README, "Method": one contract for prefill, partitioned
// forward and decode).
#include "kb_contract.cuh"
#include "kb_launch.h"

namespace kb {

// One warp per output row (b, h, r): lane l owns columns 4l..4l+3.
__global__ void __launch_bounds__(256) kb_seg_fold_kernel(const float* __restrict__ part,
                                                          __nv_bfloat16* __restrict__ o, long long rows, int L,
                                                          int start, int seg_tiles, int n_seg) {
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  const int r = static_cast<int>(row % L);
  const int n_kv = (start + r) / kTileKeys + 1;                   // C1: tiles 0..floor(p / 128)
  const int ns = (n_kv + seg_tiles - 1) / seg_tiles;              // this row's segments
  const float* p = part + static_cast<size_t>(row) * n_seg * kPartFloats;
  float4 acc_o = reinterpret_cast<const float4*>(p)[lane];        // segment 0 as it is
  const float4 s0 = reinterpret_cast<const float4*>(p + 128)[0];
  RowState acc{s0.x, s0.y, s0.z};
  for (int sg = 1; sg < ns; ++sg) {
    const float* q = p + static_cast<size_t>(sg) * kPartFloats;
    const float4 so = reinterpret_cast<const float4*>(q)[lane];
    const float4 st = reinterpret_cast<const float4*>(q + 128)[0];
    const RowState seg{st.x, st.y, st.z};
    const FoldScale f = fold_state(acc, seg);
    acc_o.x = fold_o(acc_o.x, so.x, f);
    acc_o.y = fold_o(acc_o.y, so.y, f);
    acc_o.z = fold_o(acc_o.z, so.z, f);
    acc_o.w = fold_o(acc_o.w, so.w, f);
  }
  const float inv_l = row_inv_l(acc);
  uint2 w;
  w.x = pack_bf16x2(__fmul_rn(acc_o.x, inv_l), __fmul_rn(acc_o.y, inv_l));
  w.y = pack_bf16x2(__fmul_rn(acc_o.z, inv_l), __fmul_rn(acc_o.w, inv_l));
  reinterpret_cast<uint2*>(o + static_cast<size_t>(row) * kHeadDim)[lane] = w;
}

cudaError_t launch_seg_fold(const float* part, void* o, long long rows, int L, int start, int seg_tiles, int n_seg,
                            cudaStream_t s) {
  kb_seg_fold_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, s>>>(
      part, static_cast<__nv_bfloat16*>(o), rows, L, start, seg_tiles, n_seg);
  return cudaGetLastError();
}

// One CTA per output row, thread t owns column t.  The row's partials come to
// shared memory together, 64 segments at a time, and are folded left to right:
// a row of 64 segments waits for memory once (eight at a time, in registers, a
// token at 64K took 55 us, so 43).  Launched ahead of the partials' kernel's end (it waits for it here), so
// that its own launch costs no time.
constexpr int kFoldChunk = 64;

__global__ void __launch_bounds__(kHeadDim) kb_rows_fold_kernel(const RowsFoldArgs args) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (*reinterpret_cast<const volatile uint32_t*>(args.err) != 0) return;    // the partials are not there
  const int row = static_cast<int>(blockIdx.x);
  const int r = row % args.L, b = row / args.L / args.Hq;
  int start = args.start, rows = args.L;
  if (args.ctx_lens != nullptr) start = args.ctx_lens[b] - args.L;
  if (args.starts != nullptr) {
    start = args.starts[b];
    rows = args.lens[b];
  }
  if (r >= rows) return;
  const int n_kv = (start + r) / kTileKeys + 1;                   // C1: tiles 0..floor(p / 128)
  const int ns = min((n_kv + kSegTiles - 1) / kSegTiles, args.n_seg);
  const int t = static_cast<int>(threadIdx.x);
  const float* p = args.part + static_cast<size_t>(row) * args.n_seg * kPartFloats;
  __shared__ __align__(16) float held[kFoldChunk][kPartFloats];
  RowState acc = row_state_init();
  float acc_o = 0.0f;
  for (int s0 = 0; s0 < ns; s0 += kFoldChunk) {
    const int n = min(kFoldChunk, ns - s0);
    const float4* from = reinterpret_cast<const float4*>(p + static_cast<size_t>(s0) * kPartFloats);
    __syncthreads();                                              // (the chunk before has been folded)
    for (int x = t; x < n * (kPartFloats / 4); x += kHeadDim)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(&held[0][4 * x])), "l"(from + x) : "memory");
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&held[i][kHeadDim]);
      const float os = held[i][t];
      const RowState seg{v.x, v.y, v.z};
      if (s0 + i == 0) {                                          // segment 0 as it is
        acc = seg;
        acc_o = os;
      } else {
        const FoldScale f = fold_state(acc, seg);
        acc_o = fold_o(acc_o, os, f);
      }
    }
  }
  static_cast<__nv_bfloat16*>(args.o)[static_cast<size_t>(row) * kHeadDim + t] =
      __float2bfloat16_rn(__fmul_rn(acc_o, row_inv_l(acc)));
}

cudaError_t launch_rows_fold(const RowsFoldArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hq * a.L), 1, 1);
  cfg.blockDim = dim3(kHeadDim, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kb_rows_fold_kernel, a);
}

}  // namespace kb

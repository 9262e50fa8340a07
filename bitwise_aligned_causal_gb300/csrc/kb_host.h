// kb_host.h -- host-side checks and device state shared by the C entry points
// of kb_host.cu and kb_host_sparse.cu (internal; the public C ABI is
// include/kb_attn.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/kb_attn.h"

namespace kb {

constexpr int kMaxRows = 1 << 22;     // positions per sequence (4M)
constexpr int kMaxDevices = 64;

// What the entry points need to know about the current device.
struct HostDevice {
  int index;
  uint32_t* err;       // the library's error word there
  int sm_count;
  const int* cluster_fit;   // clusters of 2, 4, 8 narrow packed CTAs it runs at once (entries 1, 2, 3)
};

kb_status host_device(HostDevice* out);
// Record a failed CUDA call for kb_attn_last_cuda_error and map it to a status.
kb_status host_cuda_fail(cudaError_t e);
// Device (or managed) memory reachable from the current device?
kb_status host_device_pointer(const void* p);
// Tensor map of whole 128-row tiles: box {64 columns, 128 rows, 2 halves} of
// a [planes, rows, 128] bf16 tensor (kb_host.cu).
kb_status host_rows_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t planes, uint64_t plane_stride);
// Tensor map of query rows packed by GQA group: box {64 columns, 32 rows,
// 4 heads, 2 halves} of a [planes * 4 heads, rows, 128] bf16 tensor, so one
// load brings the 32 rows of a KV head's four query heads as one 128-row tile
// (row 32 * head + r) in two swizzled slabs.
kb_status host_group_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t groups);
kb_status host_check_heads(int B, int Hq, int Hkv);
// A page table: pages_per_seq * page_size positions per sequence, page_size a
// multiple of 128.
kb_status host_check_paging(const int* block_table, int pages_per_seq, int page_size, int num_pages, int Hkv);

inline bool host_aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

}  // namespace kb

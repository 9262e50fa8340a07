// kb_host.h -- host-side checks and device state shared by the C entry points
// of kb_host.cu, kb_host_sparse.cu and kb_host_cache.cu (internal; the public
// C ABI is include/kb_attn.h).
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
// The same with boxes of one column half (tma_load_half).
kb_status host_halves_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t planes, uint64_t plane_stride);
// Tensor map of whole 128-row tiles of a cache held in 8 bits: box {128 bytes,
// 128 rows} of a [planes, rows, 128] byte tensor, 128-byte swizzle.
kb_status host_bytes_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t planes, uint64_t plane_stride);
// Tensor map of query rows packed by GQA group: box {64 columns, 32 rows,
// 4 heads, 2 halves} of a [planes * 4 heads, rows, 128] bf16 tensor, so one
// load brings the 32 rows of a KV head's four query heads as one 128-row tile
// (row 32 * head + r) in two swizzled slabs.
kb_status host_group_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t groups);
// CTAs per (sub-chunk, batch, KV head) of the packed kernel's fold mode.
int host_choose_cluster(int sm_count, const int* cluster_fit, int L, int n_sub, int B, int Hkv, int n_kv_max);
kb_status host_check_heads(int B, int Hq, int Hkv);
// A page table: pages_per_seq * page_size positions per sequence, page_size a
// multiple of 128.
kb_status host_check_paging(const int* block_table, int pages_per_seq, int page_size, int num_pages, int Hkv);

inline bool host_aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

inline kb_status host_done(cudaError_t e) { return e == cudaSuccess ? KB_OK : host_cuda_fail(e); }

inline kb_status host_device_pointers(const void* const* p, int n) {
  for (int i = 0; i < n; ++i)
    if (p[i] != nullptr) {
      const kb_status s = host_device_pointer(p[i]);
      if (s != KB_OK) return s;
    }
  return KB_OK;
}

inline kb_status host_check_table(const float* table, int n_pos, int rot_dim) {
  if (!host_aligned(table, 16)) return KB_ERR_INVALID_ARG;
  if (n_pos < 1 || rot_dim < 2) return KB_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > 128 || n_pos > kMaxRows) return KB_ERR_UNSUPPORTED;
  return KB_OK;
}

// Batch, head and row strides of a [*, *, *, 128] view, in elements.
inline kb_status host_check_strides(const long long* st) {
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % 8 != 0) return KB_ERR_INVALID_ARG;
  return KB_OK;
}

// Per-sequence starts and lens (device int32 arrays; both null: `start` and L rows).
inline kb_status host_check_ragged(const int* starts, const int* lens) {
  if (lens != nullptr && starts == nullptr) return KB_ERR_INVALID_ARG;
  if (!host_aligned(starts, 4) || !host_aligned(lens, 4)) return KB_ERR_INVALID_ARG;
  return KB_OK;
}

// The cache's capacity in positions: kv_cap, or the page table's.
inline kb_status host_cache_rows(int* cap, int kv_cap, const int* block_table, int pages_per_seq, int page_size,
                                 int num_pages, int Hkv) {
  if (block_table != nullptr) {
    const kb_status s = host_check_paging(block_table, pages_per_seq, page_size, num_pages, Hkv);
    if (s != KB_OK) return s;
    *cap = pages_per_seq * page_size;
    return KB_OK;
  }
  if (kv_cap < 1) return KB_ERR_INVALID_ARG;
  if (kv_cap > kMaxRows) return KB_ERR_UNSUPPORTED;
  *cap = kv_cap;
  return KB_OK;
}

}  // namespace kb

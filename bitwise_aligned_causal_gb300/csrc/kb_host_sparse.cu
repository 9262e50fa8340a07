// kb_host_sparse.cu -- C entry points around block-sparse attention: rotation,
// cache append, key-block boxes, block selection, sparse attention and its
// gradient.  Declarations and their contract are in include/kb_attn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/kb_attn.h"
#include "kb_contract.cuh"
#include "kb_host.h"
#include "kb_launch.h"

namespace {

using kb::host_aligned;
using kb::kMaxRows;

kb_status done(cudaError_t e) { return e == cudaSuccess ? KB_OK : kb::host_cuda_fail(e); }

kb_status device_pointers(const void* const* p, int n) {
  for (int i = 0; i < n; ++i)
    if (p[i] != nullptr) {
      const kb_status s = kb::host_device_pointer(p[i]);
      if (s != KB_OK) return s;
    }
  return KB_OK;
}

kb_status check_table(const float* table, int n_pos, int rot_dim) {
  if (!host_aligned(table, 16)) return KB_ERR_INVALID_ARG;
  if (n_pos < 1 || rot_dim < 2) return KB_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > kb::kHeadDim || n_pos > kMaxRows) return KB_ERR_UNSUPPORTED;
  return KB_OK;
}

// Batch, head and row strides of a [*, *, *, 128] view, in elements.
kb_status check_strides(const long long* st) {
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % 8 != 0) return KB_ERR_INVALID_ARG;
  return KB_OK;
}

// Per-sequence starts and lens (device int32 arrays; both null: `start` and L rows).
kb_status check_ragged(const int* starts, const int* lens) {
  if (lens != nullptr && starts == nullptr) return KB_ERR_INVALID_ARG;
  if (!host_aligned(starts, 4) || !host_aligned(lens, 4)) return KB_ERR_INVALID_ARG;
  return KB_OK;
}

// The cache's capacity in positions: kv_cap, or the page table's.
kb_status cache_rows(int* cap, int kv_cap, const int* block_table, int pages_per_seq, int page_size, int num_pages,
                     int Hkv) {
  if (block_table != nullptr) {
    const kb_status s = kb::host_check_paging(block_table, pages_per_seq, page_size, num_pages, Hkv);
    if (s != KB_OK) return s;
    *cap = pages_per_seq * page_size;
    return KB_OK;
  }
  if (kv_cap < 1) return KB_ERR_INVALID_ARG;
  if (kv_cap > kMaxRows) return KB_ERR_UNSUPPORTED;
  *cap = kv_cap;
  return KB_OK;
}

}  // namespace

extern "C" {

kb_status kb_attn_rope_table(float* table, int n_pos, int rot_dim, const double* inv_freq, void* stream) {
  if (!table || !inv_freq || !host_aligned(inv_freq, 8)) return KB_ERR_INVALID_ARG;
  kb_status s = check_table(table, n_pos, rot_dim);
  if (s != KB_OK) return s;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {table, inv_freq};
  if ((s = device_pointers(p, 2)) != KB_OK) return s;
  return done(kb::launch_rope_table(table, n_pos, rot_dim, inv_freq, static_cast<cudaStream_t>(stream)));
}

kb_status kb_attn_rope(const void* x, const long long* strides, void* out, const float* table, int n_pos, int rot_dim,
                       int interleaved, int inverse, int B, int H, int L, int start, void* stream) {
  if (!x || !out || !strides || !table || !host_aligned(x, 16) || !host_aligned(out, 16)) return KB_ERR_INVALID_ARG;
  kb_status s = check_table(table, n_pos, rot_dim);
  if (s != KB_OK) return s;
  if ((s = check_strides(strides)) != KB_OK) return s;
  if (B < 1 || H < 1 || L < 1 || start < 0 || start > n_pos - L) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * ((H + 3) / 4) * ((L + 3) / 4) > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {x, out, table};
  if ((s = device_pointers(p, 3)) != KB_OK) return s;
  kb::RopeArgs a{};
  a.x = x;
  a.sb = strides[0];
  a.sh = strides[1];
  a.sl = strides[2];
  a.out = out;
  a.table = table;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  a.B = B;
  a.H = H;
  a.L = L;
  a.start = start;
  a.err = dev.err;
  return done(kb::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

kb_status kb_attn_append(const void* q, const void* k, const void* v, const long long* strides, void* q_out,
                         void* k_cache, void* v_cache, void* boxes, const float* table, int n_pos, int rot_dim,
                         int interleaved, int B, int Hq, int Hkv, int L, int start, const int* starts,
                         const int* lens, int kv_cap, const int* block_table, int pages_per_seq, int page_size,
                         int num_pages, void* stream) {
  if (!k || !v || !k_cache || !v_cache || !strides || (q == nullptr) != (q_out == nullptr)) return KB_ERR_INVALID_ARG;
  const void* p[] = {q, k, v, q_out, k_cache, v_cache, boxes, table, starts, lens, block_table};
  for (int i = 0; i < 8; ++i)
    if (!host_aligned(p[i], 16)) return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(B, Hq, Hkv);
  if (s != KB_OK) return s;
  if (table != nullptr && (s = check_table(table, n_pos, rot_dim)) != KB_OK) return s;
  for (int i = q == nullptr ? 1 : 0; i < 3; ++i)
    if ((s = check_strides(strides + 3 * i)) != KB_OK) return s;
  if ((s = check_ragged(starts, lens)) != KB_OK) return s;
  int cap = 0;
  if ((s = cache_rows(&cap, kv_cap, block_table, pages_per_seq, page_size, num_pages, Hkv)) != KB_OK) return s;
  if (L < 1 || L > cap) return KB_ERR_INVALID_ARG;
  if (starts == nullptr && (start < 0 || start > cap - L || (table != nullptr && start > n_pos - L)))
    return KB_ERR_INVALID_ARG;
  if ((static_cast<long long>(L) / kb::kTileKeys + 2) * B * Hkv > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  if ((s = device_pointers(p, 11)) != KB_OK) return s;
  kb::AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = strides[i];
    a.ks[i] = strides[3 + i];
    a.vs[i] = strides[6 + i];
  }
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.boxes = boxes;
  a.table = table;
  a.n_pos = n_pos;
  a.rot_dim = table != nullptr ? rot_dim : kb::kHeadDim;
  a.interleaved = interleaved != 0;
  a.B = B;
  a.Hkv = Hkv;
  a.L = L;
  a.start = start;
  a.starts = starts;
  a.lens = lens;
  a.kv_cap = cap;
  a.block_table = block_table;
  a.pages_per_seq = pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.err = dev.err;
  return done(kb::launch_append(a, false, static_cast<cudaStream_t>(stream)));
}

kb_status kb_attn_block_boxes(const void* k_cache, void* boxes, int B, int Hkv, int kv_len, const int* kv_lens,
                              int kv_cap, const int* block_table, int pages_per_seq, int page_size, int num_pages,
                              void* stream) {
  if (!k_cache || !boxes || !host_aligned(k_cache, 16) || !host_aligned(boxes, 16) || !host_aligned(kv_lens, 4))
    return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(B, kb::kGroup * Hkv, Hkv);
  if (s != KB_OK) return s;
  int cap = 0;
  if ((s = cache_rows(&cap, kv_cap, block_table, pages_per_seq, page_size, num_pages, Hkv)) != KB_OK) return s;
  if (kv_len < 1 || kv_len > cap) return KB_ERR_INVALID_ARG;
  if ((static_cast<long long>(kv_len) / kb::kTileKeys + 2) * B * Hkv > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {k_cache, boxes, kv_lens, block_table};
  if ((s = device_pointers(p, 4)) != KB_OK) return s;
  kb::AppendArgs a{};
  a.k_cache = const_cast<void*>(k_cache);
  a.boxes = boxes;
  a.rot_dim = kb::kHeadDim;
  a.B = B;
  a.Hkv = Hkv;
  a.L = kv_len;
  a.lens = kv_lens;
  a.kv_cap = cap;
  a.block_table = block_table;
  a.pages_per_seq = pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.err = dev.err;
  return done(kb::launch_append(a, true, static_cast<cudaStream_t>(stream)));
}

kb_status kb_attn_select_blocks(const void* q, const void* boxes, int* blocks, int B, int Hq, int Hkv, int L,
                                int n_select, int keep_first, int keep_last, int start, const int* starts,
                                const int* lens, int n_blocks, const int* block_table, int pages_per_seq,
                                int page_size, int num_pages, void* stream) {
  if (!q || !boxes || !blocks || !host_aligned(q, 16) || !host_aligned(boxes, 16) || !host_aligned(blocks, 4))
    return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(B, Hq, Hkv);
  if (s != KB_OK) return s;
  if ((s = check_ragged(starts, lens)) != KB_OK) return s;
  if (n_select < 1 || keep_first < 0 || keep_last < 1 || keep_first > n_select || keep_last > n_select - keep_first)
    return KB_ERR_INVALID_ARG;
  if (n_select > KB_MAX_SELECT) return KB_ERR_UNSUPPORTED;
  if (block_table == nullptr && (n_blocks < 1 || n_blocks > kMaxRows / kb::kTileKeys))
    return n_blocks < 1 ? KB_ERR_INVALID_ARG : KB_ERR_UNSUPPORTED;
  int cap = 0;
  if ((s = cache_rows(&cap, n_blocks * kb::kTileKeys, block_table, pages_per_seq, page_size, num_pages, Hkv)) != KB_OK)
    return s;
  if (L < 1 || L > cap || (starts == nullptr && (start < 0 || start > cap - L))) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * Hkv * L > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {q, boxes, blocks, starts, lens, block_table};
  if ((s = device_pointers(p, 6)) != KB_OK) return s;
  kb::SelectArgs a{};
  a.q = q;
  a.boxes = boxes;
  a.blocks = blocks;
  a.B = B;
  a.Hkv = Hkv;
  a.L = L;
  a.n = n_select;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.start = start;
  a.starts = starts;
  a.lens = lens;
  a.kv_cap = cap;
  a.blocks_per_plane = block_table != nullptr ? page_size / kb::kTileKeys : n_blocks;
  a.max_blocks = (starts != nullptr ? cap : start + L - 1) / kb::kTileKeys + (starts != nullptr ? 0 : 1);
  a.block_table = block_table;
  a.pages_per_seq = pages_per_seq;
  a.num_pages = num_pages;
  a.err = dev.err;
  return done(kb::launch_select(a, dev.index, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// kb_host_sparse.cu -- C entry points around block-sparse attention: rotation,
// cache append, key-block boxes, block selection, sparse attention and its
// gradient.  Declarations and their contract are in include/kb_attn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/kb_attn.h"
#include "kb_contract.cuh"
#include "kb_host.h"
#include "kb_launch.h"
#include "kb_sparse.cuh"

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

// Position tiles of 32 that L consecutive positions can touch.
long long max_tiles32(long long L) { return (L + kb::kUnitRows - 2) / kb::kUnitRows + 1; }

long long align256(long long n) { return (n + 255) / 256 * 256; }

// Workspace of a plan: the walks' lengths, then the walks.
struct PlanSizes {
  long long units, cap, bytes;
};
PlanSizes plan_sizes(int B, int Hkv, int L, int n_select, long long max_blocks) {
  PlanSizes p;
  p.units = static_cast<long long>(B) * Hkv * max_tiles32(L);
  p.cap = std::min<long long>(static_cast<long long>(kb::kUnitRows) * n_select, max_blocks);
  p.bytes = align256(p.units * 4) + p.units * p.cap * 8;
  return p;
}

// Where the backward's row masks start: one per unit and key block, behind the walks.
long long masks_at(const PlanSizes& p) { return align256(p.bytes); }

// The backward's workspace behind the plan's: row masks; counts and tickets
// (zeroed by every call); jobs and their number; fp32 sums.
struct BwdSizes {
  long long n_split;                                   // key blocks that two CTAs may share
  long long masks, counts, tickets, jobs, sums, bytes; // offsets, size
};
BwdSizes bwd_sizes(const PlanSizes& p, int B, int Hkv, int S) {
  BwdSizes b;
  const long long blocks = (S + kb::kTileKeys - 1) / kb::kTileKeys, groups = static_cast<long long>(B) * Hkv;
  // rows from 128 j on can list block j, and a shared one has 32 * (kSparseSplitSteps - 1) + 1 at least
  const long long spare = S - (kb::kSparseSplitSteps - 1LL) * kb::kUnitRows;
  b.n_split = spare > 0 ? std::min((spare + kb::kTileKeys - 1) / kb::kTileKeys, blocks) : 0;
  b.masks = masks_at(p);
  b.counts = align256(b.masks + p.units * blocks * 4);
  b.tickets = b.counts + groups * blocks * 4;
  b.jobs = align256(b.tickets + groups * b.n_split * 4);
  b.sums = align256(b.jobs + 8 + groups * (blocks + b.n_split) * 8);
  b.bytes = b.sums + groups * b.n_split * 2 * (2LL * kb::kTileKeys * kb::kHeadDim * 4);
  return b;
}

struct SparseCall {
  const void *q, *k, *v;
  void* o;
  float* lse;
  const int* blocks;
  int n_select, B, Hq, Hkv, L, start;
  const int *starts, *lens;
  int kv_cap;
  const int* block_table;
  int pages_per_seq, page_size, num_pages;
  void* workspace;
  size_t workspace_bytes;
};

// Checks that every block-sparse forward makes; *cap gets the cache's positions.
kb_status check_sparse(const SparseCall& c, int* cap, kb::HostDevice* dev) {
  if (!c.q || !c.k || !c.v || !c.o || !c.blocks) return KB_ERR_INVALID_ARG;
  for (const void* p : {c.q, c.k, c.v, static_cast<const void*>(c.o)})
    if (!host_aligned(p, 16)) return KB_ERR_INVALID_ARG;
  if (!host_aligned(c.blocks, 4) || !host_aligned(c.lse, 4)) return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(c.B, c.Hq, c.Hkv);
  if (s != KB_OK) return s;
  if ((s = check_ragged(c.starts, c.lens)) != KB_OK) return s;
  if (c.n_select < 1) return KB_ERR_INVALID_ARG;
  if (c.n_select > KB_MAX_SELECT) return KB_ERR_UNSUPPORTED;
  if ((s = cache_rows(cap, c.kv_cap, c.block_table, c.pages_per_seq, c.page_size, c.num_pages, c.Hkv)) != KB_OK) return s;
  if (c.L < 1 || c.L > *cap || (c.starts == nullptr && (c.start < 0 || c.start > *cap - c.L))) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(c.B) * c.Hkv * max_tiles32(c.L) > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  if ((s = kb::host_device(dev)) != KB_OK) return s;
  const void* p[] = {c.q, c.k, c.v, c.o, c.lse, c.blocks, c.starts, c.lens, c.block_table, c.workspace};
  return device_pointers(p, 10);
}

// K/V maps: a contiguous uniform cache ends at the call's last key (later rows
// read as zeros), a ragged batch maps the whole cache, a pool its pages.
kb_status cache_maps(const SparseCall& c, CUtensorMap* tk, CUtensorMap* tv) {
  const uint64_t row_bytes = kb::kHeadDim * 2u;
  const bool paged = c.block_table != nullptr;
  const uint64_t stride_rows = static_cast<uint64_t>(paged ? c.page_size : c.kv_cap);
  const uint64_t rows = paged || c.starts != nullptr ? stride_rows : static_cast<uint64_t>(c.start) + c.L;
  const uint64_t planes = static_cast<uint64_t>(paged ? c.num_pages : c.B) * c.Hkv;
  const kb_status s = kb::host_rows_map(tk, c.k, rows, planes, stride_rows * row_bytes);
  if (s != KB_OK) return s;
  return kb::host_rows_map(tv, c.v, rows, planes, stride_rows * row_bytes);
}

// Units, walks and workspace of a call; with_masks: the backward's row masks too.
kb_status fill_plan(const SparseCall& c, int cap, uint32_t* err, bool with_masks, kb::SparseArgs* a) {
  a->o = c.o;
  a->lse = c.lse;
  a->blocks = c.blocks;
  a->n_select = c.n_select;
  a->B = c.B;
  a->Hq = c.Hq;
  a->Hkv = c.Hkv;
  a->L = c.L;
  a->start = c.start;
  a->starts = c.starts;
  a->lens = c.lens;
  a->kv_cap = cap;
  a->max_blocks = ((c.starts != nullptr ? cap : c.start + c.L) + kb::kTileKeys - 1) / kb::kTileKeys;
  a->block_table = c.block_table;
  a->pages_per_seq = c.pages_per_seq;
  a->page_size = c.page_size;
  a->num_pages = c.num_pages;
  a->err = err;
  const PlanSizes full = plan_sizes(c.B, c.Hkv, c.L, c.n_select, a->max_blocks);
  const BwdSizes bwd = bwd_sizes(full, c.B, c.Hkv, c.L);
  const long long need = with_masks ? bwd.bytes : full.bytes;
  if (c.workspace == nullptr || !host_aligned(c.workspace, 256) || c.workspace_bytes < static_cast<size_t>(need))
    return KB_ERR_INVALID_ARG;
  a->n_tiles = static_cast<int>(c.starts != nullptr ? max_tiles32(c.L)
                                                    : (c.start + c.L - 1) / kb::kUnitRows - c.start / kb::kUnitRows + 1);
  a->n_units = c.B * c.Hkv * a->n_tiles;
  a->walk_cap = static_cast<int>(full.cap);
  a->walk_len = static_cast<int*>(c.workspace);
  a->walks = reinterpret_cast<uint2*>(static_cast<char*>(c.workspace) + align256(full.units * 4));
  if (with_masks) {
    a->masks = reinterpret_cast<uint32_t*>(static_cast<char*>(c.workspace) + bwd.masks);
    a->row_counts = reinterpret_cast<int*>(static_cast<char*>(c.workspace) + bwd.counts);
  }
  return KB_OK;
}

kb_status sparse_forward(const SparseCall& c, void* stream) {
  int cap = 0;
  kb::HostDevice dev;
  kb_status s = check_sparse(c, &cap, &dev);
  if (s != KB_OK) return s;
  kb::SparseArgs a{};
  if ((s = fill_plan(c, cap, dev.err, false, &a)) != KB_OK) return s;
  CUtensorMap tq, tk, tv;
  if ((s = kb::host_group_map(&tq, c.q, static_cast<uint64_t>(c.L), static_cast<uint64_t>(c.B) * c.Hkv)) != KB_OK) return s;
  if ((s = cache_maps(c, &tk, &tv)) != KB_OK) return s;
  cudaError_t e = kb::launch_sparse_plan(a, dev.index, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = kb::launch_sparse_tile(tq, tk, tv, a, dev.index, dev.sm_count, static_cast<cudaStream_t>(stream));
  return done(e);
}

// CTAs per (b, KV head) of a block-sparse token: the largest cluster whose
// clusters all run at once, when the batch alone would leave SMs idle (the
// rule of the dense token, with the segments a list can name).
int sparse_cluster(const kb::HostDevice& dev, int B, int Hkv, int n_select, int max_blocks) {
  const long long units = static_cast<long long>(B) * Hkv;
  if (2 * units > dev.sm_count) return 1;
  const int ns = std::min(n_select, (max_blocks + kb::kSegTiles - 1) / kb::kSegTiles);
  const long long slots = kb::packed_partial_slots(kb::kGroup, true);
  for (int i = 3, c = 8; i >= 1; --i, c /= 2)
    if (c <= ns && units <= dev.cluster_fit[i] && (ns + c - 1) / c <= slots) return c;
  return 1;
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
  return done(kb::launch_append(a, false, dev.sm_count, static_cast<cudaStream_t>(stream)));
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
  return done(kb::launch_append(a, true, dev.sm_count, static_cast<cudaStream_t>(stream)));
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

size_t kb_attn_sparse_workspace_bytes(int B, int Hkv, int L, int n_select, int kv_cap) {
  if (B < 1 || Hkv < 1 || L < 1 || n_select < 1 || n_select > KB_MAX_SELECT || kv_cap < 1 || kv_cap > kMaxRows) return 0;
  return static_cast<size_t>(plan_sizes(B, Hkv, L, n_select, (kv_cap + kb::kTileKeys - 1) / kb::kTileKeys).bytes);
}

kb_status kb_attn_sparse_chunk(const void* q, const void* k, const void* v, void* o, const int* blocks, int n_select,
                               int B, int Hq, int Hkv, int L, int start, const int* starts, const int* lens, int kv_cap,
                               const int* block_table, int pages_per_seq, int page_size, int num_pages, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const SparseCall c{q, k, v, o, nullptr, blocks, n_select, B, Hq, Hkv, L, start, starts, lens, kv_cap, block_table,
                     pages_per_seq, page_size, num_pages, workspace, workspace_bytes};
  return sparse_forward(c, stream);
}

kb_status kb_attn_sparse_prefill_lse(const void* q, const void* k, const void* v, void* o, float* lse,
                                     const int* blocks, int n_select, int B, int Hq, int Hkv, int S, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (lse == nullptr) return KB_ERR_INVALID_ARG;
  const SparseCall c{q, k, v, o, lse, blocks, n_select, B, Hq, Hkv, S, 0, nullptr, nullptr, S, nullptr, 0, 0, 0,
                     workspace, workspace_bytes};
  return sparse_forward(c, stream);
}

kb_status kb_attn_sparse_decode(const void* q, const void* k, const void* v, void* o, const int* blocks, int n_select,
                                int B, int Hq, int Hkv, int ctx_len, const int* ctx_lens, int kv_cap,
                                const int* block_table, int pages_per_seq, int page_size, int num_pages, void* stream) {
  if (ctx_lens == nullptr && ctx_len < 1) return KB_ERR_INVALID_ARG;
  // ctx_lens plays the part of starts in the checks: device positions, whole cache mapped
  const SparseCall c{q, k, v, o, nullptr, blocks, n_select, B, Hq, Hkv, 1, ctx_lens != nullptr ? 0 : ctx_len - 1, ctx_lens,
                     nullptr, kv_cap, block_table, pages_per_seq, page_size, num_pages, nullptr, 0};
  int cap = 0;
  kb::HostDevice dev;
  kb_status s = check_sparse(c, &cap, &dev);
  if (s != KB_OK) return s;
  CUtensorMap tk, tv;
  if ((s = cache_maps(c, &tk, &tv)) != KB_OK) return s;
  kb::PackedArgs a{};
  a.q = q;
  a.o = o;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.L = 1;
  a.start = c.start;
  a.ctx_lens = ctx_lens;
  a.max_ctx = cap;
  a.block_table = block_table;
  a.pages_per_seq = pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.n_sub = 1;
  a.fold_seg = kb::kSegTiles;
  a.blocks = blocks;
  a.n_select = n_select;
  const int max_blocks = ((ctx_lens != nullptr ? cap : ctx_len) + kb::kTileKeys - 1) / kb::kTileKeys;
  a.cluster = sparse_cluster(dev, B, Hkv, n_select, max_blocks);
  a.lean = a.cluster == 1 && static_cast<long long>(B) * Hkv > dev.sm_count;
  a.err = dev.err;
  return done(kb::launch_packed(tk, tv, a, 1, static_cast<cudaStream_t>(stream)));
}

size_t kb_attn_sparse_backward_workspace_bytes(int B, int Hkv, int S, int n_select) {
  if (kb_attn_sparse_workspace_bytes(B, Hkv, S, n_select, S) == 0) return 0;
  const long long blocks = (S + kb::kTileKeys - 1) / kb::kTileKeys;
  return static_cast<size_t>(bwd_sizes(plan_sizes(B, Hkv, S, n_select, blocks), B, Hkv, S).bytes);
}

kb_status kb_attn_sparse_backward(const void* q, const void* k, const void* v, const void* o, const void* dout,
                                  const float* lse, float* delta, const int* blocks, int n_select, void* dq, void* dk,
                                  void* dv, int B, int Hq, int Hkv, int S, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (!dout || !lse || !delta || !dq || !dk || !dv) return KB_ERR_INVALID_ARG;
  const void* outs[] = {dout, dq, dk, dv, lse, delta};
  for (int i = 0; i < 6; ++i)
    if (!host_aligned(outs[i], i < 4 ? 16 : 4)) return KB_ERR_INVALID_ARG;
  const SparseCall c{q, k, v, const_cast<void*>(o), nullptr, blocks, n_select, B, Hq, Hkv, S, 0, nullptr, nullptr, S,
                     nullptr, 0, 0, 0, workspace, workspace_bytes};
  int cap = 0;
  kb::HostDevice dev;
  kb_status s = check_sparse(c, &cap, &dev);
  if (s != KB_OK) return s;
  if ((s = device_pointers(outs, 6)) != KB_OK) return s;
  kb::SparseBwdArgs a{};
  if ((s = fill_plan(c, cap, dev.err, true, &a.plan)) != KB_OK) return s;
  if (2LL * a.plan.max_blocks * B * Hkv > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  a.q = q;
  a.dout = dout;
  const BwdSizes bwd = bwd_sizes(plan_sizes(B, Hkv, S, n_select, a.plan.max_blocks), B, Hkv, S);
  char* const ws = static_cast<char*>(workspace);
  a.n_split = static_cast<int>(bwd.n_split);
  a.tickets = reinterpret_cast<int*>(ws + bwd.tickets);
  a.n_jobs = reinterpret_cast<int*>(ws + bwd.jobs);
  a.jobs = reinterpret_cast<int2*>(ws + bwd.jobs + 8);
  a.sums = reinterpret_cast<float4*>(ws + bwd.sums);
  a.lse = lse;
  a.delta = delta;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  CUtensorMap tq, tk, tv, tdo;
  const uint64_t rows = static_cast<uint64_t>(S), groups = static_cast<uint64_t>(B) * Hkv;
  if ((s = kb::host_group_map(&tq, q, rows, groups)) != KB_OK) return s;
  if ((s = kb::host_group_map(&tdo, dout, rows, groups)) != KB_OK) return s;
  if ((s = cache_maps(c, &tk, &tv)) != KB_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(a.plan.row_counts, 0, static_cast<size_t>(bwd.jobs - bwd.counts), st);
  if (e == cudaSuccess) e = kb::launch_sparse_plan(a.plan, dev.index, st);
  if (e == cudaSuccess) e = kb::launch_bwd_delta(o, dout, delta, static_cast<long long>(B) * Hq * S, st);
  if (e == cudaSuccess) e = kb::launch_sparse_backward(tq, tk, tv, tdo, a, dev.index, dev.sm_count, st);
  return done(e);
}

}  // extern "C"

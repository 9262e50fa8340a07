// kb_launch.h -- host-side launchers of the attention kernels (internal; the
// public C ABI is include/kb_attn.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/kb_attn.h"

namespace kb {

struct PrefillArgs {
  void* o;          // [B, Hq, L, 128] bf16 output rows start..start+L-1
  int B, Hq, Hkv;
  int L;            // query rows in this call
  int start;        // absolute position of query row 0
  int first_tile;   // floor(start / 128)
  int n_tiles;      // absolute query tiles touched by [start, start+L)
  const int* block_table;  // optional device [B, pages_per_seq]: paged K/V pools
  int pages_per_seq, page_size, num_pages;
  const int* starts;       // optional device [B]: per-sequence start (ragged batch; then
  const int* lens;         //   L is the row stride of q and o and lens[b] <= L rows are used)
  int kv_cap;              // keys per sequence the cache can hold
  int group_major;         // CTA order: 1 = (b, g) slowest, 0 = query tile slowest
  float* lse;              // optional [B, Hq, L] fp32: natural-log log-sum-exp of each row's scaled scores
  int seg_tiles;           // C5 segment length in key tiles (0: the whole row is one segment)
  int max_ctas;            // CTAs of a persistent launch (one per SM)
  int persistent;          // schedule: kSchedOnePerCta, kSchedPairs or kSchedSnake
  uint32_t* err;    // device error word
};

// Query rows packed by GQA group (decode and chunks of at most 32 rows).
struct PackedArgs {
  const void* q;           // [B, Hq, L, 128] bf16
  void* o;                 // [B, Hq, L, 128] bf16
  int B, Hq, Hkv;
  int L;                   // query rows per (batch, head)
  int start;               // absolute position of query row 0 (when ctx_lens is null)
  const int* ctx_lens;     // optional device [B]: row L-1 of batch b sits at ctx_lens[b] - 1
  int max_ctx;             // largest valid ctx_lens entry (cache capacity)
  const int* block_table;  // optional device [B, pages_per_seq]: paged K/V pools
  int pages_per_seq, page_size, num_pages;
  const int* starts;       // optional device [B]: per-sequence start and row count (ragged
  const int* lens;         //   batch); L is then the row stride of q and o
  int n_sub;               // sub-chunks per (b, kv head) in the grid (1 or 2)
  // fold mode (part == nullptr): C5 segments of fold_seg key tiles, cut into
  // contiguous blocks over a cluster of `cluster` CTAs per (sub, b, g); the
  // cluster's first CTA folds them all and writes o
  int fold_seg, cluster;
  // workspace mode (part != nullptr): CTA (seg, sub, b, g) runs key tiles
  // [seg * seg_tiles, +seg_tiles) from the fresh state and writes the rows'
  // partial (O[128], m, mc, l) to part[((b*Hq + h)*L + r)*n_seg + seg][132]
  int seg_tiles, n_seg;
  float* part;
  // block-sparse tokens (L = 1, fold mode): device [B, Hkv, n_select] listed key blocks
  const int* blocks;
  int n_select;
  bool lean;               // more units than SMs (cluster 1): the shape of which two CTAs share an SM
  uint32_t* err;
};

constexpr int kPartFloats = 132;   // one partial: O[128], m, mc, l, pad

constexpr int kMaxPackedRows = 32;   // query rows per (batch, head) the packed kernel takes

// One 128-row query tile per CTA, one CTA per SM, three S buffers in TMEM
// and separate Q K^T / P V issuers, so the tensor pipe works on later key
// tiles while the softmax runs (CTA shape 3).
constexpr int kShapeOneTilePerSm = 3;
// The same kernel with the persistent launch forced (tests of the schedule):
// 4 with pairs of query tiles, 5 with the snake.
constexpr int kShapePersistent = 4;
constexpr int kShapeSnake = 5;
// The tile kernel's schedules (PrefillArgs::persistent).
constexpr int kSchedOnePerCta = 0;   // one CTA per unit
constexpr int kSchedPairs = 1;       // persistent, balanced pairs of query tiles, group-major
constexpr int kSchedSnake = 2;       // persistent, single units longest first, dealt back and forth
cudaError_t launch_prefill_s2(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PrefillArgs& a, cudaStream_t s);
// n_sub: 1, or 2 when the chunk crosses a 128-position tile boundary.
cudaError_t launch_packed(const CUtensorMap& tk, const CUtensorMap& tv, const PackedArgs& a, int n_sub,
                          cudaStream_t s);
// Partials a CTA of the narrow packed kernel can keep in shared memory for
// the cluster's first CTA, with n_rows packed rows.
uint32_t packed_partial_slots(int n_rows, bool sparse = false);
// Clusters of 2, 4 and 8 CTAs (entries 1, 2, 3) of the narrow packed kernel
// the current device runs at once; entry 0 is unused.
void packed_cluster_capacity(int (&active)[4]);
// Gradient of a whole-sequence causal prefill (query row i at position i).
struct BwdArgs {
  const void* o;           // [B, Hq, S, 128] bf16 forward output
  const void* dout;        // [B, Hq, S, 128] bf16 gradient of the output
  const float* lse;        // [B, Hq, S] natural-log log-sum-exp from the forward
  float* delta;            // [B, Hq, S] out: rowsum(dout * o)
  void* dq;                // [B, Hq, S, 128] bf16 out
  void* dk;                // [B, Hkv, S, 128] bf16 out
  void* dv;                // [B, Hkv, S, 128] bf16 out
  int B, Hq, Hkv, S;
  int n_tiles;             // ceil(S / 128)
  int group_major;         // CTA order of the dq kernel (as PrefillArgs)
  uint32_t* err;
};
// delta, then dq (query-major), then dk/dv (key-major), all on stream s.
// tq, tdo: [B*Hq planes, S rows]; tk, tv: [B*Hkv planes, S rows].
cudaError_t launch_backward(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& tdo, const BwdArgs& a, cudaStream_t s);
// delta[row] = rowsum(dout * o) of `rows` rows of 128.
cudaError_t launch_bwd_delta(const void* o, const void* dout, float* delta, long long rows, cudaStream_t s);
// C5 fold of the packed kernel's per-segment partials, one warp per row
// (rows = B*Hq*L, row r of a (b, h) at position start + r), then C4 into o.
cudaError_t launch_seg_fold(const float* part, void* o, long long rows, int L, int start, int seg_tiles, int n_seg,
                            cudaStream_t s);

// Rotation of rows x[b, h, i] (strides in elements, last dimension contiguous)
// at positions start + i into contiguous out [B, H, L, 128] (kb_append.cu).
struct RopeArgs {
  const void* x;
  long long sb, sh, sl;
  void* out;
  const float* table;      // [positions, rot_dim / 2, 2] (cos, sin)
  int rot_dim;
  bool interleaved, inverse;
  int B, H, L;
  int start;
  uint32_t* err;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);
// (cos, sin) of position * inv_freq[plane], positions 0..n_pos-1.
cudaError_t launch_rope_table(float* table, int n_pos, int rot_dim, const double* inv_freq, cudaStream_t s);

// Append L new rows per sequence to a K/V cache, turned by their positions.
struct AppendArgs {
  const void *q, *k, *v;       // [B, Hq or Hkv, L, 128], last dimension contiguous; q may be null
  long long qs[3], ks[3], vs[3];   // their batch, head and row strides in elements
  void* q_out;                 // [B, Hq, L, 128] contiguous
  void *k_cache, *v_cache;     // [B, Hkv, kv_cap, 128], or pools [num_pages, Hkv, page_size, 128]
  void* boxes;                 // optional: [planes, blocks per plane, 2, 128] bf16
  const float* table;          // as RopeArgs; null: no rotation
  int n_pos, rot_dim;
  bool interleaved;
  int B, Hkv, L;
  int start;
  const int* starts;           // optional device [B]: per-sequence start ...
  const int* lens;             // ... and row count (else L)
  int kv_cap;                  // positions per sequence the cache can hold
  const int* block_table;
  int pages_per_seq, page_size, num_pages;
  uint32_t* err;
};
// only_boxes: read the cache's keys at the rows' positions and make their
// blocks' boxes anew (q, k, v unused).
cudaError_t launch_append(const AppendArgs& a, bool only_boxes, int sm_count, cudaStream_t s);

// Choice of key blocks per query row (kb_select.cu).
struct SelectArgs {
  const void* q;               // [B, Hq, L, 128] bf16
  const void* boxes;           // [planes, blocks_per_plane, 2, 128] bf16
  int* blocks;                 // [B, Hkv, L, n]
  int B, Hkv, L, n;
  int keep_first, keep_last;
  int start;
  const int* starts;           // optional device [B] ...
  const int* lens;             // ... and row counts (else L)
  int kv_cap;
  int blocks_per_plane;        // boxes per (batch, KV head), or per (page, KV head)
  int max_blocks;              // blocks of the longest row the call can hold
  const int* block_table;
  int pages_per_seq, num_pages;
  uint32_t* err;
};
cudaError_t launch_select(const SelectArgs& a, int device, cudaStream_t s);

// Block-sparse attention over listed key blocks (kb_sparse.cuh, kb_sparse*.cu).
struct SparseArgs {
  void* o;                     // [B, Hq, L, 128] bf16
  float* lse;                  // optional [B, Hq, L]
  const int* blocks;           // [B, Hkv, L, n_select]
  int n_select;
  int B, Hq, Hkv, L;
  int start;
  const int* starts;           // optional device [B] ...
  const int* lens;             // ... and row counts (else L)
  int kv_cap;                  // positions per sequence the cache can hold
  int max_blocks;              // key blocks of the longest row the call can hold
  const int* block_table;
  int pages_per_seq, page_size, num_pages;
  int n_tiles;                 // units per (b, KV head): position tiles a sequence can touch
  int n_units;                 // B * Hkv * n_tiles
  int walk_cap;                // entries a unit's walk can have
  int* walk_len;               // workspace [n_units]: entries (-1: no such unit)
  uint2* walks;                // workspace [n_units][walk_cap]
  // backward: workspace [B * Hkv][max_blocks][n_tiles], the row mask of
  // position tile t for key block j (written for the blocks up to the tile's own)
  uint32_t* masks;
  int* row_counts;             // backward: workspace [B * Hkv][max_blocks], rows that listed a block (zeroed before)
  uint32_t* err;
};
cudaError_t launch_sparse_plan(const SparseArgs& a, int device, cudaStream_t s);
// tq: host_group_map of q; tk, tv: host_rows_map of the cache.
cudaError_t launch_sparse_tile(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const SparseArgs& a, int device, int sm_count, cudaStream_t s);

// Steps of 32 positions from which on two CTAs share a key block's gradient.
constexpr int kSparseSplitSteps = 128;

// Gradient of whole-sequence block-sparse attention (kb_sparse_bwd.cu).
struct SparseBwdArgs {
  const void *q, *dout;        // [B, Hq, S, 128] bf16
  const float* lse;            // [B, Hq, S]
  const float* delta;          // [B, Hq, S]
  void *dq, *dk, *dv;
  int n_split;                 // key blocks 0 .. n_split-1 may have kSparseSplitSteps steps or more
  float4* sums;                // workspace [B * Hkv][n_split][2 CTAs]: fp32 dv and dk, 128 KB each
  int* tickets;                // workspace [B * Hkv][n_split], zeroed before
  int2* jobs;                  // workspace: the dk/dv kernel's jobs, longest first ...
  int* n_jobs;                 // ... and how many
  SparseArgs plan;             // units, walks and masks of the call
};
// tq, tdo: host_group_map of q and dout; tk, tv: host_rows_map of k and v.
cudaError_t launch_sparse_backward(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CUtensorMap& tdo, const SparseBwdArgs& a, int device, int sm_count,
                                   cudaStream_t s);

cudaError_t launch_wait_probe(uint32_t* err, unsigned long long limit_ns, cudaStream_t s);

}  // namespace kb

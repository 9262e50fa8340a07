// kb_host_cache.cu -- C entry points of smaller caches: a cache held in 8 bits
// and the attention over it, rotation by positions of several axes.
// Declarations and their contract are in include/kb_attn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/kb_attn.h"
#include "kb_contract.cuh"
#include "kb_host.h"
#include "kb_launch.h"

namespace {

using kb::host_aligned;
using kb::host_cache_rows;
using kb::host_check_ragged;
using kb::host_check_strides;
using kb::host_check_table;
using kb::host_device_pointers;
using kb::host_done;
using kb::kMaxRows;

long long blocks_of(long long rows) { return (rows + kb::kTileKeys - 1) / kb::kTileKeys; }

long long align256(long long n) { return (n + 255) / 256 * 256; }

// An attention call over a cache held in 8 bits.
struct Call8 {
  const void *q, *k, *v;
  const int8_t *k_exp, *v_exp;
  void* o;
  int B, Hq, Hkv, L, start;
  const int *starts, *lens, *ctx_lens;
  int kv_cap;
  const int* block_table;
  int pages_per_seq, page_size, num_pages;
};

kb_status check_call(const Call8& c, int* cap, kb::HostDevice* dev) {
  if (!c.q || !c.k || !c.v || !c.k_exp || !c.v_exp || !c.o) return KB_ERR_INVALID_ARG;
  for (const void* p : {c.q, c.k, c.v, static_cast<const void*>(c.o)})
    if (!host_aligned(p, 16)) return KB_ERR_INVALID_ARG;
  if (!host_aligned(c.starts, 4) || !host_aligned(c.lens, 4) || !host_aligned(c.ctx_lens, 4)) return KB_ERR_INVALID_ARG;
  if ((c.starts == nullptr) != (c.lens == nullptr)) return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(c.B, c.Hq, c.Hkv);
  if (s != KB_OK) return s;
  if ((s = host_cache_rows(cap, c.kv_cap, c.block_table, c.pages_per_seq, c.page_size, c.num_pages, c.Hkv)) != KB_OK) return s;
  if (c.L < 1 || c.L > *cap) return KB_ERR_INVALID_ARG;
  if (c.starts == nullptr && c.ctx_lens == nullptr && (c.start < 0 || c.start > *cap - c.L)) return KB_ERR_INVALID_ARG;
  if ((s = kb::host_device(dev)) != KB_OK) return s;
  const void* p[] = {c.q, c.k, c.v, c.k_exp, c.v_exp, c.o, c.starts, c.lens, c.ctx_lens, c.block_table};
  return host_device_pointers(p, 10);
}

// Segments of 1024 keys of the longest sequence a call over `rows` positions can have.
long long segments_of(long long rows) { return (blocks_of(rows) + kb::kSegTiles - 1) / kb::kSegTiles; }

// Bytes of the segments' partials of a call that reads the bytes, where CTAs
// can share a KV head's segments: 0 for batches that fill the SMs without, and
// where the partials would pass 1 GB.
constexpr long long kMaxSplitUnits = 304;

// Tokens whose segments find an SM each in clusters: a cluster's CTAs meet in
// shared memory and need no workspace (5 segments of one sequence: the same 16 us
// on the GPU, 11 instead of 20 on the host).  Clusters of up to four fill four
// fifths of the 152 SMs, larger ones less (16 of seven take two waves).
bool in_clusters(int B, int Hkv, int L, long long rows) {
  const long long n = segments_of(rows);
  return L == 1 && n >= 2 && n <= 8 && static_cast<long long>(B) * Hkv * n <= (n <= 4 ? 120 : 96);
}

long long partial_bytes(int B, int Hkv, int L, long long rows) {
  if (static_cast<long long>(B) * Hkv >= kMaxSplitUnits || segments_of(rows) < 2 || in_clusters(B, Hkv, L, rows)) return 0;
  const long long n = static_cast<long long>(B) * Hkv * kb::kGroup * L * segments_of(rows) * kb::kPartFloats * 4;
  return n <= (1LL << 30) ? align256(n) : 0;
}

// Sub-chunks of a call: the rows of one tile's positions each, of 32 positions in a chunk of more than 32 rows.
int sub_chunks(int L, int start, bool ragged) {
  const int cell = L > kb::kMaxPackedRows ? kb::kMaxPackedRows : kb::kTileKeys;
  if (L == 1) return 1;                                               // (one row never crosses a tile boundary)
  return ragged ? (L - 2) / cell + 2 : (start + L - 1) / cell - start / cell + 1;
}

// CTAs that share the segments of a unit (a sub-chunk of a batch entry and KV
// head): the number for which the waves of CTAs take the least time, and that
// time in us.  A segment counts as 7.8 us (tokens) or 10.5 (chunks), a CTA's
// start and end as 6, the fold of the partials as 5 and their bytes, written and
// read, as 2 MB a us (fitted to timings of 1 to 19 CTAs at 16K, 32K and 64K,
// and of 64 to 256 rows at 28K and 32K).
struct Split {
  int ctas;
  double us;
};
Split choose_split(int sm_count, long long units, long long segments, bool token, long long part) {
  const double seg_us = token ? 7.8 : 10.5;
  auto cost = [&](long long split) {
    const long long waves = (units * split + sm_count - 1) / sm_count;
    return waves * (static_cast<double>((segments + split - 1) / split) * seg_us + 6.0) +
           (split > 1 ? 5.0 + static_cast<double>(part) / 2e6 : 0.0);
  };
  Split best{1, cost(1)};
  for (int n = 2; part > 0 && n <= segments && n <= sm_count; ++n)
    if (cost(n) < best.us) best = {n, cost(n)};
  return best;
}

// Tokens: the time in us of runs of all segments, one per SM, cut where the
// SMs' shares end; a piece of a KV head begins and ends in 4 us.
double flat_us(int sm_count, long long units, long long segments, long long part) {
  const long long run = (units * segments + sm_count - 1) / sm_count;
  return run * 7.8 + (static_cast<double>(run) / segments + 1.0) * 4.0 + 9.0 + static_cast<double>(part) / 2e6;
}

// The time in us of a chunk's other way: its keys and values into bf16 in the
// workspace (3 bytes moved for each, at 5.5 TB/s), then the bf16 chunk, 0.8 us a
// tile of a head's rows and a tile of keys on one SM (64 to 1000 rows at 32K;
// a ragged batch's grid has the tiles that its rows can touch).
double gathered_us(int sm_count, int B, int Hkv, int L, int start, bool ragged, long long rows) {
  const long long per_head = ragged ? (L + kb::kTileRows - 2) / kb::kTileRows + 1 : (start + L - 1) / kb::kTileRows - start / kb::kTileRows + 1;
  const long long tiles = static_cast<long long>(B) * Hkv * kb::kGroup * per_head;
  return 2.0 + static_cast<double>(B) * Hkv * rows * kb::kHeadDim * 6 / 5.5e6 + (tiles + sm_count - 1) / sm_count * (blocks_of(rows) * 0.8 + 2.0);
}

// The packed kernels read the bytes.
kb_status packed8(const Call8& c, int cap, const kb::HostDevice& dev, void* workspace, size_t workspace_bytes, void* stream) {
  const bool ragged = c.starts != nullptr;
  const int n_sub = sub_chunks(c.L, c.start, ragged);
  kb::PackedArgs a{};
  a.q = c.q;
  a.o = c.o;
  a.B = c.B;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.L = c.L;
  a.start = c.start;
  a.ctx_lens = c.ctx_lens;
  a.max_ctx = cap;
  a.block_table = c.block_table;
  a.pages_per_seq = c.pages_per_seq;
  a.page_size = c.page_size;
  a.num_pages = c.num_pages;
  a.starts = c.starts;
  a.lens = c.lens;
  a.n_sub = n_sub;
  const long long keys = ragged || c.ctx_lens != nullptr ? cap : static_cast<long long>(c.start) + c.L;
  a.fold_seg = kb::kSegTiles;
  a.cluster = in_clusters(c.B, c.Hkv, c.L, keys) ? static_cast<int>(segments_of(keys)) : 1;
  a.k_exp = c.k_exp;
  a.v_exp = c.v_exp;
  a.plane_rows = c.block_table != nullptr ? c.page_size : c.kv_cap;
  a.err = dev.err;
  // the maps end where the attention's do: a contiguous uniform cache at the call's last key
  const bool paged = c.block_table != nullptr;
  const uint64_t rows = paged || ragged || c.ctx_lens != nullptr ? static_cast<uint64_t>(a.plane_rows) : static_cast<uint64_t>(keys);
  const uint64_t planes = static_cast<uint64_t>(paged ? c.num_pages : c.B) * c.Hkv;
  const uint64_t stride = static_cast<uint64_t>(a.plane_rows) * kb::kHeadDim;
  CUtensorMap tk, tv;
  kb_status s = kb::host_bytes_map(&tk, c.k, rows, planes, stride);
  if (s != KB_OK) return s;
  if ((s = kb::host_bytes_map(&tv, c.v, rows, planes, stride)) != KB_OK) return s;
  const long long part = partial_bytes(c.B, c.Hkv, c.L, keys);
  int share = 1, flat = 0;
  if (workspace != nullptr) {
    if (!host_aligned(workspace, 256) || workspace_bytes < static_cast<size_t>(part)) return KB_ERR_INVALID_ARG;
    if ((s = kb::host_device_pointer(workspace)) != KB_OK) return s;
    if (part > 0) {
      const long long units = static_cast<long long>(c.B) * c.Hkv * (c.L > kb::kMaxPackedRows ? n_sub : 1);
      const Split best = choose_split(dev.sm_count, units, segments_of(keys), c.L <= kb::kMaxRows8, part);
      share = best.ctas;
      if (c.L == 1 && flat_us(dev.sm_count, units, segments_of(keys), part) < best.us) flat = dev.sm_count;
    }
  }
  const auto launch = c.L <= kb::kMaxRows8 ? kb::launch_decode8 : kb::launch_packed;
  if (share == 1 && flat == 0) return host_done(launch(tk, tv, a, n_sub, static_cast<cudaStream_t>(stream)));
  a.cluster = 1;
  a.part = static_cast<float*>(workspace);
  a.n_seg = static_cast<int>(segments_of(keys));
  a.split = flat > 0 ? 0 : share;
  a.ctas = flat;
  if ((s = host_done(launch(tk, tv, a, n_sub, static_cast<cudaStream_t>(stream)))) != KB_OK) return s;
  kb::RowsFoldArgs f{};
  f.part = a.part;
  f.o = c.o;
  f.B = c.B;
  f.Hq = c.Hq;
  f.L = c.L;
  f.n_seg = a.n_seg;
  f.start = c.start;
  f.starts = c.starts;
  f.lens = c.lens;
  f.ctx_lens = c.ctx_lens;
  f.err = dev.err;
  return host_done(kb::launch_rows_fold(f, static_cast<cudaStream_t>(stream)));
}

// Bytes of one of the two bf16 caches that a longer chunk is computed from.
long long gathered_bytes(int B, int Hkv, long long rows) { return align256(static_cast<long long>(B) * Hkv * rows * kb::kHeadDim * 2); }

}  // namespace

extern "C" {

kb_status kb_attn_rope_axes(const void* x, const long long* strides, void* out, const float* table, int n_pos, int rot_dim,
                            int interleaved, int inverse, const int* positions, int n_axes, const unsigned char* plane_axes,
                            int B, int H, int L, void* stream) {
  if (!x || !out || !strides || !table || !positions || !plane_axes) return KB_ERR_INVALID_ARG;
  if (!host_aligned(x, 16) || !host_aligned(out, 16) || !host_aligned(positions, 4)) return KB_ERR_INVALID_ARG;
  kb_status s = host_check_table(table, n_pos, rot_dim);
  if (s != KB_OK) return s;
  if ((s = host_check_strides(strides)) != KB_OK) return s;
  if (B < 1 || H < 1 || L < 1 || n_axes < 1) return KB_ERR_INVALID_ARG;
  if (n_axes > kb::kMaxAxes) return KB_ERR_UNSUPPORTED;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (plane_axes[i] >= n_axes) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * ((H + 3) / 4) * ((L + 3) / 4) > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {x, out, table, positions};
  if ((s = host_device_pointers(p, 4)) != KB_OK) return s;
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
  a.positions = positions;
  a.n_axes = n_axes;
  a.n_pos = n_pos;
  for (int i = 0; i < rot_dim / 2; ++i)
    a.plane_axes[i / kb::kPlanesPerLane] |= static_cast<uint64_t>(plane_axes[i]) << (8 * (i % kb::kPlanesPerLane));
  a.err = dev.err;
  return host_done(kb::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

kb_status kb_attn_append_8bit(const void* q, const void* k, const void* v, const long long* strides, void* q_out,
                              void* k_cache, void* v_cache, signed char* k_exp, signed char* v_exp, const float* table,
                              int n_pos, int rot_dim, int interleaved, int B, int Hq, int Hkv, int L, int start,
                              const int* starts, const int* lens, int kv_cap, const int* block_table, int pages_per_seq,
                              int page_size, int num_pages, void* stream) {
  if (!k || !v || !strides || !k_cache || !v_cache || !k_exp || !v_exp || (q == nullptr) != (q_out == nullptr))
    return KB_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, static_cast<const void*>(q_out), static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
    if (!host_aligned(p, 16)) return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(B, Hq, Hkv);
  if (s != KB_OK) return s;
  if (table != nullptr && (s = host_check_table(table, n_pos, rot_dim)) != KB_OK) return s;
  for (int i = q == nullptr ? 1 : 0; i < 3; ++i)
    if ((s = host_check_strides(strides + 3 * i)) != KB_OK) return s;
  if ((s = host_check_ragged(starts, lens)) != KB_OK) return s;
  int cap = 0;
  if ((s = host_cache_rows(&cap, kv_cap, block_table, pages_per_seq, page_size, num_pages, Hkv)) != KB_OK) return s;
  if (L < 1 || L > cap) return KB_ERR_INVALID_ARG;
  if (starts == nullptr && (start < 0 || start > cap - L || (table != nullptr && start > n_pos - L))) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * Hkv * (blocks_of(L) + 1) > 0x3FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {q, k, v, q_out, k_cache, v_cache, k_exp, v_exp, table, starts, lens, block_table};
  if ((s = host_device_pointers(p, 12)) != KB_OK) return s;
  kb::Append8Args x{};
  kb::AppendArgs& a = x.a;
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
  x.k_exp = reinterpret_cast<int8_t*>(k_exp);
  x.v_exp = reinterpret_cast<int8_t*>(v_exp);
  return host_done(kb::launch_append8(x, static_cast<cudaStream_t>(stream)));
}

kb_status kb_attn_cache_values(const void* cache, const signed char* exps, void* out, long long planes, int rows, void* stream) {
  if (!cache || !exps || !out || !host_aligned(cache, 16) || !host_aligned(out, 16)) return KB_ERR_INVALID_ARG;
  if (planes < 1 || rows < 1) return KB_ERR_INVALID_ARG;
  if (rows > kMaxRows || planes > 0x7FFFFFFFLL / blocks_of(rows)) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  kb_status s = kb::host_device(&dev);
  if (s != KB_OK) return s;
  const void* p[] = {cache, exps, out};
  if ((s = host_device_pointers(p, 3)) != KB_OK) return s;
  kb::Values8Args a{};
  a.cache = cache;
  a.exps = reinterpret_cast<const int8_t*>(exps);
  a.out = out;
  a.planes = planes;
  a.rows = rows;
  a.blocks = static_cast<int>(blocks_of(rows));
  a.err = dev.err;
  return host_done(kb::launch_cache_values(a, static_cast<cudaStream_t>(stream)));
}

size_t kb_attn_chunk_8bit_workspace_bytes(int B, int Hkv, int L, int rows) {
  if (B < 1 || Hkv < 1 || L < 1 || rows < L || rows > kMaxRows) return 0;
  if (L <= kb::kMaxPackedRows) return static_cast<size_t>(partial_bytes(B, Hkv, L, rows));
  return static_cast<size_t>(std::max(2 * gathered_bytes(B, Hkv, rows), partial_bytes(B, Hkv, L, rows)));
}

kb_status kb_attn_chunk_8bit(const void* q, const void* k, const void* v, const signed char* k_exp, const signed char* v_exp,
                             void* o, int B, int Hq, int Hkv, int L, int start, const int* starts, const int* lens,
                             int kv_cap, const int* block_table, int pages_per_seq, int page_size, int num_pages,
                             void* workspace, size_t workspace_bytes, void* stream) {
  Call8 c{q, k, v, reinterpret_cast<const int8_t*>(k_exp), reinterpret_cast<const int8_t*>(v_exp), o, B, Hq, Hkv, L,
          starts ? 0 : start, starts, lens, nullptr, kv_cap, block_table, pages_per_seq, page_size, num_pages};
  int cap = 0;
  kb::HostDevice dev;
  kb_status s = check_call(c, &cap, &dev);
  if (s != KB_OK) return s;
  if (L <= kb::kMaxPackedRows) return packed8(c, cap, dev, workspace, workspace_bytes, stream);
  const int rows = starts != nullptr ? cap : start + L;
  const size_t need = kb_attn_chunk_8bit_workspace_bytes(B, Hkv, L, rows);
  if (workspace == nullptr || !host_aligned(workspace, 256) || workspace_bytes < need) return KB_ERR_INVALID_ARG;
  if ((s = kb::host_device_pointer(workspace)) != KB_OK) return s;
  if (static_cast<long long>(B) * Hkv * blocks_of(rows) > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  const long long units = static_cast<long long>(B) * Hkv * sub_chunks(L, c.start, starts != nullptr);
  if (units <= 8LL * dev.sm_count && choose_split(dev.sm_count, units, segments_of(rows), false, partial_bytes(B, Hkv, L, rows)).us <
                                         gathered_us(dev.sm_count, B, Hkv, L, c.start, starts != nullptr, rows))
    return packed8(c, cap, dev, workspace, workspace_bytes, stream);
  kb::Gather8Args a{};
  a.k = k;
  a.v = v;
  a.k_exp = c.k_exp;
  a.v_exp = c.v_exp;
  a.k_out = workspace;
  a.v_out = static_cast<char*>(workspace) + gathered_bytes(B, Hkv, rows);
  a.B = B;
  a.Hkv = Hkv;
  a.L = L;
  a.rows = rows;
  a.blocks = static_cast<int>(blocks_of(rows));
  a.starts = starts;
  a.lens = lens;
  a.kv_cap = kv_cap;
  a.block_table = block_table;
  a.pages_per_seq = pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.err = dev.err;
  if ((s = host_done(kb::launch_cache_gather(a, static_cast<cudaStream_t>(stream)))) != KB_OK) return s;
  if (starts != nullptr)
    return kb_attn_chunk_varlen(q, a.k_out, a.v_out, o, B, Hq, Hkv, L, starts, lens, rows, nullptr, 0, 0, 0, stream);
  return kb_attn_chunk(q, a.k_out, a.v_out, o, B, Hq, Hkv, L, start, rows, stream);
}

kb_status kb_attn_decode_8bit(const void* q, const void* k, const void* v, const signed char* k_exp, const signed char* v_exp,
                              void* o, int B, int Hq, int Hkv, int ctx_len, const int* ctx_lens, int kv_cap,
                              const int* block_table, int pages_per_seq, int page_size, int num_pages, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (ctx_lens == nullptr && ctx_len < 1) return KB_ERR_INVALID_ARG;
  Call8 c{q, k, v, reinterpret_cast<const int8_t*>(k_exp), reinterpret_cast<const int8_t*>(v_exp), o, B, Hq, Hkv, 1,
          ctx_lens ? 0 : ctx_len - 1, nullptr, nullptr, ctx_lens, kv_cap, block_table, pages_per_seq, page_size, num_pages};
  int cap = 0;
  kb::HostDevice dev;
  const kb_status s = check_call(c, &cap, &dev);
  return s != KB_OK ? s : packed8(c, cap, dev, workspace, workspace_bytes, stream);
}

kb_status kb_attn_key_weights(const void* q, const void* k, const float* lse, float* weights, int B, int Hq, int Hkv, int L,
                              int start, const int* starts, const int* lens, int kv_cap, const int* block_table,
                              int pages_per_seq, int page_size, int num_pages, void* stream) {
  if (!q || !k || !lse || !weights || !host_aligned(q, 16) || !host_aligned(k, 16)) return KB_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(lse), static_cast<const void*>(weights), static_cast<const void*>(starts),
                        static_cast<const void*>(lens)})
    if (!host_aligned(p, 4)) return KB_ERR_INVALID_ARG;
  if ((starts == nullptr) != (lens == nullptr)) return KB_ERR_INVALID_ARG;
  kb_status s = kb::host_check_heads(B, Hq, Hkv);
  if (s != KB_OK) return s;
  int cap = 0;
  if ((s = host_cache_rows(&cap, kv_cap, block_table, pages_per_seq, page_size, num_pages, Hkv)) != KB_OK) return s;
  if (L < 1 || L > cap || (starts == nullptr && (start < 0 || start > cap - L))) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * Hkv * blocks_of(cap) > 0x7FFFFFFFLL) return KB_ERR_UNSUPPORTED;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {q, k, lse, weights, starts, lens, block_table};
  if ((s = host_device_pointers(p, 7)) != KB_OK) return s;
  // K map as the attention's: a contiguous uniform cache ends at the call's last key
  const uint64_t row_bytes = kb::kHeadDim * 2u;
  const bool paged = block_table != nullptr;
  const uint64_t stride_rows = static_cast<uint64_t>(paged ? page_size : kv_cap);
  const uint64_t rows = paged || starts != nullptr ? stride_rows : static_cast<uint64_t>(start) + L;
  const bool few = L <= kb::kMaxPackedRows;
  CUtensorMap tq, tk;
  if ((s = (few ? kb::host_rows_map : kb::host_halves_map)(&tk, k, rows, static_cast<uint64_t>(paged ? num_pages : B) * Hkv,
                                                          stride_rows * row_bytes)) != KB_OK)
    return s;
  // (a group's four heads are one run of rows)
  const uint64_t group_rows = static_cast<uint64_t>(kb::kGroup) * L;
  if (!few && (s = kb::host_rows_map(&tq, q, group_rows, static_cast<uint64_t>(B) * Hkv, group_rows * row_bytes)) != KB_OK) return s;
  kb::WeightsArgs a{};
  a.q = q;
  a.lse = lse;
  a.weights = weights;
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
  const int max_keys = starts != nullptr ? cap : start + L;
  const auto st = static_cast<cudaStream_t>(stream);
  return host_done(few ? kb::launch_weights(tk, a, max_keys, dev.sm_count, st)
                       : kb::launch_weights_rows(tq, tk, a, max_keys, dev.sm_count, st));
}

kb_status kb_attn_evict(void* k, void* v, const float* weights, float* weights_out, int* kept, int B, int Hkv, const int* lens,
                        int keep, int keep_first, int keep_last, int kv_cap, const int* block_table, int pages_per_seq,
                        int page_size, int num_pages, void* stream) {
  if (!k || !v || k == v || !weights || !weights_out || !kept || !lens || !host_aligned(k, 16) || !host_aligned(v, 16))
    return KB_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(weights), static_cast<const void*>(weights_out), static_cast<const void*>(kept),
                        static_cast<const void*>(lens)})
    if (!host_aligned(p, 4)) return KB_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1) return KB_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * Hkv > (1LL << 24)) return KB_ERR_UNSUPPORTED;
  int cap = 0;
  kb_status s = host_cache_rows(&cap, kv_cap, block_table, pages_per_seq, page_size, num_pages, Hkv);
  if (s != KB_OK) return s;
  if (keep < 1 || keep > cap || keep_first < 0 || keep_last < 0 || keep_first > keep - keep_last) return KB_ERR_INVALID_ARG;
  kb::HostDevice dev;
  if ((s = kb::host_device(&dev)) != KB_OK) return s;
  const void* p[] = {k, v, weights, weights_out, kept, lens, block_table};
  if ((s = host_device_pointers(p, 7)) != KB_OK) return s;
  kb::EvictArgs a{};
  a.k = k;
  a.v = v;
  a.weights = weights;
  a.weights_out = weights_out;
  a.kept = kept;
  a.B = B;
  a.Hkv = Hkv;
  a.lens = lens;
  a.keep = keep;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.kv_cap = cap;
  a.block_table = block_table;
  a.pages_per_seq = pages_per_seq;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.err = dev.err;
  return host_done(kb::launch_evict(a, dev.sm_count, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

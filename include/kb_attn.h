/*
 * kb_attn.h -- C ABI of libkb_attn.so: bitwise-aligned causal grouped-query
 * attention forward for NVIDIA GB300 (sm_103a).
 *
 * The operation (KernelBraid README, sections "Features" and "Usage / Use a
 * selected kernel"): BF16 causal attention over contiguous
 * [batch, heads, sequence, head_dim] tensors, 32 query heads sharing 8 KV
 * heads (query head h reads KV head h / 4), head_dim 128, scale 1/sqrt(128).
 * For a query row at absolute position p the output is
 *     o = sum_{j<=p} softmax_j(q . k_j / sqrt(128)) v_j.
 *
 * The three entry points follow one numerical contract (README "Method":
 * the contract connects full-sequence prefill, partitioned forward execution
 * and one-token decode; "Advantages": prefill and incremental decode give
 * bitwise-identical outputs).  A row at position p computed by
 * kb_attn_prefill, by kb_attn_chunk (any split of the sequence) and by
 * kb_attn_decode (ctx_len = p + 1) has the same bf16 bits.
 *
 * Contract version 3 (kb_contract_version): key tiles of 128 keys visited in
 * ascending order; one tcgen05 MMA shape and k-order; one per-row online
 * softmax (fp32 max and sum, one exp2 path, scale 1/sqrt(128)); one final
 * normalisation; and a fixed, length-determined split of every row's keys
 * into segments of 1024 keys (8 tiles) anchored at key 0, each segment run
 * from the fresh softmax state and the segments folded left to right by one
 * fold function.  The split lets a small-batch decode of a long context run
 * its segments on several SMs at once while prefill folds the same segments
 * in order, so both stay bit-identical.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers on the current CUDA device,
 *    bf16, contiguous, 16-byte aligned, owned by the caller.  The library
 *    never allocates, frees or keeps them.
 *  - Hq must equal 4 * Hkv (the GQA group size of the contract); head_dim is
 *    fixed at 128.  Other shapes return KB_ERR_UNSUPPORTED.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream) and do not synchronise the host.  Argument errors are
 *    reported before anything is enqueued.  A device-side wait that gave up
 *    (never expected) is reported by kb_attn_check_device_status.
 *  - Outputs are valid only once kb_attn_check_device_status has returned
 *    KB_OK after the call.  KB_OK from an entry point means only that the
 *    arguments passed the host checks and the kernels were enqueued.  When a
 *    kernel gives up on a wait or finds a device-resident argument out of
 *    range (a page index, a per-sequence length) it records that in the
 *    library's per-device error word; until kb_attn_check_device_status reads
 *    and clears that word, every later kernel on the device skips its work
 *    and leaves its output unwritten, although its entry point returns KB_OK.
 *  - The sizes are all the library sees of the buffers: it cannot check that
 *    a buffer is as large as its shape says.  A caller that passes sizes
 *    larger than its allocations makes the kernels read or write past them.
 *  - Rows of the KV cache beyond the visible context are never used, so they
 *    may hold anything (including NaN bit patterns).
 */
#ifndef KB_ATTN_H
#define KB_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kb_status {
    KB_OK = 0,
    KB_ERR_INVALID_ARG = 1,   /* null or misaligned pointer, non-positive size, not device memory */
    KB_ERR_UNSUPPORTED = 2,   /* shape outside the contract (Hq != 4*Hkv, sizes too large) */
    KB_ERR_CUDA = 3,          /* a CUDA runtime or driver call failed */
    KB_ERR_TIMEOUT = 4        /* a bounded device-side wait gave up (see kb_attn_check_device_status) */
} kb_status;

/*
 * Full-sequence causal prefill (README "Usage": unified_prefill(q, k, v, H_Q, H_KV)).
 *   q, o : [B, Hq, S, 128]   query rows are positions 0..S-1; o has q's shape
 *   k, v : [B, Hkv, S, 128]
 * Identical to kb_attn_chunk(q, k, v, o, B, Hq, Hkv, S, 0, S, stream).
 */
kb_status kb_attn_prefill(const void* q, const void* k, const void* v, void* o,
                          int B, int Hq, int Hkv, int S, void* stream);

/*
 * Partitioned (chunked) forward against a KV cache (README "Method":
 * partitioned forward execution; "Usage": prompt/answer splits).
 *   q, o : [B, Hq, L, 128]       query row i is absolute position start + i
 *   k, v : [B, Hkv, kv_cap, 128] rows 0..start+L-1 must already hold the keys
 *                                and values of every position up to the chunk's
 *                                last row (the caller appends the chunk's own
 *                                K/V before the call)
 * Requires L >= 1, start >= 0, start + L <= kv_cap.
 */
kb_status kb_attn_chunk(const void* q, const void* k, const void* v, void* o,
                        int B, int Hq, int Hkv, int L, int start, int kv_cap, void* stream);

/*
 * One-token decode (README "Usage": unified_decode(q[:, :, -1:], k, v, H_Q, H_KV)).
 *   q, o : [B, Hq, 1, 128]       the query sits at position ctx_len - 1
 *   k, v : [B, Hkv, kv_cap, 128] rows 0..ctx_len-1 are the visible context
 * Requires 1 <= ctx_len <= kv_cap.
 */
kb_status kb_attn_decode(const void* q, const void* k, const void* v, void* o,
                         int B, int Hq, int Hkv, int ctx_len, int kv_cap, void* stream);

/*
 * Partitioned (chunked) forward against a paged KV cache: as kb_attn_chunk,
 * with the keys and values of every sequence in pages of a shared pool (the
 * page table is this library's addition; the pages show only a contiguous
 * cache).
 *   q, o         : [B, Hq, L, 128]; query row i is absolute position start + i
 *   k_pages,
 *   v_pages      : pools [num_pages, Hkv, page_size, 128] bf16; positions
 *                  0..start+L-1 of every sequence must be written
 *   block_table  : device int32 [B, pages_per_seq]; key position p of batch b
 *                  lives in page block_table[b, p / page_size], row p % page_size
 * page_size must be a positive multiple of 128; start + L <= pages_per_seq *
 * page_size.  Bits equal kb_attn_chunk on the same data laid out contiguously.
 * An out-of-range page index is found on the device and reported by the next
 * kb_attn_check_device_status as KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_chunk_paged(const void* q, const void* k_pages, const void* v_pages, void* o,
                              int B, int Hq, int Hkv, int L, int start, const int* block_table,
                              int pages_per_seq, int page_size, int num_pages, void* stream);

/*
 * Ragged batch: chunked forward where every sequence has its own start
 * position and row count (device int32 arrays), against a contiguous cache
 * (block_table == NULL) or a paged pool.  A full prefill of sequences of
 * different lengths is starts[b] = 0, lens[b] = S_b.  (The per-sequence
 * lengths are this library's addition; the pages' workloads are uniform.)
 *   q, o     : [B, Hq, L_max, 128]; row i < lens[b] of batch b is position
 *              starts[b] + i; rows lens[b]..L_max-1 are neither read for any
 *              other row nor written
 *   k, v     : block_table == NULL: [B, Hkv, kv_cap, 128]
 *              else pools [num_pages, Hkv, page_size, 128] addressed as in
 *              kb_attn_chunk_paged (kv_cap is then pages_per_seq * page_size)
 *   starts,
 *   lens     : device int32 [B]; 0 <= lens[b] <= L_max, starts[b] >= 0,
 *              starts[b] + lens[b] <= kv_cap; keys 0..starts[b]+lens[b]-1 of
 *              every sequence must be written, later cache rows may hold anything
 * Bits equal kb_attn_chunk on each sequence alone.  Out-of-range starts, lens
 * or page indices are found on the device: those sequences are not written and
 * the next kb_attn_check_device_status returns KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_chunk_varlen(const void* q, const void* k, const void* v, void* o,
                               int B, int Hq, int Hkv, int L_max, const int* starts, const int* lens,
                               int kv_cap, const int* block_table, int pages_per_seq, int page_size,
                               int num_pages, void* stream);

/*
 * One-token decode over a paged KV cache, one context length per sequence
 * (README "Usage": unified_decode; the page table is this library's
 * addition, the pages show only a contiguous cache).
 *   q, o         : [B, Hq, 1, 128]; the query of batch b sits at position ctx_lens[b] - 1
 *   k_pages,
 *   v_pages      : pools [num_pages, Hkv, page_size, 128] bf16
 *   block_table  : device int32 [B, pages_per_seq]; key position p of batch b lives in
 *                  page block_table[b, p / page_size] at row p % page_size
 *   ctx_lens     : device int32 [B], each in 1 .. pages_per_seq * page_size
 * page_size must be a positive multiple of 128.  Page rows past a sequence's
 * context may hold anything.  Bits equal kb_attn_decode on the same keys and
 * values laid out contiguously.  Out-of-range ctx_lens or page indices are
 * found on the device: the affected rows are not written and the next
 * kb_attn_check_device_status returns KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_decode_paged(const void* q, const void* k_pages, const void* v_pages, void* o,
                               int B, int Hq, int Hkv, const int* block_table, int pages_per_seq,
                               int page_size, int num_pages, const int* ctx_lens, void* stream);

/*
 * Synchronises `stream`, then reads and clears the library's device-side
 * error word on the current device.  Returns KB_ERR_TIMEOUT if any kernel
 * since the last check gave up on a bounded wait (its output is then
 * undefined), KB_ERR_INVALID_ARG if a kernel found a device-resident argument
 * out of range, KB_ERR_CUDA if the synchronisation failed, else KB_OK.
 */
kb_status kb_attn_check_device_status(void* stream);

/*
 * Test hook for the failure path: enqueues a one-CTA kernel that waits on a
 * barrier nothing will signal, giving up after `limit_us` microseconds
 * (1..1000000).  A following kb_attn_check_device_status returns
 * KB_ERR_TIMEOUT.  Faults and hangs nothing.
 */
kb_status kb_attn_debug_wait_timeout(int limit_us, void* stream);

/*
 * Explicit segment length (contract C5 with seg_tiles instead of 8): a row's
 * key tiles are cut into segments of seg_tiles 128-key tiles anchored at key
 * 0; each segment runs the tile steps from the fresh state and the segments
 * are folded left to right by the contract's fold function, then normalised.
 * Every entry point below gives the same bits for a row at position p when
 * called with the same seg_tiles (>= 1).  seg_tiles = 8 gives the default
 * entry points' bits; a seg_tiles of at least the row's tile count is the
 * unsplit online softmax (contract version 2's default).  These calls run a
 * different fold path from the default entry points (short chunks write
 * per-segment partials to a workspace that a second kernel folds), so with
 * seg_tiles = 8 they also cross-check the default path's bits.
 *
 * kb_attn_prefill_seg: as kb_attn_prefill (no workspace).
 * kb_attn_chunk_seg:   as kb_attn_chunk.  Chunks of at most 32 rows (and
 *   decode) run one CTA per (segment, batch, KV head) and need a device
 *   workspace of kb_attn_seg_workspace_bytes(B, Hq, L, start, seg_tiles)
 *   bytes (16-byte aligned, caller-owned, contents scratch); longer chunks
 *   fold in the kernel and ignore it.  Too small a workspace returns
 *   KB_ERR_INVALID_ARG.
 * kb_attn_decode_seg:  as kb_attn_decode (a chunk of one row at ctx_len-1).
 * Paged and ragged caches are not offered in this mode (KB_ERR_UNSUPPORTED).
 */
kb_status kb_attn_prefill_seg(const void* q, const void* k, const void* v, void* o,
                              int B, int Hq, int Hkv, int S, int seg_tiles, void* stream);
kb_status kb_attn_chunk_seg(const void* q, const void* k, const void* v, void* o,
                            int B, int Hq, int Hkv, int L, int start, int kv_cap, int seg_tiles,
                            void* workspace, size_t workspace_bytes, void* stream);
kb_status kb_attn_decode_seg(const void* q, const void* k, const void* v, void* o,
                             int B, int Hq, int Hkv, int ctx_len, int kv_cap, int seg_tiles,
                             void* workspace, size_t workspace_bytes, void* stream);
/*
 * kb_attn_decode_seg without a caller workspace: the partials go to a 4 MiB
 * scratch array the library owns (one per device, part of the loaded module),
 * so the call allocates nothing and takes nothing but the decode's tensors.
 * It serves callers that cannot allocate device memory at the point of the
 * call: a serving loop whose memory pool is already handed out, or code that
 * must not enter the CUDA allocator (which may synchronise the device) in its
 * decode step.  No paper counterpart: it is a deployment variant of
 * kb_attn_decode_seg.
 * Requests needing more than 4 MiB of partials (B * Hq * segments * 528 bytes)
 * return KB_ERR_UNSUPPORTED before anything is enqueued.  The scratch is
 * shared and keeps the last call's contents (every call overwrites the part
 * it reads): calls of this entry point on one device that overlap on the GPU
 * race, so issue them on one stream.  The first call of any entry point on a
 * device looks up the scratch's device address (cudaGetSymbolAddress); make
 * that first call before any stream capture.  Bits equal kb_attn_decode_seg's.
 */
kb_status kb_attn_decode_seg_static(const void* q, const void* k, const void* v, void* o,
                                    int B, int Hq, int Hkv, int ctx_len, int kv_cap, int seg_tiles,
                                    void* stream);
/* Workspace bytes kb_attn_chunk_seg / kb_attn_decode_seg need for a chunk of
 * L <= 32 rows at positions start..start+L-1 (0 for bad arguments or L > 32). */
size_t kb_attn_seg_workspace_bytes(int B, int Hq, int L, int start, int seg_tiles);

/*
 * Training forward: kb_attn_prefill plus each row's log-sum-exp, which the
 * backward needs (README "Motivation": the RL policy update differentiates
 * the same attention).
 *   q, o, k, v : as kb_attn_prefill; o gets the same bits as kb_attn_prefill
 *   lse        : [B, Hq, S] fp32, device, 4-byte aligned, caller-owned;
 *                lse[b,h,i] = ln sum_{j<=i} exp(q_i . k_j / sqrt(128))
 * Always runs the default tile kernel (CTA shape 3), whose bits every other
 * shape reproduces.
 */
kb_status kb_attn_prefill_lse(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int Hq, int Hkv, int S, void* stream);

/*
 * Backward of the whole-sequence causal prefill (query row i at position i):
 * the gradients of q, k and v for a given gradient dout of the output.
 *   q, dout, o : [B, Hq, S, 128] bf16; o and lse from kb_attn_prefill_lse
 *   k, v       : [B, Hkv, S, 128] bf16
 *   lse        : [B, Hq, S] fp32 (input)
 *   delta      : [B, Hq, S] fp32 (output): delta[b,h,i] = dout_i . o_i
 *   dq         : [B, Hq, S, 128] bf16 (output)
 *   dk, dv     : [B, Hkv, S, 128] bf16 (output); each sums the four query
 *                heads of its group
 * With P the softmax rows recomputed from lse, dP_ij = dout_i . v_j and
 * dS_ij = P_ij (dP_ij - delta_i):
 *   dq_i = sum_j dS_ij k_j / sqrt(128),  dk_j = sum_{h,i} dS_ij q_i / sqrt(128),
 *   dv_j = sum_{h,i} P_ij dout_i   (P and dS rounded to bf16 for the products,
 *   fp32 accumulation, bf16 outputs).
 * No atomics: every output element is summed by one CTA in a fixed order, so
 * repeated calls give identical bits.  All pointers are device memory,
 * caller-owned; errors as for the forward entry points.
 */
kb_status kb_attn_backward(const void* q, const void* k, const void* v, const void* o, const void* dout,
                           const float* lse, float* delta, void* dq, void* dk, void* dv,
                           int B, int Hq, int Hkv, int S, void* stream);

/*
 * Position rotation (rotary embedding).  A row of 128 values at position p is
 * turned in rot_dim/2 planes; plane i holds values i and i + rot_dim/2 (or,
 * with interleaved != 0, values 2i and 2i+1) and turns by p * inv_freq[i]:
 *   a' = a cos - b sin,  b' = b cos + a sin   (fp32, rounded to bf16 once);
 * values from rot_dim on pass unchanged.  Without a paper counterpart: the
 * pages' attention takes queries and keys that are already turned.
 *
 * kb_attn_rope_table fills table [n_pos, rot_dim/2, 2] fp32 (16-byte aligned)
 * with (cos, sin) of p * inv_freq[i], angles formed in 64 bits; inv_freq is a
 * device array of rot_dim/2 doubles.  rot_dim: a multiple of 16 up to 128.
 *
 * kb_attn_rope turns x [B, H, L, 128] at positions start..start+L-1 (all
 * below n_pos) into contiguous out [B, H, L, 128].  strides: host array of
 * x's batch, head and row strides in elements (multiples of 8; the last
 * dimension is contiguous).  out may be x itself when x is contiguous, and
 * must not overlap it otherwise.  inverse != 0 turns by the negative angle,
 * which is the gradient of the rotation (dx from dout).
 */
kb_status kb_attn_rope_table(float* table, int n_pos, int rot_dim, const double* inv_freq, void* stream);
kb_status kb_attn_rope(const void* x, const long long* strides, void* out, const float* table, int n_pos,
                       int rot_dim, int interleaved, int inverse, int B, int H, int L, int start,
                       void* stream);

/*
 * Append L new positions per sequence to a KV cache: turns q and k by their
 * positions, writes k and v into the cache, q into q_out, and widens the
 * boxes of the key blocks that the new keys fall into.
 *   q       : [B, Hq, L, 128], k, v: [B, Hkv, L, 128] bf16 views; strides is a
 *             host array of nine: q's batch, head and row strides in elements,
 *             then k's, then v's (multiples of 8, last dimension contiguous),
 *             so slices of one fused projection need no copy.  q and q_out may
 *             be NULL together.
 *   q_out   : [B, Hq, L, 128] contiguous; may be q itself when q is contiguous,
 *             and must not overlap it otherwise
 *   k_cache,
 *   v_cache : block_table == NULL: [B, Hkv, kv_cap, 128], else pools
 *             [num_pages, Hkv, page_size, 128] as in kb_attn_chunk_paged
 *   boxes   : NULL, or bf16 [B, Hkv, ceil(kv_cap/128), 2, 128], or with a page
 *             table [num_pages, Hkv, page_size/128, 2, 128]: per block of 128
 *             keys the upper and lower bound of every channel (see
 *             kb_attn_block_boxes)
 *   table   : from kb_attn_rope_table, or NULL (no rotation)
 *   start   : position of row 0 of every sequence when starts is NULL
 *   starts,
 *   lens    : NULL, or device int32 [B]: row i < lens[b] (L rows when lens is
 *             NULL) of sequence b goes to position starts[b] + i; rows from
 *             lens[b] on are neither read nor written
 * A block whose first key is among the new ones gets a new box; any other
 * touched block's box must hold its earlier keys' bounds and is widened, so
 * keys overwritten inside a block leave their old bounds in its box until
 * kb_attn_block_boxes makes it anew.
 * Keys, queries and boxes have the same bits for any split of a sequence into
 * appends.  No two sequences may append to the same page.  Out-of-range
 * starts, lens or page indices are found on the device: that sequence (or
 * block) is not written and the next kb_attn_check_device_status returns
 * KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_append(const void* q, const void* k, const void* v, const long long* strides, void* q_out,
                         void* k_cache, void* v_cache, void* boxes, const float* table, int n_pos,
                         int rot_dim, int interleaved, int B, int Hq, int Hkv, int L, int start,
                         const int* starts, const int* lens, int kv_cap, const int* block_table,
                         int pages_per_seq, int page_size, int num_pages, void* stream);

/*
 * Boxes of the blocks of a cache's first kv_len keys (kv_lens[b] of sequence
 * b when kv_lens is not NULL, each in 0..kv_len).  With E the smallest
 * integer in -100..100 for which the block's largest |key| is at most
 * 127 * 2^(E-7), the upper bound of a channel is ceil(max 2^(7-E)) 2^(E-7)
 * and the lower one floor(min 2^(7-E)) 2^(E-7).  Layouts as in kb_attn_append;
 * boxes of blocks beyond are left as they were.  Keys are finite: infinities
 * saturate, and the bounds of a block with a NaN are unspecified.
 */
kb_status kb_attn_block_boxes(const void* k_cache, void* boxes, int B, int Hkv, int kv_len,
                              const int* kv_lens, int kv_cap, const int* block_table, int pages_per_seq,
                              int page_size, int num_pages, void* stream);

/* Most blocks a row can choose. */
#define KB_MAX_SELECT 128

/*
 * Choose the key blocks that each query row attends to (one list per row and
 * KV head, shared by its four query heads).
 *   q      : [B, Hq, L, 128] bf16 contiguous, turned; row i at position start
 *            + i, or starts[b] + i for i < lens[b] (as in kb_attn_append)
 *   boxes  : block_table == NULL: [B, Hkv, n_blocks, 2, 128], else
 *            [num_pages, Hkv, page_size/128, 2, 128]
 *   blocks : int32 [B, Hkv, L, n_select] (output): ascending block indices,
 *            -1 behind the last; rows from lens[b] on are left as they were
 * A row at position p has the blocks 0 .. p/128.  The first keep_first and the
 * last keep_last >= 1 of them (the last holds the row's own key) are always
 * taken, the others by score until n_select are taken, ties to the lowest
 * block.  Score: t_h = rint(q_h 2^(15-E)) of the group's four heads with their
 * common E (as for a box), u = sum_h t_h, n = rint(u 2^(7-E')) with E' that of
 * u, score = sum_d max(n_d upper_d, n_d lower_d).  Every step is exact, so the
 * choice does not depend on the batch, the split or the kernel.  More than 32
 * blocks by score out of more than 256 are chosen row by row, about six times
 * slower than 32.  The choice is defined for
 * boxes from kb_attn_append and kb_attn_block_boxes; where `boxes` holds
 * anything else (infinities, NaN, memory that was never written) a row's list
 * is some n_select distinct blocks of its own, ascending, the kept ones among
 * them.
 * keep_first + keep_last <= n_select <= KB_MAX_SELECT.  Out-of-range starts or
 * lens are found on the device (that sequence's rows are not written), as are
 * page indices (the row's list is then any list within its blocks); the next
 * kb_attn_check_device_status returns KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_select_blocks(const void* q, const void* boxes, int* blocks, int B, int Hq, int Hkv, int L,
                                int n_select, int keep_first, int keep_last, int start, const int* starts,
                                const int* lens, int n_blocks, const int* block_table, int pages_per_seq,
                                int page_size, int num_pages, void* stream);

/*
 * Block-sparse attention: as the dense entry points, but a row sees only the
 * keys of its listed blocks of 128 (up to its own position).
 *   blocks : device int32 [B, Hkv, L, n_select]: the key blocks of row i of KV
 *            head g's four query heads, -1 for none, in any order (naming one
 *            twice changes nothing; blocks past the row's own hold no visible
 *            key).  An index below -1, or at or above the cache's number of
 *            blocks, is found on the device and reported by the next
 *            kb_attn_check_device_status as KB_ERR_INVALID_ARG.
 * A row's result is the contract's walk over its listed blocks alone, with the
 * contract's segments, so it has the same bits in a chunk of any split and as
 * a new token, and equals the dense entry points' bits when its list holds
 * every block.  A row that lists nothing is zero (log-sum-exp -inf), whatever
 * its q holds.  In a chunk or a whole sequence V of the cache's visible rows must
 * be finite: 32 neighbouring positions are computed together, and V of a block
 * that only a neighbour listed is multiplied by weights of exactly zero.
 *
 * kb_attn_sparse_chunk: rows at start..start+L-1 of every sequence, or (starts
 * != NULL) at starts[b].., lens[b] of them (L when lens is NULL), against a
 * contiguous cache [B, Hkv, kv_cap, 128] or (block_table != NULL) pools
 * [num_pages, Hkv, page_size, 128], as kb_attn_chunk, _paged and _varlen.
 * kb_attn_sparse_prefill_lse: a whole sequence with lse [B, Hq, S] fp32, as
 * kb_attn_prefill_lse.
 * Both need a device workspace (256-byte aligned, caller-owned, contents
 * scratch) of kb_attn_sparse_workspace_bytes(B, Hkv, L, n_select, kv_cap)
 * bytes, kv_cap being the cache's positions per sequence (pages_per_seq *
 * page_size of a paged one); calls that can overlap on the GPU need one each.
 * kb_attn_sparse_decode: one token per sequence at position ctx_len - 1, or
 * (ctx_lens != NULL, device int32 [B]) at ctx_lens[b] - 1; no workspace.
 */
size_t kb_attn_sparse_workspace_bytes(int B, int Hkv, int L, int n_select, int kv_cap);
kb_status kb_attn_sparse_chunk(const void* q, const void* k, const void* v, void* o, const int* blocks,
                               int n_select, int B, int Hq, int Hkv, int L, int start, const int* starts,
                               const int* lens, int kv_cap, const int* block_table, int pages_per_seq,
                               int page_size, int num_pages, void* workspace, size_t workspace_bytes,
                               void* stream);
kb_status kb_attn_sparse_prefill_lse(const void* q, const void* k, const void* v, void* o, float* lse,
                                     const int* blocks, int n_select, int B, int Hq, int Hkv, int S,
                                     void* workspace, size_t workspace_bytes, void* stream);
kb_status kb_attn_sparse_decode(const void* q, const void* k, const void* v, void* o, const int* blocks,
                                int n_select, int B, int Hq, int Hkv, int ctx_len, const int* ctx_lens,
                                int kv_cap, const int* block_table, int pages_per_seq, int page_size,
                                int num_pages, void* stream);

/*
 * Backward of kb_attn_sparse_prefill_lse: as kb_attn_backward, over the listed
 * keys (the lists themselves take no gradient).  o and lse from the forward
 * with the same q, k, v and blocks; delta [B, Hq, S] fp32 is an output.  A row
 * that lists nothing has dq = 0 and no part in dk and dv, whatever its q and
 * dout hold; a block that no row lists has dk = dv = 0.  K and V are finite.
 * Every sum has one order: repeated calls give identical bits, and a
 * sequence's gradients do not depend on the batch or on n_select.  workspace:
 * 256-byte aligned scratch of kb_attn_sparse_backward_workspace_bytes(B, Hkv,
 * S, n_select).  Per KV head of a sequence that is S^2 / 1024 bytes of row masks
 * and, from S = 4065 on, 256 KB for every block with 4065 positions or more from
 * its first on: at S = 131072, B = 1 and 8 KV heads 0.13 GB and 2.1 GB.
 */
size_t kb_attn_sparse_backward_workspace_bytes(int B, int Hkv, int S, int n_select);
kb_status kb_attn_sparse_backward(const void* q, const void* k, const void* v, const void* o, const void* dout,
                                  const float* lse, float* delta, const int* blocks, int n_select, void* dq,
                                  void* dk, void* dv, int B, int Hq, int Hkv, int S, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Rotation by positions of several axes (time, height and width of a patch; or
 * one axis: a position per token, as a cache needs whose rows are no longer
 * the positions).  As kb_attn_rope, with plane i of row (b, l) turned by
 * p * inv_freq[i], p = positions[plane_axes[i]][b][l].
 *   positions  : device int32 [n_axes, B, L], 1 <= n_axes <= 4
 *   plane_axes : host array of rot_dim/2 axis numbers below n_axes
 * out may be x itself when x is contiguous, and must not overlap it otherwise.
 * A position outside 0 .. n_pos-1 is found on the device: that row is not
 * written, others may not be, and the next kb_attn_check_device_status returns
 * KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_rope_axes(const void* x, const long long* strides, void* out, const float* table, int n_pos,
                            int rot_dim, int interleaved, int inverse, const int* positions, int n_axes,
                            const unsigned char* plane_axes, int B, int H, int L, void* stream);

/*
 * A KV cache held in 8 bits: e4m3 bytes laid out as the bf16 caches, [B, Hkv,
 * kv_cap, 128] or pools [num_pages, Hkv, page_size, 128] (16-byte aligned), and
 * for each block of 128 rows an exponent, int8 [B, Hkv, ceil(kv_cap/128)] or
 * [num_pages, Hkv, page_size/128], of K and V each.  A byte stands for its
 * e4m3 value times 2^E, which bf16 holds exactly.
 * How values get there: E is the smallest integer in -100..100 for which the
 * block's largest magnitude is at most 448 * 2^E; a value is rounded to four
 * significant bits (ties to even), and to zero (of its sign) where the rounded
 * magnitude lies below 2^(E-6); beyond 448 * 2^100 values saturate.  A value
 * that is not finite makes E 127 and all bytes of the block's keys so far 0x7F:
 * a block with exponent 127 reads as NaN throughout, until its first row is
 * written anew.  Exponents below -100 or in 101..126 are read as the nearer of
 * -100 and 100.
 *
 * kb_attn_append_8bit: as kb_attn_append (without boxes).  Keys are rounded
 * from the fp32 rotation to bytes at once.  Where later keys enlarge a block's
 * E, its earlier bytes are brought to it; a block has the same bytes and E for
 * any split of its keys into appends.  Keys overwritten inside a block leave
 * their E, until the block's first row is written anew.
 *
 * kb_attn_cache_values: out [planes, rows, 128] bf16 = what a whole cache or
 * pool (planes = B * Hkv or num_pages * Hkv, rows = kv_cap or page_size)
 * stands for.  Rows that were never written give whatever their bytes say.
 *
 * kb_attn_chunk_8bit, kb_attn_decode_8bit: rows at start .. start+L-1 of every
 * sequence, or (starts and lens != NULL, device int32 [B]) lens[b] rows at
 * starts[b]..; one token at ctx_len - 1, or (ctx_lens != NULL) at ctx_lens[b] -
 * 1.  Contiguous caches, or pools where block_table != NULL.  The result has
 * the bits of kb_attn_chunk, _paged, _varlen and kb_attn_decode on a bf16 cache
 * that holds the same values, so a row has the same bits in any split over the
 * same cache; a later append that enlarges a block's E can change its smallest
 * values (those below 2^(E-6)) for rows computed after it.
 * workspace: device scratch (256-byte aligned, caller-owned) of
 * kb_attn_chunk_8bit_workspace_bytes(B, Hkv, L, rows) bytes (L = 1 for a
 * decode), rows being start + L, or the cache's positions per sequence when
 * starts or ctx_lens is given; calls that can overlap on the GPU need one each.
 * L <= 32 reads the bytes; several CTAs share the keys of a KV head where the
 * batch leaves SMs idle: through a workspace where its size is not 0 (with NULL
 * it runs without, slower, with the same bits), else through shared memory.
 * From 304 (batch, KV head) pairs on, and where it would pass 1 GB, the size is
 * 0 and a CTA has a KV head's keys to itself.  A longer chunk needs its workspace: it reads the bytes as
 * well where few rows see many keys, else it is computed from the visible
 * values in bf16, in the workspace; the bits are the same.  Its size is at least
 * that of two bf16 caches of `rows` positions (512 bytes each for B * Hkv *
 * rows of them, twice what the 8-bit caches take), whichever way is taken.
 */
kb_status kb_attn_append_8bit(const void* q, const void* k, const void* v, const long long* strides, void* q_out,
                              void* k_cache, void* v_cache, signed char* k_exp, signed char* v_exp,
                              const float* table, int n_pos, int rot_dim, int interleaved, int B, int Hq, int Hkv,
                              int L, int start, const int* starts, const int* lens, int kv_cap,
                              const int* block_table, int pages_per_seq, int page_size, int num_pages,
                              void* stream);
kb_status kb_attn_cache_values(const void* cache, const signed char* exps, void* out, long long planes, int rows,
                               void* stream);
size_t kb_attn_chunk_8bit_workspace_bytes(int B, int Hkv, int L, int rows);
kb_status kb_attn_chunk_8bit(const void* q, const void* k, const void* v, const signed char* k_exp,
                             const signed char* v_exp, void* o, int B, int Hq, int Hkv, int L, int start,
                             const int* starts, const int* lens, int kv_cap, const int* block_table,
                             int pages_per_seq, int page_size, int num_pages, void* workspace,
                             size_t workspace_bytes, void* stream);
kb_status kb_attn_decode_8bit(const void* q, const void* k, const void* v, const signed char* k_exp,
                              const signed char* v_exp, void* o, int B, int Hq, int Hkv, int ctx_len,
                              const int* ctx_lens, int kv_cap, const int* block_table, int pages_per_seq,
                              int page_size, int num_pages, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * kb_attn_chunk (starts and lens NULL) or kb_attn_chunk_varlen, contiguous or
 * paged, plus each row's log-sum-exp as kb_attn_prefill_lse gives it: lse
 * [B, Hq, L] fp32, rows from lens[b] on left as they were.  o has the same bits
 * as without; L = 1 is a decode.
 */
kb_status kb_attn_chunk_lse(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                            int Hkv, int L, int start, const int* starts, const int* lens, int kv_cap,
                            const int* block_table, int pages_per_seq, int page_size, int num_pages, void* stream);

/*
 * Add the attention weight that each cached key gets from a call's rows:
 *   weights[b, g, j] += sum over rows i with j <= p_i, and heads h of group g,
 *                       of exp(q_i . k_j / sqrt(128) - lse[b, h, i])
 * with p_i = start + i, or starts[b] + i for i < lens[b] (both device int32
 * [B], or both NULL).
 *   q       : [B, Hq, L, 128] bf16, k: a contiguous cache or pools, as in
 *             kb_attn_chunk_varlen; lse: [B, Hq, L] fp32 from kb_attn_chunk_lse
 *             or kb_attn_prefill_lse of the same rows
 *   weights : [B, Hkv, kv_cap] fp32 (pages_per_seq * page_size of a paged
 *             cache), by position whatever the pages; entries of keys that no
 *             row sees are left as they were
 * A row whose lse is -inf (it saw nothing) or +inf adds nothing.  Every sum has
 * one order that depends on the call's sizes and lengths alone: repeated calls
 * give identical bits.  Out-of-range starts, lens or page indices are found on
 * the device (the sequence's, or that key block's, weights stay) and reported
 * by the next kb_attn_check_device_status as KB_ERR_INVALID_ARG.
 */
kb_status kb_attn_key_weights(const void* q, const void* k, const float* lse, float* weights, int B, int Hq,
                              int Hkv, int L, int start, const int* starts, const int* lens, int kv_cap,
                              const int* block_table, int pages_per_seq, int page_size, int num_pages,
                              void* stream);

/*
 * Cut each sequence's cache to at most `keep` keys per KV head.  Of the n =
 * lens[b] keys (device int32 [B], 0..capacity) of every KV head the first
 * keep_first and the last keep_last stay, and of the others those of the
 * largest weights until `keep` are kept, ties to the lowest row; a NaN counts
 * as larger than any number.  The kept rows of K and V move to rows 0 ..
 * min(n, keep)-1 in their old order, in place; rows behind are left as they
 * were.  A sequence of at most `keep` keys stays as it is.
 *   k, v        : bf16 contiguous caches [B, Hkv, kv_cap, 128] or pools, in
 *                 which no two sequences share a page; not the same buffer
 *   weights     : [B, Hkv, kv_cap] fp32 (positions per sequence of a paged
 *                 cache) as kb_attn_key_weights adds them
 *   weights_out : the same shape: the kept keys' weights, zero behind; may be
 *                 weights itself, and must not overlap it otherwise
 *   kept        : int32 [B, Hkv, keep] (output): the old rows of the kept keys,
 *                 ascending, -1 behind the last
 * keep_first + keep_last <= keep <= capacity.  New keys go to row min(n, keep)
 * on; their positions are no longer their rows (kb_attn_rope_axes).  Boxes of
 * the cache's blocks must be made anew (kb_attn_block_boxes).  An out-of-range
 * lens or page index is found on the device (nothing of that sequence moves)
 * and reported by the next kb_attn_check_device_status as KB_ERR_INVALID_ARG.
 * After KB_ERR_TIMEOUT (a wait between the move's CTAs gave up) some rows have
 * moved and others have not: the caches' contents are undefined.
 */
kb_status kb_attn_evict(void* k, void* v, const float* weights, float* weights_out, int* kept, int B, int Hkv,
                        const int* lens, int keep, int keep_first, int keep_last, int kv_cap,
                        const int* block_table, int pages_per_seq, int page_size, int num_pages, void* stream);

/*
 * Prefill/chunk with an explicit kernel shape, for tests of the contract:
 * q_tiles_per_cta = 3 runs the tile kernel (one 128-row query tile per CTA,
 * one CTA per SM, three score buffers, so Q K^T of later key tiles overlaps
 * the softmax of the current one), launched persistent (CTAs walk balanced
 * pairs of query tiles, or single tiles longest first dealt to the CTAs
 * back and forth) or one CTA per tile as the sizes suit; 4 is 3 with the
 * persistent launch on pairs forced, 5 with the back-and-forth deal forced;
 * 0 runs the packed kernel (the 4 heads of a
 * GQA group times the chunk's rows in one MMA tile; L <= 32).  Other values
 * return KB_ERR_INVALID_ARG.  kb_attn_chunk, kb_attn_prefill and
 * kb_attn_decode pick packed for L <= 32 and 3 otherwise.  Every shape gives
 * the same bits.
 */
kb_status kb_attn_chunk_cta_shape(const void* q, const void* k, const void* v, void* o,
                                  int B, int Hq, int Hkv, int L, int start, int kv_cap,
                                  int q_tiles_per_cta, void* stream);

/* The cudaError_t code (as int) and its description for the most recent
 * KB_ERR_CUDA returned on the calling host thread; 0 / "no error" if none. */
int kb_attn_last_cuda_error(void);
const char* kb_attn_last_cuda_error_string(void);

/* Static description of a status code (never NULL). */
const char* kb_status_string(kb_status s);

/* Version of the numerical contract; outputs are bit-identical across builds
 * with the same contract version on the same GPU architecture. */
int kb_contract_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KB_ATTN_H */

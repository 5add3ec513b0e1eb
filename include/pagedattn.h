/*
 * pagedattn.h -- C ABI of the GB300 (sm_103a) paged KV-cache attention library
 * (libpagedattn.so).
 *
 * The library implements the composition a model layer performs on its KV
 * cache: a slot-mapped write of each new token's K and V into a pool of
 * 16-token pages, then grouped-query causal softmax attention that reads the
 * pool back through a per-request block table, for full prefill, suffix
 * (chunked) prefill and single-query decode.
 *
 * Sources (web pages; cited by title and section):
 *   [C] "test(rocm): ReshapeAndCache->PagedAttention composition at real dims"
 *       -- What changed; maintainer review and rework (slot mapping derived
 *       from the block table, anti-vacuity guard).
 *   [R] "fix(rocm): stabilize direct paged CK attention for bitwise R/R"
 *       -- intro and Changes (fixed arithmetic schedule, real maximum query
 *       length, no implicit FMA contraction, tail-page sanitising, 64-bit
 *       addressing, one query per decode row, graph-cache identity including
 *       the KV scheduling bound); Additional checks (bitwise matrix).
 *
 * Conventions shared by every entry point:
 *   - All device buffers are owned by the caller.  The library never
 *     allocates device memory, never synchronises the stream (except
 *     pa_check_errors) and never reads device memory on the host, so calls
 *     are asynchronous on `stream` and can be captured in a CUDA graph.
 *   - Element types: q, key, value, caches and out are BF16 (passed as
 *     void*); slot_mapping is int64; block tables, lengths and
 *     query_start_loc are int32; lse is fp32.
 *   - Strides are in ELEMENTS; the head dimension is always contiguous.
 *   - Arguments are validated on the host before anything is launched; a
 *     failing check returns a status and launches nothing.  There is no
 *     fallback path: an unsupported shape is an error.
 *   - Device-side metadata errors (a block id outside [0, num_blocks), a slot
 *     past the pool, seq_len < query length, a length above its bound, a
 *     query_start_loc that decreases) never fault: the affected rows are
 *     written as NaN (attention) or skipped (cache write), other rows are
 *     untouched, and the first error is latched in a device flag read by
 *     pa_check_errors.  A request whose query range is inverted
 *     (query_start_loc[b+1] < query_start_loc[b]) owns no rows; its
 *     neighbours are checked against the bounds with the ranges they read.
 *   - `stream` is a cudaStream_t (0 = legacy default stream).
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *pa_stream_t; /* same type as cudaStream_t */

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, negative size, bad stride */
    PA_ERR_UNSUPPORTED = 2,  /* shape outside the supported set (see below) */
    PA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required */
    PA_ERR_BAD_METADATA = 4, /* device-side metadata error (pa_check_errors) */
    PA_ERR_TIMEOUT = 5,      /* an in-kernel wait ran past its limit */
    PA_ERR_CUDA = 6          /* a CUDA runtime call failed */
} pa_status;

/*
 * One paged KV cache: a K view and a V view with one shared set of strides.
 * Element (block, token-in-block, kv-head, d) of K is at
 *   k + block*block_stride + token*token_stride + head*head_stride + d.
 * The pages' pools map onto it as follows ([R] Additional checks names the
 * "separate", "interleaved" and ">2 GB" layouts):
 *   separate    : K and V are two [num_blocks, 16, Hkv, Dh] tensors;
 *   interleaved : one [num_blocks, 2, 16, Hkv, Dh] tensor, K = [:,0], V = [:,1]
 *                 (block_stride = 2*16*Hkv*Dh).
 * Offsets are computed in 64 bits, so a view may exceed 2**31 elements.
 * Requirements: block_size == 16; head_dim in {128, 256, 512}; k and v
 * 16-byte aligned; every stride a multiple of 8 elements (16 bytes).
 * kv_tile selects the KV tile of the attention's fixed arithmetic ("fix(rocm):
 * stabilize direct paged CK attention for bitwise R/R", Changes: fixed tile
 * 128, tile 64 also supported; Additional checks: each tile passes the bitwise
 * matrix on its own).  0 means 128 at head dims 128 and 256 and 64 at 512;
 * head dim 128 also takes 64.  Results are bitwise reproducible within one
 * tile (prefill, suffix and decode agree); the two tiles round differently.
 * Another value returns PA_ERR_INVALID_ARG, a tile the head dim lacks
 * PA_ERR_UNSUPPORTED.  The cache write and the gather ignore it.
 */
typedef struct {
    void *k;
    void *v;
    int64_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t kv_tile;  /* attention KV tile: 0 = the head dim's default (see below) */
    int64_t block_stride;
    int64_t token_stride;
    int64_t head_stride;
} pa_kv_cache;

/*
 * Sets kernel attributes (dynamic shared memory) for the current device.
 * Called implicitly by the first launch on a device; call it explicitly
 * before capturing a CUDA graph ([R] Changes: warm before graph capture).
 */
PA_API pa_status pa_init(void);

/*
 * ReshapeAndCache ([C] What changed and review rework).  For every token i
 * in [0, num_tokens) with slot = slot_mapping[i] >= 0, copies the Dh BF16
 * values of each KV head h from key[i][h][:] and value[i][h][:] into block
 * slot/16, offset slot%16, head h of the K and V views.  A negative slot
 * marks a padding token and is skipped.  A slot >= num_blocks*16 is not
 * written and latches PA_ERR_BAD_METADATA with first_bad_index = i.
 *   key, value        : [num_tokens, Hkv, Dh] BF16, token stride
 *                       key_tok_stride / value_tok_stride (elements, >= Hkv*Dh,
 *                       multiple of 8), heads contiguous; 16-byte aligned.
 *   slot_mapping      : [num_tokens] int64 on the device.
 *   cache             : host struct describing the device pool (read only).
 * Duplicate non-negative slots are undefined (the pages' mapping never makes
 * them).  num_tokens == 0 launches nothing.
 */
PA_API pa_status pa_reshape_and_cache(const void *key, int64_t key_tok_stride, const void *value,
                               int64_t value_tok_stride, int64_t num_tokens,
                               const pa_kv_cache *cache, const int64_t *slot_mapping,
                               pa_stream_t stream);

/*
 * Bytes of scratch that pa_paged_attention needs for these bounds (split-KV
 * partial states and arrival counters).  The same bounds must be passed to
 * pa_paged_attention.  Returns 0 for invalid arguments.
 */
PA_API size_t pa_paged_attention_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim,
                                         int32_t max_query_len, int32_t max_seq_len);

/*
 * PagedAttention ([C] What changed; [R] Changes and Additional checks).
 * For request b (0 <= b < num_seqs) with q_b = query_start_loc[b+1] -
 * query_start_loc[b] new tokens and L_b = seq_lens[b] cached tokens (the new
 * tokens included, already written by pa_reshape_and_cache), query i of the
 * request sits at position p = L_b - q_b + i and attends causally to keys
 * 0..p.  Query head h uses KV head h / (Hq/Hkv).  Key j of request b lives
 * in block block_tables[b*max_blocks_per_seq + j/16] at offset j%16; table
 * columns at or past ceil(L_b/16) are never read.
 *   out[t][h][:] = softmax_j(scale * q[t][h].K_j) . V_j   (BF16, RNE)
 *   lse[t][h]    = ln(sum_j exp(scale * q[t][h].K_j))     (fp32, may be NULL)
 * Decode is query_start_loc = {0, 1, ..., num_seqs} ([R] Changes: one query
 * per row of metadata).
 *
 *   q                 : [num_q_tokens, Hq, Dh] BF16, token stride q_tok_stride
 *                       (elements, >= Hq*Dh, multiple of 8), heads contiguous.
 *   out               : [num_q_tokens, Hq, Dh] BF16, contiguous.  Rows of
 *                       tokens owned by no request are left untouched.
 *   lse               : [num_q_tokens, Hq] fp32, contiguous, or NULL.
 *                       out and lse may be device memory or page-locked host
 *                       memory mapped into the device's address space (the
 *                       kernels write them with plain stores).
 *   block_tables      : [num_seqs, max_blocks_per_seq] int32.
 *   seq_lens          : [num_seqs] int32.  query_start_loc: [num_seqs+1] int32,
 *                       non-decreasing, last entry <= num_q_tokens.
 *   max_query_len, max_seq_len : host-side upper bounds of q_b and L_b.  They
 *                       size the grid and the workspace only; any valid bound
 *                       gives bitwise-identical results ([R] Changes: real
 *                       maximum query length; KV scheduling bound in the graph
 *                       identity).  A request exceeding them latches
 *                       PA_ERR_BAD_METADATA.
 *   scale             : softmax scale, finite and > 0 (typically 1/sqrt(Dh)).
 *   workspace         : device scratch of at least
 *                       pa_paged_attention_workspace_size(...) bytes, 256-byte
 *                       aligned, zero-filled before its first use; the library
 *                       leaves it ready for the next call (after a call that
 *                       reports PA_ERR_TIMEOUT, zero-fill it again).  One
 *                       workspace must not be used by two calls that may run
 *                       concurrently.
 * Supported: head_dim in {128, 256, 512}; Hq % Hkv == 0; Hq/Hkv <= 128.
 *
 * Arithmetic is fixed ([R] intro: one schedule for strict agreement): every
 * (token, head) row is computed by the same sequence of operations whatever
 * the batch, the other requests, the query length or the bounds, so a
 * token's output and lse are bitwise identical in full prefill, suffix
 * prefill and decode.
 */
PA_API pa_status pa_paged_attention(const void *q, int64_t num_q_tokens, int64_t q_tok_stride,
                             int32_t num_q_heads, const pa_kv_cache *cache,
                             const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *seq_lens, const int32_t *query_start_loc,
                             int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len,
                             float scale, void *out, float *lse, void *workspace,
                             size_t workspace_bytes, pa_stream_t stream);

/*
 * Copies `bytes` bytes from `src` to device memory `dst` with a kernel on
 * `stream`, for step inputs that arrive in host memory.  `src` is page-locked
 * host memory mapped into the device's address space (cudaHostAlloc, or
 * cudaHostRegister with cudaHostRegisterMapped) or device memory; the kernel
 * reads it directly (on a coherent CPU-GPU link, one round trip instead of a
 * copy-engine transfer).
 *   - The paper (the source pages) has no counterpart to this entry point.
 *   - Launched with programmatic stream serialization: it waits for the
 *     preceding grid of the stream to complete before it writes dst (and,
 *     unless src_ready, before it reads src), and lets the next kernel of the
 *     stream (for instance the cache write of pa_reshape_and_paged_attention,
 *     which waits for it in turn) be scheduled meanwhile.
 *   - src_ready != 0 is the caller's statement that no kernel in flight on
 *     the GPU writes src (for instance host memory filled by the host before
 *     the call): the kernel then reads src at once, while the preceding grid
 *     may still run.
 *   - dst and src 16-byte aligned, not overlapping; otherwise
 *     PA_ERR_INVALID_ARG and nothing is launched.  bytes == 0 launches nothing.
 * The attention calls may likewise be given `out` and `lse` in page-locked,
 * mapped host memory: their kernels write the results there directly.
 */
PA_API pa_status pa_copy_to_device(void *dst, const void *src, size_t bytes, int32_t src_ready,
                                   pa_stream_t stream);

/*
 * PagedAttention for callers that cannot allocate device memory.
 *
 * Some callers cannot call cudaMalloc at all: code that runs while a CUDA
 * graph is being captured (allocation is not a capturable operation), or an
 * engine whose device memory is entirely reserved by its own pool allocator
 * and that therefore has no buffer to hand over as the workspace that
 * pa_paged_attention wants.  This variant takes the same arguments minus the
 * workspace and uses instead a scratch array built into the library: a
 * file-scope device array of PA_NOALLOC_SCRATCH_BYTES bytes that every GPU
 * which loads the library holds until the process exits.
 *   - The paper (the source pages) has no counterpart to this entry point.
 *   - It allocates nothing: no cudaMalloc, cudaFree or allocating library
 *     routine.  It clears the scratch's arrival counters with
 *     cudaMemsetAsync on `stream`, then launches the same kernel as
 *     pa_paged_attention with the scratch as its workspace.
 *   - The first call on a device looks up the scratch array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - If the bounds need more scratch than PA_NOALLOC_SCRATCH_BYTES (see
 *     pa_paged_attention_workspace_size), it returns PA_ERR_WORKSPACE and
 *     launches nothing.
 *   - Every call on a device shares the one array: calls that may overlap on
 *     the GPU (different streams without ordering) race on it.
 */
#define PA_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
PA_API pa_status pa_paged_attention_noalloc(const void *q, int64_t num_q_tokens, int64_t q_tok_stride,
                                            int32_t num_q_heads, const pa_kv_cache *cache,
                                            const int32_t *block_tables, int32_t max_blocks_per_seq,
                                            const int32_t *seq_lens, const int32_t *query_start_loc,
                                            int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len,
                                            float scale, void *out, float *lse, pa_stream_t stream);

/*
 * The whole composition of [C] What changed in one call: ReshapeAndCache of
 * the num_new_tokens new tokens, then PagedAttention over the updated pool.
 * The arguments and results are those of pa_reshape_and_cache followed by
 * pa_paged_attention on `stream` (same meaning, layout and ownership); the
 * outputs are bitwise identical to that pair of calls.
 *   - Both argument sets are validated before anything is launched.
 *   - What it adds: the attention grid is scheduled while the cache write
 *     still runs.  It reads the metadata, the block tables and q and sets up
 *     its pipeline at once; only its K/V copies wait until the cache write
 *     has completed and its stores are visible.
 *   - For that reason q, block_tables, seq_lens and query_start_loc must not
 *     share bytes with the pool, and out, lse and the workspace must share
 *     none with the pool, key, value or slot_mapping.  An overlap returns
 *     PA_ERR_INVALID_ARG and launches nothing.
 *   - num_new_tokens == 0 launches only the attention, which then waits for
 *     whatever precedes it on the stream like pa_paged_attention.  An empty
 *     attention batch launches only the cache write.
 *   - Head dim 512 always waits at entry (no early reads).
 */
PA_API pa_status pa_reshape_and_paged_attention(
    const void *key, int64_t key_tok_stride, const void *value, int64_t value_tok_stride,
    int64_t num_new_tokens, const int64_t *slot_mapping, const void *q, int64_t num_q_tokens,
    int64_t q_tok_stride, int32_t num_q_heads, const pa_kv_cache *cache, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
    int32_t max_query_len, int32_t max_seq_len, float scale, void *out, float *lse, void *workspace,
    size_t workspace_bytes, pa_stream_t stream);

/*
 * Compact active-block gather of one KV head ("ROCm: harden compact
 * peer-local KV prefill for Gemma-4", Scope and Required hardening: the
 * block-table-selected pages of one K/V head packed for transfer, with
 * shuffled and sparse blocks, page boundaries, invalid metadata and byte
 * budgets).  Request b with L_b = seq_lens[b] tokens selects the
 * n_b = ceil(L_b / 16) pages block_tables[b][0..n_b-1].  With
 * off_b = n_0 + ... + n_{b-1} and total = off_{num_seqs}:
 *   packed_k[off_b + p][t][:] = K[block_tables[b][p]][t][kv_head][:]
 *   packed_v[off_b + p][t][:] = V[block_tables[b][p]][t][kv_head][:]
 *   compact_tables[b][p]      = off_b + p for p < n_b, -1 for p >= n_b
 *   compact_offsets[b]        = off_b, compact_offsets[num_seqs] = total
 * Whole pages are copied (a partial last page carries its tail rows as they
 * are in the pool).  The packed buffers form a pool of their own with one KV
 * head ({k, v, capacity_pages, 16, 1, Dh, 0, 16*Dh, Dh, Dh}); attention over
 * it with compact_tables and the group's query heads gives the same bits as
 * attention over the full pool.
 *   cache             : the pool (read only).  kv_head in [0, Hkv).
 *   block_tables      : [num_seqs, max_blocks_per_seq] int32, seq_lens
 *                       [num_seqs] int32, both on the device.
 *   packed_k, packed_v: [capacity_pages, 16, Dh] BF16 each, contiguous,
 *                       16-byte aligned, caller-owned (may be NULL when
 *                       capacity_pages == 0).
 *   compact_tables    : [num_seqs, max_blocks_per_seq] int32 (written).
 *   compact_offsets   : [num_seqs + 1] int32 (written).
 * Errors latched on the device and read with pa_check_errors:
 *   - a length outside [0, max_blocks_per_seq*16]: that request gets no
 *     pages; PA_ERR_BAD_METADATA, index = the request;
 *   - a block id outside [0, num_blocks): that packed page is NaN;
 *     PA_ERR_BAD_METADATA, index = the request;
 *   - total > capacity_pages: only compact_offsets is written (so the caller
 *     learns the size it needs); PA_ERR_WORKSPACE, index = total.
 * Host errors: PA_ERR_INVALID_ARG (bad head, sizes or pointers, or an
 * output that shares bytes with the pool, block_tables, seq_lens or another
 * output),
 * PA_ERR_UNSUPPORTED (num_seqs > 512 or num_seqs*max_blocks_per_seq >
 * INT32_MAX).  num_seqs == 0 launches nothing.  The launch waits for the
 * work before it on the stream (it may be launched early with programmatic
 * stream serialization and waits in the kernel).
 */
PA_API pa_status pa_gather_kv_head(const pa_kv_cache *cache, int32_t kv_head, const int32_t *block_tables,
                                   int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs,
                                   void *packed_k, void *packed_v, int64_t capacity_pages,
                                   int32_t *compact_tables, int32_t *compact_offsets, pa_stream_t stream);

/*
 * Metadata of one serving step, built on the device: new pages from a free
 * list, block tables, slots and positions of the new tokens, lengths and
 * query starts -- the inputs of pa_reshape_and_cache and pa_paged_attention.
 * The paper (the source pages) has no counterpart to this entry point.
 * Request b has c_b = context_lens[b] cached tokens and brings
 * n_b = query_lens[b] new ones.  With have_b = ceil(c_b/16), need_b =
 * ceil((c_b+n_b)/16) - have_b, first_b = need_0 + .. + need_{b-1} and
 * start_b = n_0 + .. + n_{b-1}:
 *   block_tables[b][have_b + j]  = free_pages[cursor + first_b + j], j < need_b
 *   seq_lens[b]                  = c_b + n_b
 *   query_start_loc[b]           = start_b (and [num_seqs] = their sum)
 *   positions[start_b + i]       = c_b + i,                          i < n_b
 *   slot_mapping[start_b + i]    = block_tables[b][pos/16]*16 + pos%16
 *   positions[t] = slot_mapping[t] = -1 for the padding tokens t from the
 *                                  sum of the n_b up to num_tokens
 *   *cursor_out                  = *cursor_in + the sum of the need_b
 *   context_lens, query_lens : [num_seqs] int32.
 *   block_tables   : [num_seqs, max_blocks_per_seq] int32; columns below
 *                    have_b are read, the need_b new ones written, the rest
 *                    left as they are.
 *   free_pages     : [num_free_pages] int32; pages from index *cursor_in on
 *                    are free.  cursor_in NULL means 0.  num_blocks: pages of
 *                    the pool.
 *   slot_mapping   : [num_tokens] int64.  positions: [num_tokens] int32.
 *   seq_lens       : [num_seqs] int32.  query_start_loc: [num_seqs+1] int32.
 *   cursor_out     : [1] int32.
 *   seq_lens may be context_lens and cursor_out may be cursor_in (all inputs
 *   are read before anything is written), so a captured graph of a decode
 *   step advances its own state.  No other output may share bytes with an
 *   input or another output (PA_ERR_INVALID_ARG).
 * Errors latched on the device:
 *   - c_b or n_b negative, or c_b + n_b > max_blocks_per_seq*16: the request
 *     brings no tokens, its seq_lens entry is c_b (0 if c_b itself is out of
 *     range); PA_ERR_BAD_METADATA, index = the request;
 *   - a page id outside [0, num_blocks): the slots in it are -1 (a new one
 *     still enters the table); PA_ERR_BAD_METADATA, index = the request;
 *   - more new pages than free ones (PA_ERR_WORKSPACE, index = the pages
 *     needed), more new tokens than num_tokens, or a cursor outside
 *     [0, num_free_pages] (PA_ERR_BAD_METADATA, index = num_seqs): the step
 *     is empty -- every seq_lens entry is c_b as above, every query start 0,
 *     every token padding, tables and cursor unchanged.
 * num_seqs in [0, 8192] (PA_ERR_UNSUPPORTED above); num_seqs == 0 launches
 * nothing.  num_tokens == 0 is allowed (slot_mapping, positions unused).
 */
PA_API pa_status pa_build_step_metadata(const int32_t *context_lens, const int32_t *query_lens, int32_t num_seqs,
                                        int32_t *block_tables, int32_t max_blocks_per_seq,
                                        const int32_t *free_pages, int32_t num_free_pages,
                                        const int32_t *cursor_in, int32_t *cursor_out, int64_t num_blocks,
                                        int64_t *slot_mapping, int32_t *positions, int64_t num_tokens,
                                        int32_t *seq_lens, int32_t *query_start_loc, pa_stream_t stream);

/*
 * Norm of every query and key head and the rotation by position, in one pass
 * over the new tokens (the step between a layer's projections and its cache
 * write).  The paper (the source pages) has no counterpart to this entry
 * point.  For every token t with p = positions[t] >= 0 and every head row x
 * of q and k:
 *   y = x / sqrt(mean(x_i^2) + eps) * (weight + weight_offset)   (norm), then
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)       (rotation)
 * for the rot_dim/2 pairs (a, b) = (i, i + rot_dim/2), or (2i, 2i+1) with
 * interleaved != 0; cos = cos_sin[p][i], sin = cos_sin[p][rot_dim/2 + i].
 * Elements from rot_dim on are not rotated.  Sums and products are fp32; the
 * result is rounded to BF16 once.  Rows of a token with p < 0 (padding) are
 * left untouched.  A token with p >= max_positions gets NaN rows and latches
 * PA_ERR_BAD_METADATA (index = the token).
 *   q [T, Hq, Dh], k [T, Hkv, Dh] : BF16, token strides in elements (>= the
 *                   row, multiple of 8), heads contiguous, 16-byte aligned
 *                   (slices of a fused projection are fine).
 *   q_out, k_out  : the same shapes, their own token strides.  q_out may be q
 *                   and k_out may be k (same pointer and stride: in place).
 *   q_weight, k_weight : [Dh] BF16, or NULL for no norm of q or k.
 *   weight_offset : added to the weights (1 for weights stored less one).
 *   positions     : [T] int32.  cos_sin: [max_positions, rot_dim] fp32,
 *                   contiguous, 16-byte aligned.
 *   eps           : finite, >= 0.  rot_dim: a multiple of 16 in [16, Dh].
 *                   head_dim 128, 256 or 512 (PA_ERR_UNSUPPORTED otherwise).
 * Outputs may not share bytes with anything else (PA_ERR_INVALID_ARG), but
 * rows of tensors with one token stride may interleave.  T == 0 launches
 * nothing.
 */
PA_API pa_status pa_qk_norm_rope(const void *q, int64_t q_tok_stride, int32_t num_q_heads, const void *k,
                                 int64_t k_tok_stride, int32_t num_kv_heads, int32_t head_dim, int64_t num_tokens,
                                 const int32_t *positions, const float *cos_sin, int64_t max_positions,
                                 int32_t rot_dim, int32_t interleaved, const void *q_weight, const void *k_weight,
                                 float weight_offset, float eps, void *q_out, int64_t q_out_tok_stride, void *k_out,
                                 int64_t k_out_tok_stride, pa_stream_t stream);

/*
 * pa_qk_norm_rope with the cache write of pa_reshape_and_cache in the same
 * pass: the rotated keys and the values go into the pool at slot_mapping, and
 * no k_out is written.  A negative slot skips the token's cache write; a slot
 * past the pool latches PA_ERR_BAD_METADATA (index = the token) and is
 * skipped, as is the cache write of a token with a bad or negative position.
 * Results are bitwise those of pa_qk_norm_rope followed by
 * pa_reshape_and_cache (the slots of a call have to differ).  The pool may not
 * share bytes with the other arguments (PA_ERR_INVALID_ARG).
 */
PA_API pa_status pa_qk_norm_rope_and_cache(
    const void *q, int64_t q_tok_stride, int32_t num_q_heads, const void *k, int64_t k_tok_stride, const void *value,
    int64_t value_tok_stride, int64_t num_tokens, const int32_t *positions, const float *cos_sin,
    int64_t max_positions, int32_t rot_dim, int32_t interleaved, const void *q_weight, const void *k_weight,
    float weight_offset, float eps, void *q_out, int64_t q_out_tok_stride, const pa_kv_cache *cache,
    const int64_t *slot_mapping, pa_stream_t stream);

/*
 * A paged KV cache held in 4 bits.  The paper (the source pages) has no
 * counterpart to it.  Sixteen neighbouring head-dim elements of a token share
 * one scale: an element's value is
 *   code (e2m1: 0, .5, 1, 1.5, 2, 3, 4, 6, with a sign) * scale (e4m3) *
 *   k_scale or v_scale.
 * That value is exact in BF16 (two significant bits times four, times a power
 * of two).  For one page and KV head, K and V each have a contiguous RECORD of
 * 9*head_dim bytes:
 *   K : codes [16 tokens][Dh/2 bytes], then scales [16 tokens][Dh/16];
 *   V : codes [Dh/2][16 tokens],       then scales [Dh/16][16 tokens].
 * A code byte holds elements 2i (low half) and 2i+1 of a token.  The record
 * of (block, head) starts at k + block*block_stride + head*head_stride, in
 * BYTES (v likewise).  Pools map onto it as two [num_blocks, Hkv, 9*Dh] byte
 * tensors or one [num_blocks, 2, Hkv, 9*Dh] one.
 * Requirements: block_size == 16; head_dim in {128, 256, 512}; k and v
 * 16-byte aligned; strides positive multiples of 16 below 2^32, head_stride
 * >= 9*Dh;
 * k_scale and v_scale powers of two in [2^-32, 2^32]; reserved == 0.
 */
typedef struct {
    void *k;
    void *v;
    int64_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t reserved;
    int64_t block_stride;
    int64_t head_stride;
    float k_scale;
    float v_scale;
} pa_quant_cache;

/*
 * pa_reshape_and_cache into a 4-bit pool.  For the 16 elements x of a block,
 * with x' = x / k_scale (or v_scale):
 *   scale = e4m3(max|x'| / 6), saturating at 448; code = e2m1(x' / scale),
 * both to nearest, ties to even, saturating; a zero scale gives zero codes,
 * and a block that holds a NaN or an infinity reads back as NaN.  Arguments,
 * padding (negative slots) and errors as for pa_reshape_and_cache; key and
 * value may not share bytes with the pool (PA_ERR_INVALID_ARG).  The slots of
 * a call have to differ: what two tokens leave in one slot is a mixture.
 */
PA_API pa_status pa_reshape_and_cache_quant(const void *key, int64_t key_tok_stride, const void *value,
                                            int64_t value_tok_stride, int64_t num_tokens,
                                            const pa_quant_cache *cache, const int64_t *slot_mapping,
                                            pa_stream_t stream);

/*
 * Reads the pages that the block tables select back as a BF16 pool: the
 * counterpart of pa_gather_kv_head for a 4-bit cache, for every KV head.
 * Request b selects the n_b = ceil(L_b/16) pages block_tables[b][0..n_b-1];
 * with off_b = n_0 + .. + n_{b-1},
 *   k_out[off_b + p][t][h][:] = the values of K[block_tables[b][p]], token t,
 *                               head h (exact), v_out likewise;
 *   compact_tables[b][p] = off_b + p for p < n_b, -1 beyond;
 *   compact_offsets[b] = off_b, compact_offsets[num_seqs] = the total.
 * k_out and v_out ([capacity_pages, 16, Hkv, Dh] BF16, contiguous) are a pool
 * that the library's BF16 calls take.  Whole pages are converted.
 *   compact_tables : [num_seqs, max_blocks_per_seq] int32.
 * Errors on the device as for pa_gather_kv_head: a bad length selects no
 * pages, a bad block id gives a NaN page, a total above capacity_pages writes
 * only compact_offsets (PA_ERR_WORKSPACE, index = total).  Outputs may not
 * share bytes with the pool, the metadata or each other.  num_seqs <= 8192.
 */
PA_API pa_status pa_dequantize_kv(const pa_quant_cache *cache, const int32_t *block_tables,
                                  int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs, void *k_out,
                                  void *v_out, int64_t capacity_pages, int32_t *compact_tables,
                                  int32_t *compact_offsets, pa_stream_t stream);

/*
 * Bytes of scratch that pa_paged_attention_quant needs for these bounds.
 * max_pages: an upper bound of the pages of all requests together, or 0 for
 * num_seqs * ceil(max_seq_len / 16).  Returns 0 for invalid arguments.
 * Smaller bounds may need more (their calls take another way, see below): a
 * workspace for several calls is as large as the largest of their sizes.
 */
PA_API size_t pa_paged_attention_quant_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                      int32_t head_dim, int32_t max_query_len, int32_t max_seq_len,
                                                      int64_t max_pages);

/*
 * pa_paged_attention over a 4-bit pool: the softmax attention of q over the
 * values that the pool stands for.  Arguments, ownership and errors as for
 * pa_paged_attention; max_pages as in the workspace size.
 *   - Few tokens (max_query_len at most 2 * floor(32 / (Hq/Hkv)), at head dim
 *     512 at most 2 * floor(16 / (Hq/Hkv)): decode steps, drafted tokens; above
 *     1024 requests half of that): kernels that read the codes directly.  They
 *     have a fixed schedule of their own: a row's results are bitwise the same
 *     whatever the batch, the other requests and the bounds (within that
 *     limit).
 *   - More tokens where that is faster, by the bounds alone (num_seqs, the
 *     heads, max_query_len, max_seq_len; pa_last_launch_info tells): the same
 *     kernels, and the same bits.
 *   - More tokens otherwise: the selected pages are read back into the
 *     workspace (as by pa_dequantize_kv), and pa_paged_attention's kernel runs
 *     over them: bitwise its results on the read-back pool.
 *   The two ways round differently: the direct kernels take q (times a power
 *   of two per row) and the probabilities in f16, the BF16 attention takes the
 *   probabilities in BF16.  Sums, maxima and lse are fp32 in both.  The direct
 *   kernels hold for scores (scale * q.k) up to fp32's range, the BF16 attention
 *   for scores below 2^30.
 *   - Hq/Hkv above 32 (16 at head dim 512): no row tile holds a token's heads,
 *     so every call, decode steps too, goes by way of the read-back.
 *   - More than max_pages (> 0) selected pages: PA_ERR_WORKSPACE is latched
 *     (index = the pages) and all rows are NaN.
 *   - A bad block id makes all rows of its request NaN.  Keys past a
 *     request's length never matter, whatever their bytes.
 *   - workspace: at least pa_paged_attention_quant_workspace_size(...) bytes
 *     for the call's bounds, 256-byte aligned; it needs no particular contents,
 *     and calls with different bounds may share it one after another.
 *   - out, lse and the workspace may not share bytes with an input or with one
 *     another (PA_ERR_INVALID_ARG).
 *   - When the direct kernels latch PA_ERR_TIMEOUT, the rows of the requests
 *     that a wait ran out for are NaN or, where one step takes all of a
 *     request's keys, may be left as they were.
 * num_seqs <= 2048, and num_seqs times the pages of max_seq_len at most 2^28.
 */
PA_API pa_status pa_paged_attention_quant(const void *q, int64_t num_q_tokens, int64_t q_tok_stride,
                                          int32_t num_q_heads, const pa_quant_cache *cache,
                                          const int32_t *block_tables, int32_t max_blocks_per_seq,
                                          const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
                                          int32_t max_query_len, int32_t max_seq_len, int64_t max_pages, float scale,
                                          void *out, float *lse, void *workspace, size_t workspace_bytes,
                                          pa_stream_t stream);

/*
 * Pages between requests.  The paper (the source pages) has no counterpart to
 * the calls from here to pa_compact_pages.  They keep the owners of pages in
 * an array shares [num_blocks] int32: shares[p] counts the owners of page p
 * beyond its first, so that it is 0 for a free page and for a page of one
 * request, and pa_build_step_metadata needs to know nothing of it.
 * free_pages is a stack whose entries from the cursor on are free: that call
 * and forks take from the cursor upwards, releases put back below it.
 *   In place: seq_lens may be context_lens, shares_out shares_in, cursor_out
 * cursor_in and tables_out block_tables (the same pointer: all inputs are read
 * before anything is written, or by the thread that writes), so a captured
 * graph advances its own state.  No other output may share bytes with an input
 * or another output (PA_ERR_INVALID_ARG).  With shares_out != shares_in all of
 * shares_out is written.
 *   num_seqs <= 8192, num_forks <= 8192, num_seqs * max_blocks_per_seq <=
 * INT32_MAX (PA_ERR_UNSUPPORTED above).
 */

/*
 * Copies pages within the pools of num_caches layers: for every pair i with
 * src_pages[i] >= 0, page dst_pages[i] of K and of V of each cache becomes
 * page src_pages[i] (all 16 tokens, all heads).  Pairs with a negative source,
 * or with the source as destination, are skipped: lists may be padded.
 *   caches      : host array; sizes and strides of all caches are the same
 *                 (PA_ERR_INVALID_ARG otherwise).  num_caches <= 128.
 *   src_pages, dst_pages : [num_pairs] int32 on the device, outside the pools.
 * A page outside [0, num_blocks) copies nothing and latches
 * PA_ERR_BAD_METADATA (index = the pair).  The pairs of a call are copied in no
 * order: its destinations have to differ from one another and from its sources.
 * num_pairs == 0 or num_caches == 0 launches nothing.
 */
PA_API pa_status pa_copy_pages(const pa_kv_cache *caches, int32_t num_caches, const int32_t *src_pages,
                               const int32_t *dst_pages, int64_t num_pairs, pa_stream_t stream);

/* pa_copy_pages within 4-bit pools: whole records, codes and scales.  (The
 * caches' k_scale and v_scale may differ: each page stays in its pool.) */
PA_API pa_status pa_copy_pages_quant(const pa_quant_cache *caches, int32_t num_caches, const int32_t *src_pages,
                                     const int32_t *dst_pages, int64_t num_pairs, pa_stream_t stream);

/*
 * Forks requests: fork i gives the empty request c = children[i] the first
 * l = fork_lens[i] tokens of request p = parents[i] (all of them where
 * fork_lens is NULL).
 *   block_tables[c][j] = block_tables[p][j] and one owner more for that page,
 *                        for the l/16 whole pages;
 *   where l % 16 != 0, block_tables[c][l/16] = the next free page, and
 *   copy_src[i], copy_dst[i] = the parent's page and the new one: a list for
 *                        pa_copy_pages, once for every pool.  Otherwise both -1.
 *   seq_lens[c] = l; seq_lens[b] = context_lens[b] for all others.
 *   *cursor_out = *cursor_in + the new pages, which go to the forks in order.
 * So a page that tokens are yet to be written to has one owner.
 *   parents, children, fork_lens, copy_src, copy_dst : [num_forks] int32.
 *   context_lens, seq_lens : [num_seqs] int32.  block_tables: [num_seqs,
 *                        max_blocks_per_seq]; other entries are left alone.
 * Errors latched on the device:
 *   - a parent or child outside [0, num_seqs), a child that is not empty or
 *     that an earlier fork of the call names too, l outside [0,
 *     context_lens[p]], a context past its table row: the fork does nothing;
 *     PA_ERR_BAD_METADATA, index = the fork;
 *   - a page outside [0, num_blocks): its entry is copied (or the free page
 *     taken) all the same, but no owner is counted and no copy listed;
 *     PA_ERR_BAD_METADATA, index = the fork;
 *   - more new pages than free ones (PA_ERR_WORKSPACE, index = the pages
 *     needed), a cursor outside [0, num_free_pages] (PA_ERR_BAD_METADATA, index
 *     = num_forks): no fork does anything.
 * num_seqs == 0 launches nothing.
 */
PA_API pa_status pa_fork_requests(const int32_t *parents, const int32_t *children, const int32_t *fork_lens,
                                  int32_t num_forks, const int32_t *context_lens, int32_t num_seqs,
                                  int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *shares_in,
                                  int32_t *shares_out, int64_t num_blocks, const int32_t *free_pages,
                                  int32_t num_free_pages, const int32_t *cursor_in, int32_t *cursor_out,
                                  int32_t *seq_lens, int32_t *copy_src, int32_t *copy_dst, pa_stream_t stream);

/*
 * Releases pages: request b keeps its first keep_lens[b] tokens (0: it has
 * ended; negative: it stays as it is) and gives up the pages past them, in
 * columns ceil(keep/16) .. ceil(context/16)-1 of its table row.  Each loses an
 * owner; one that has none left goes onto the free stack:
 *   free_pages[*cursor_in - n + k] = the k-th of the n freed pages, in the
 *     order (request, column) of the reference that was its last;
 *   *cursor_out = *cursor_in - n;  seq_lens[b] = keep_lens[b] (or
 *     context_lens[b]).
 * The table is left as it is.  Several requests of a call may own a page.
 * Errors latched on the device:
 *   - context_lens[b] outside [0, max_blocks_per_seq*16], or keep_lens[b] >
 *     context_lens[b]: the request stays as it is; PA_ERR_BAD_METADATA, index
 *     = the request;
 *   - tokens that stay end inside a page which other requests own too (at the
 *     call's start): the next token would be written into it; the same (fork
 *     the request instead);
 *   - a page outside [0, num_blocks) is passed over, a page given up more often
 *     than it had owners is freed once; the same;
 *   - more freed pages than *cursor_in (PA_ERR_WORKSPACE, index = the pages), a
 *     cursor outside [0, num_free_pages] or more than 2^30 given up pages
 *     (PA_ERR_BAD_METADATA, index = num_seqs): nothing is released.
 * num_seqs == 0 launches nothing.
 */
PA_API pa_status pa_release_pages(const int32_t *context_lens, const int32_t *keep_lens, int32_t num_seqs,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *shares_in,
                                  int32_t *shares_out, int64_t num_blocks, int32_t *free_pages,
                                  int32_t num_free_pages, const int32_t *cursor_in, int32_t *cursor_out,
                                  int32_t *seq_lens, pa_stream_t stream);

/* Bytes of scratch for pa_compact_pages (any contents); 0 for invalid sizes. */
PA_API size_t pa_compact_pages_workspace_size(int64_t num_blocks);

/*
 * Plans the compaction of a pool: with n pages in use by the requests' tables
 * (context_lens[b] tokens each), the k-th page in use from page n on moves to
 * the k-th unused page below n, so that pages 0 .. n-1 are in use afterwards.
 *   copy_src[k], copy_dst[k] = the k-th move, ascending; -1 from the number of
 *                   moves up to max_moves: a list for pa_copy_pages;
 *   tables_out[b][j] = the new place of block_tables[b][j], for the columns in
 *                   use (others are left alone);
 *   shares_out      = shares_in moved along, 0 from page n on;
 *   free_pages[num_free_pages - num_blocks + p] = p for n <= p < num_blocks,
 *   *cursor_out     = num_free_pages - num_blocks + n;
 *   counts[0], counts[1] = n and the number of moves.
 * Pages that only the free list holds are unused; a page held elsewhere has to
 * be in some table.  num_free_pages >= num_blocks (PA_ERR_INVALID_ARG);
 * num_blocks <= 2^20 (PA_ERR_UNSUPPORTED).
 *   workspace : pa_compact_pages_workspace_size(num_blocks) bytes, 256-byte
 *               aligned, any contents.
 * Errors latched on the device:
 *   - context_lens[b] outside [0, max_blocks_per_seq*16]: none of the row's
 *     pages count, its entries are not written; a page outside [0, num_blocks)
 *     keeps its entry; PA_ERR_BAD_METADATA, index = the request;
 *   - more than max_moves moves: nothing moves (tables_out and shares_out are
 *     the inputs, *cursor_out is *cursor_in, free_pages stays, the lists are
 *     -1); PA_ERR_WORKSPACE, index = the moves.
 */
PA_API pa_status pa_compact_pages(const int32_t *context_lens, int32_t num_seqs, const int32_t *block_tables,
                                  int32_t *tables_out, int32_t max_blocks_per_seq, const int32_t *shares_in,
                                  int32_t *shares_out, int64_t num_blocks, int32_t *free_pages,
                                  int32_t num_free_pages, const int32_t *cursor_in, int32_t *cursor_out,
                                  int32_t *copy_src, int32_t *copy_dst, int32_t max_moves, int32_t *counts,
                                  void *workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * What changes the scores of pa_paged_attention_scored.  All fields 0 (or no
 * struct): plain causal attention.
 */
typedef struct {
    float soft_cap;             /* scores z become soft_cap * tanh(z / soft_cap); 0: no cap,
                                   else within [2^-20, 2^20] */
    int32_t window;             /* a token sees the `window` keys that end at its position; 0: all */
    const float *slopes;        /* [Hq]: slopes[h] * |p - j| is taken off the score of key j for a
                                   token at position p, after the cap; NULL: no bias */
    const int32_t *prefix_lens; /* [num_seqs]: every token of request b sees keys 0 .. prefix_lens[b]-1,
                                   whatever the other rules (at most its length); NULL: no prefix */
    const int32_t *first_keys;  /* [num_q_tokens]: token t sees no key before first_keys[t] (but the
                                   prefix): the start of its document; NULL: 0 */
} pa_score_rules;

/*
 * Bytes of scratch that pa_paged_attention_scored needs for these bounds.
 * Returns 0 for invalid arguments and where none is needed.  Smaller bounds may
 * need more: a workspace for several calls is as large as the largest of their
 * sizes.
 */
PA_API size_t pa_paged_attention_scored_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                       int32_t head_dim, int32_t max_query_len, int32_t max_seq_len);

/*
 * pa_paged_attention with rules for the scores: a cap by tanh, a bias by
 * distance, a sliding window, a prefix that all tokens see (first tokens kept
 * beside a window; a prompt read in both directions), documents packed into one
 * context.  The paper (the source pages) has no counterpart to it.  A token of
 * request b at position p, with L = seq_lens[b], sees key j where
 *   j < L and ((first_keys[t] <= j <= p and p - j < window) or j < prefix_lens[b]).
 *   z_j = scale * q.K_j;  z_j = soft_cap * tanh(z_j / soft_cap);
 *   z_j = z_j - slopes[h] * |p - j|
 *   out = sum_j exp(z_j) V_j / sum_j exp(z_j),  lse = ln(sum_j exp(z_j))
 * over the keys that it sees; a token that sees none gets zeros and lse -inf.
 * Arguments, ownership and errors as for pa_paged_attention; kv_tile is
 * ignored.  Differences:
 *   - Keys that a token does not see never matter to it, whatever their bytes
 *     (NaN included), and the table entry of a page that no token of the request
 *     sees a key of may be anything.  A bad id of another page makes the rows that
 *     see a key of it NaN and latches PA_ERR_BAD_METADATA (index = the request).
 *   - Pages that a window has left behind are needed by this call no more.  The
 *     calls above know nothing of it: pa_release_pages gives up a request's last
 *     pages only, and a fork, a release or a compaction takes every entry up to the
 *     request's length for a page that the request owns.
 *   - Sums, maxima and lse are fp32, the probabilities BF16.  A call's results
 *     are bitwise reproducible; other bounds, or the token in another call, may
 *     round differently (the fixed schedule of pa_paged_attention is not kept).
 *     The cap costs a score about 2^-21 of the cap, above a cap of 55 2^-19 of the score.
 *   - Where a value (V) of a key that rows compute together is infinite or NaN, or so
 *     large that a sum overflows before its division, the rows whose result that makes
 *     not finite are computed again, each over its own keys: right, but slow (0.6 to 1
 *     us for each key of a row) and rounded differently.
 *   - workspace: pa_paged_attention_scored_workspace_size(...) bytes, 256-byte
 *     aligned, any contents; calls with different bounds may share it one after
 *     another.
 *   - out, lse and the workspace may not share bytes with an input or with one
 *     another (PA_ERR_INVALID_ARG).
 *   - A query_start_loc that decreases may leave rows unwritten: its requests
 *     may form more row tiles than the bounds below allow for.
 * Limits (PA_ERR_UNSUPPORTED), with G = Hq / Hkv <= 128 and head dims of 128, 256
 * and 512: num_seqs <= 8192; num_seqs * max_query_len * Hq <= INT32_MAX;
 * max_seq_len <= INT32_MAX - 4096; where max_query_len * G > 32, with
 *   tiles = min(num_seqs * ceil(max_query_len * G / R), num_q_tokens * G / R + num_seqs),
 *   R = 256 at head dim 128 if max_query_len * G > 128, else 128,
 * num_seqs + tiles <= 23998 and tiles * Hkv * (max_seq_len / 128 + 4) < 2^30, and
 * where it is not, num_seqs * Hkv < 2^26 and num_seqs * Hkv * (max_seq_len / 32 + 2)
 * < 2^31.
 */
PA_API pa_status pa_paged_attention_scored(const void *q, int64_t num_q_tokens, int64_t q_tok_stride,
                                           int32_t num_q_heads, const pa_kv_cache *cache,
                                           const int32_t *block_tables, int32_t max_blocks_per_seq,
                                           const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
                                           int32_t max_query_len, int32_t max_seq_len, float scale,
                                           const pa_score_rules *rules, void *out, float *lse, void *workspace,
                                           size_t workspace_bytes, pa_stream_t stream);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * flag.  Returns PA_OK, PA_ERR_BAD_METADATA or PA_ERR_TIMEOUT (or
 * PA_ERR_CUDA if the synchronisation failed).  *first_bad_index (may be
 * NULL) receives the token index (cache write) or request index (attention)
 * of the first recorded error, else -1.
 */
PA_API pa_status pa_check_errors(pa_stream_t stream, int64_t *first_bad_index);

/*
 * Sets the time limit of the one wait in the split-KV fold that depends on
 * other CTAs (the folders of a (request, KV head) group waiting until every
 * CTA of the group has published its chunk state), and of the waits for copied
 * pages in pa_paged_attention_quant's direct kernels, and returns the previous
 * limit.  The default is 2 s.  It exists to exercise the timeout path ("ROCm:
 * harden compact peer-local KV prefill for Gemma-4", Required hardening:
 * bounded waits, fatal after submit, no retry): with 0 the waiting CTAs give
 * up at once, latch PA_ERR_TIMEOUT and leave their share of the rows
 * unwritten; the kernel still ends normally.  While nothing is copied or
 * computed at that point, no other wait is affected.  In the direct kernels
 * every wait then gives up at once, and a CTA ends when the copies that it
 * asked for have landed (2 s at most).  The value is read at
 * each launch (a captured CUDA graph keeps the value of its capture) and is
 * process-wide.  After a call that reported PA_ERR_TIMEOUT, zero-fill the
 * workspace before reusing it (that of pa_paged_attention_quant needs no
 * particular contents).
 */
PA_API uint64_t pa_set_fold_wait_limit_ns(uint64_t limit_ns);

/* Static, human-readable name of a status code. */
PA_API const char *pa_status_string(pa_status status);

/*
 * Copies a one-line description of the calling thread's most recent launch
 * (schedule, grid, chunk count, KV tile) into buf (NUL-terminated,
 * truncated to n bytes) -- the "selected entrypoint" breadcrumb of
 * [R] Changes.
 */
PA_API void pa_last_launch_info(char *buf, size_t n);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */

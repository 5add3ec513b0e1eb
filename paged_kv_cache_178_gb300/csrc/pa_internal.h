// Internal interface between the C-ABI front end (pa_api.cu) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pa {

// Device-side error latch: the first error code and the index it concerns.
struct ErrState {
    unsigned int code;
    unsigned int pad;
    long long index;
};

enum : unsigned int { kErrBadMetadata = 4u, kErrTimeout = 5u, kErrBudget = 3u };

__device__ __forceinline__ void record_error(ErrState *e, unsigned int code, long long index)
{
    if (atomicCAS(&e->code, 0u, code) == 0u)
        atomicExch(reinterpret_cast<unsigned long long *>(&e->index),
                   static_cast<unsigned long long>(index));
}

// Validated, host-side description of one attention call.
struct AttnArgs {
    const void *q;
    int64_t num_q_tokens;
    int64_t q_tok_stride;
    int32_t num_q_heads;
    const void *k;
    const void *v;
    int64_t num_blocks;
    int32_t num_kv_heads;
    int32_t head_dim;
    int64_t block_stride, token_stride, head_stride;
    const int32_t *block_tables;
    int32_t max_blocks_per_seq;
    const int32_t *seq_lens;
    const int32_t *query_start_loc;
    int32_t num_seqs;
    int32_t max_query_len;
    int32_t max_seq_len;
    float scale;
    void *out;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    // The preceding kernel of the stream writes only the K/V pool: the
    // kernel may read everything else before that kernel has finished.
    bool early_reads;
};

// Work decomposition chosen from host scalars only.
struct AttnPlan {
    int head_dim;
    int group;          // Hq / Hkv
    int tokens_per_tile;  // query tokens per 128-row tile
    int qtiles;         // grid extent over query tiles
    int nch;            // grid extent over KV chunks (1 unless split)
    bool split;         // split-KV with partial states + in-kernel merge
    int cpu;            // split-KV: consecutive chunks per CTA (>= 1)
    int cl;             // CTAs per cluster (2: a CTA pair shares each MMA, in-CTA schedule)
    int ws_rows;        // rows per partial-state record
    size_t ws_counter_bytes;
    size_t ws_bytes;    // total workspace needed
    long long grid;     // CTAs (or clusters x 2 for Dh=512)
    int kt;             // keys per KV tile: the fixed arithmetic's tile (64 or 128)
};

bool plan_attention(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                    int32_t head_dim, int32_t max_query_len, int32_t max_seq_len, AttnPlan *plan,
                    bool allow_split = true);

// Launch the attention kernel for a validated call.  Returns a CUDA error
// code; *unsupported is set when the shape has no kernel.
cudaError_t launch_attention(const AttnArgs &a, const AttnPlan &plan, ErrState *err,
                             cudaStream_t stream, char *info, size_t info_len);

cudaError_t init_attention_attributes();

// Limit (ns) of the split-KV fold's cross-CTA wait; the setter returns the
// previous value.
uint64_t fold_wait_limit_ns();
uint64_t set_fold_wait_limit_ns(uint64_t ns);

// Head dim 512: two-CTA clusters (pa_attn512.cu).
cudaError_t init_attention512_attributes();
cudaError_t launch_attention512(const AttnArgs &a, const AttnPlan &plan, ErrState *err, cudaStream_t stream);

// Compact active-block gather of one KV head (pa_gather.cu).
cudaError_t launch_gather_kv_head(const void *k, const void *v, int64_t num_blocks, int64_t block_stride,
                                  int64_t token_stride, int64_t head_stride, int32_t kv_head, int32_t head_dim,
                                  const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens,
                                  int32_t num_seqs, void *packed_k, void *packed_v, int64_t capacity_pages,
                                  int32_t *compact_tables, int32_t *compact_offsets, ErrState *err,
                                  cudaStream_t stream, int num_sms);
constexpr int kGatherMaxSeqsHost = 512;

// Step metadata (pa_step.cu); the fields are pa_build_step_metadata's arguments.
struct StepMetaArgs {
    const int32_t *context_lens, *query_lens;
    int32_t num_seqs;
    int32_t *block_tables;
    int32_t max_blocks;
    const int32_t *free_pages;
    int32_t num_free;
    const int32_t *cursor_in;
    int32_t *cursor_out;
    int64_t num_blocks;
    int64_t *slot_mapping;
    int32_t *positions;
    int64_t num_tokens;
    int32_t *seq_lens, *query_start_loc;
};
cudaError_t launch_step_metadata(const StepMetaArgs &a, ErrState *err, cudaStream_t stream, int num_sms, int *grid);
constexpr int kScanMaxSeqsHost = 8192;  // kScanMaxSeqs of pa_scan.cuh

// Norm and rotation of q and k (pa_step.cu).  Tensor strides in 16-byte units.
struct RopeArgs {
    const uint4 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    int32_t num_q_heads, num_kv_heads, head_dim;
    int64_t num_tokens;
    const int32_t *positions;
    const float *cos_sin;
    int64_t max_positions;
    int32_t rot_dim, interleaved;
    const uint4 *q_weight, *k_weight;
    float weight_offset, eps;
    uint4 *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
    // with the cache write: the pool (k_cache not null), no k_out
    uint4 *k_cache, *v_cache;
    int64_t num_slots, block_stride, token_stride, head_stride;
    const int64_t *slot_mapping;
    int32_t steps_per_task;  // set by the launch
};
cudaError_t launch_qk_norm_rope(const RopeArgs &a, ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid);
cudaError_t init_step_attributes();

// 4-bit cache: write and read-back (pa_quant.cu).  Pool strides in bytes.
struct QuantPool {
    uint8_t *k, *v;
    int64_t num_blocks, block_stride, head_stride;
    int32_t num_kv_heads, head_dim;
    float k_scale, v_scale;
};
cudaError_t launch_quant_write(const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                               int64_t num_tokens, const QuantPool &pool, const int64_t *slot_mapping, ErrState *err,
                               cudaStream_t stream, int num_sms, int64_t *grid);
// compact_tables has out_cols columns (columns past them are not written).
// With poison_tables a total above the capacity fills compact_tables with -1,
// and the first entry of a request with a bad block id is -1.
// zero_bytes bytes at `zero` (16-byte aligned, may be 0) are cleared.
cudaError_t launch_dequantize_kv(const QuantPool &pool, const int32_t *block_tables, int32_t max_blocks,
                                 const int32_t *seq_lens, int32_t num_seqs, void *k_out, void *v_out,
                                 int64_t capacity_pages, int32_t *compact_tables, int32_t out_cols,
                                 int32_t *compact_offsets, bool poison_tables, void *zero, size_t zero_bytes,
                                 ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid);
cudaError_t init_quant_attributes();

// Attention of few rows over a 4-bit pool (pa_attn_quant.cu).
struct QuantAttnArgs {
    const void *q;
    int64_t num_q_tokens, q_tok_stride;
    int32_t num_q_heads;
    QuantPool pool;
    const int32_t *block_tables;
    int32_t max_blocks;
    const int32_t *seq_lens, *query_start_loc;
    int32_t num_seqs, max_query_len, max_seq_len;
    float scale;
    void *out;
    float *lse;
    int64_t max_pages;  // 0: what the bounds allow
    void *workspace;    // quant_attn_bytes
};
// Tiles that a request's tokens form there, at most 32 rows each (16 at head
// dim 512), or 0 when the call is not one for these kernels: more than two
// tiles a request only where that is faster than reading the pages back.
constexpr int kQuantMaxTiles = 2048;
int quant_attn_tiles(int32_t num_seqs, int32_t num_kv_heads, int head_dim, int group, int32_t max_query_len,
                     int32_t max_seq_len);
// rows: of a tile
size_t quant_attn_bytes(int32_t num_seqs, int tiles, int32_t num_kv_heads, int32_t head_dim, int rows,
                        int32_t max_seq_len, int64_t max_pages);
cudaError_t launch_quant_attention(const QuantAttnArgs &a, ErrState *err, cudaStream_t stream, char *info,
                                   size_t info_len);
cudaError_t init_quant_attention_attributes();

// Encodes a tiled tensor map (driver entry point fetched at run time).
CUresult encode_tiled(CUtensorMap *map, CUtensorMapDataType dtype, cuuint32_t rank, void *base,
                      const cuuint64_t *dims, const cuuint64_t *strides_bytes,
                      const cuuint32_t *box, CUtensorMapSwizzle swizzle);

}  // namespace pa

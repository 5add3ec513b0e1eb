// pa_paged_attention_scored: attention over the BF16 pool whose scores are
// capped, biased by distance or masked.
#include "pa_scored.h"

namespace pa {

bool scored_pool_maps(const ScoreParams &p, int32_t head_dim, CUtensorMap (&tm)[2])
{
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)p.hkv, 16, (cuuint64_t)p.num_blocks};
    const cuuint64_t strides[3] = {(cuuint64_t)p.head_stride * 2, (cuuint64_t)p.token_stride * 2,
                                   (cuuint64_t)p.block_stride * 2};
    const cuuint32_t box[4] = {64, 1, 16, 1};
    for (int i = 0; i < 2; ++i)
        if (encode_tiled(&tm[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<__nv_bfloat16 *>(i ? p.v : p.k), dims,
                         strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return false;
    return true;
}

// Few rows a request go to the kernel whose work follows the bytes, others to
// the one that fills tensor-memory tiles.  Measured, us, few rows / tiles, for 4 and 32
// requests of 4096 keys and 8 of 512, two KV heads (one at head dim 512), capped:
//   16 rows   Dh 128  10.5 / 23.8   30.1 / 40.9    8.7 / 15.8
//             Dh 256  14.5 / 27.4   50.4 / 69.4   10.4 / 18.3
//             Dh 512  16.3 / 33.7   56.0 / 97.9   11.5 / 20.2
//   32 rows   Dh 128  14.5 / 23.2   42.8 / 40.8   11.1 / 15.7
//             Dh 256  19.9 / 27.0   73.8 / 69.8   13.5 / 18.1
//             Dh 512  22.4 / 30.8   79.6 / 97.6   15.7 / 20.2
// (The few-rows kernel takes the rows of a request and KV head in one tile of at most
// 32: a second tile would read the keys again.)
static bool few_rows(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len, int32_t max_seq_len)
{
    return (int64_t)max_query_len * group <= 32 &&
           scored_rows_fits(num_seqs, hkv, head_dim, max_seq_len);
}

bool scored_supported(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_query_len,
                      int32_t max_seq_len, int64_t num_q_tokens)
{
    const int group = hq / hkv;
    return few_rows(num_seqs, hkv, group, head_dim, max_query_len, max_seq_len) ||
           scored_tiles_fits(num_seqs, hkv, group, head_dim, max_query_len, max_seq_len, num_q_tokens);
}

size_t scored_workspace_bytes(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_query_len,
                              int32_t max_seq_len)
{
    const int group = hq / hkv;
    return few_rows(num_seqs, hkv, group, head_dim, max_query_len, max_seq_len)
               ? scored_rows_bytes(num_seqs, hkv, group, head_dim, max_query_len, max_seq_len)
               : scored_tiles_bytes(group, head_dim, max_query_len);
}

static ScoreParams score_params(const AttnArgs &a, const ScoreRules &r, ErrState *err)
{
    ScoreParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.q_tok_stride = a.q_tok_stride;
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.num_blocks = a.num_blocks;
    p.block_stride = a.block_stride;
    p.token_stride = a.token_stride;
    p.head_stride = a.head_stride;
    p.block_tables = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.qsl = a.query_start_loc;
    p.slopes = r.slopes;
    p.prefix_lens = r.prefix_lens;
    p.first_keys = r.first_keys;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.err = err;
    p.num_q_tokens = a.num_q_tokens;
    p.max_blocks = a.max_blocks_per_seq;
    p.num_seqs = a.num_seqs;
    p.hq = a.num_q_heads;
    p.hkv = a.num_kv_heads;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.max_query_len = a.max_query_len;
    p.max_seq_len = a.max_seq_len;
    p.window = r.window > 0 ? r.window : INT32_MAX;
    p.scale_log2 = r.soft_cap > 0.f ? 2.f * a.scale * kLog2e / r.soft_cap : a.scale * kLog2e;
    p.cap_log2 = r.soft_cap * kLog2e;
    return p;
}

cudaError_t launch_scored_attention(const AttnArgs &a, const ScoreRules &r, ErrState *err, cudaStream_t stream,
                                    char *info, size_t info_len)
{
    const ScoreParams p = score_params(a, r, err);
    return few_rows(p.num_seqs, p.hkv, p.group, a.head_dim, p.max_query_len, p.max_seq_len)
               ? launch_scored_rows(p, a.head_dim, a.workspace, stream, info, info_len)
               : launch_scored_tiles(p, a.head_dim, a.workspace, stream, info, info_len);
}

cudaError_t init_scored_attributes()
{
    const cudaError_t e = init_scored_rows_attributes();
    return e == cudaSuccess ? init_scored_tiles_attributes() : e;
}

}  // namespace pa

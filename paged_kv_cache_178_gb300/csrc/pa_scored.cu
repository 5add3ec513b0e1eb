// pa_paged_attention_scored: attention over the BF16 pool whose scores are
// capped, biased by distance or masked.
#include <cstdio>

#include "pa_score.cuh"

namespace pa {

constexpr int kRowThreads = 256;

// A warp per (token, head) row.
template <int DH>
__global__ void __launch_bounds__(kRowThreads) scored_rows_kernel(const ScoreParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, warp = blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    const ReqMeta m = score_meta(p, b);
    if (!m.ok && blockIdx.x == 0 && threadIdx.x == 0)
        record_error(p.err, kErrBadMetadata, b);
    if (!m.sane)
        return;
    for (int64_t r = warp; r < (int64_t)m.qn * p.hq; r += (int64_t)gridDim.x * (kRowThreads / 32)) {
        if (m.ok) {
            scored_row<DH>(p, b, m, (int)(r / p.hq), (int)(r % p.hq));
            continue;
        }
        const int64_t at = (int64_t)m.qs * p.hq + r;
        for (int d = lane; d < DH; d += 32)
            p.out[at * DH + d] = __ushort_as_bfloat16(0x7FC0);
        if (lane == 0 && p.lse)
            p.lse[at] = __int_as_float(0x7FC00000);
    }
}

size_t scored_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

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
    const int64_t rows = (int64_t)a.max_query_len * a.num_q_heads;
    int64_t blocks = (rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (blocks > 4096)
        blocks = 4096;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)a.num_seqs);
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    snprintf(info, info_len, "scored attention dh=%d rows grid=%lldx%d", a.head_dim, (long long)blocks, a.num_seqs);
    return cudaLaunchKernelEx(&cfg, a.head_dim == 128   ? scored_rows_kernel<128>
                                    : a.head_dim == 256 ? scored_rows_kernel<256>
                                                        : scored_rows_kernel<512>,
                              p);
}

cudaError_t init_scored_attributes() { return cudaSuccess; }

}  // namespace pa

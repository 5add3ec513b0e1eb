// C-ABI front end of libpagedattn.so: argument validation, the cache write
// kernel (K1), the device error latch and launch breadcrumbs.  The attention
// kernel lives in pa_attn.cu.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/pagedattn.h"
#include "pa_internal.h"

namespace pa {

// One error latch per device (each device that loads the module has its own
// copy); host code reaches it through cudaGetSymbolAddress.
__device__ ErrState g_err_state;

constexpr int kMaxDevices = 64;
static std::mutex g_mu;
static ErrState *g_err_ptr[kMaxDevices];
static bool g_attr_done[kMaxDevices];
static int g_num_sms[kMaxDevices];
static thread_local char g_last_info[256] = "none";

static pa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// Per-device one-time set-up: resolve the error latch address and set kernel
// attributes.  Must run with the device current.
static pa_status device_setup(ErrState **err_out, int *num_sms = nullptr)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return PA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_attr_done[dev]) {
        void *ptr = nullptr;
        if (cudaGetSymbolAddress(&ptr, g_err_state) != cudaSuccess)
            return PA_ERR_CUDA;
        if (init_attention_attributes() != cudaSuccess || init_step_attributes() != cudaSuccess ||
            init_quant_attributes() != cudaSuccess || init_quant_attention_attributes() != cudaSuccess ||
            init_page_attributes() != cudaSuccess || init_scored_attributes() != cudaSuccess)
            return PA_ERR_CUDA;
        if (cudaDeviceGetAttribute(&g_num_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return PA_ERR_CUDA;
        g_err_ptr[dev] = static_cast<ErrState *>(ptr);
        g_attr_done[dev] = true;
    }
    if (err_out)
        *err_out = g_err_ptr[dev];
    if (num_sms)
        *num_sms = g_num_sms[dev];
    return PA_OK;
}

CUresult encode_tiled(CUtensorMap *map, CUtensorMapDataType dtype, cuuint32_t rank, void *base,
                      const cuuint64_t *dims, const cuuint64_t *strides_bytes, const cuuint32_t *box,
                      CUtensorMapSwizzle swizzle)
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (!fn)
        return CUDA_ERROR_NOT_FOUND;
    cuuint32_t elem_strides[5] = {1, 1, 1, 1, 1};
    return fn(map, dtype, rank, base, dims, strides_bytes, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// K1: slot-mapped cache write.  One thread per 16-byte vector of one
// (token, kv head, K-or-V) row.  Offsets are 64-bit.
__global__ void __launch_bounds__(256) reshape_and_cache_kernel(
    const uint4 *__restrict__ key, int64_t key_tok_stride, const uint4 *__restrict__ value,
    int64_t value_tok_stride, int64_t num_tokens, int32_t num_kv_heads, int32_t vecs_per_row,
    uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache, int64_t num_slots, int64_t block_stride,
    int64_t token_stride, int64_t head_stride, const int64_t *__restrict__ slot_mapping, ErrState *err)
{
    // Launched with programmatic stream serialization: wait for the preceding
    // grid of the stream (it may have produced key, value or slot_mapping),
    // then let the dependent grid be scheduled.  The attention that usually
    // follows may read its metadata and q from here on -- the grids before
    // this one have completed -- and waits for this grid before touching the
    // cache.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // strides arrive in 16-byte units
    const int64_t total = num_tokens * num_kv_heads * 2 * vecs_per_row;
    for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int vec = (int)(idx % vecs_per_row);
        int64_t rest = idx / vecs_per_row;
        const int which = (int)(rest % 2);
        rest /= 2;
        const int h = (int)(rest % num_kv_heads);
        const int64_t i = rest / num_kv_heads;
        // the source vector does not depend on the slot: both loads are in
        // flight together (token i's row exists whatever its slot says)
        const uint4 src = which == 0 ? __ldg(key + i * key_tok_stride + (int64_t)h * vecs_per_row + vec)
                                     : __ldg(value + i * value_tok_stride + (int64_t)h * vecs_per_row + vec);
        const int64_t slot = __ldg(slot_mapping + i);
        if (slot < 0)
            continue;
        if (slot >= num_slots) {
            if (vec == 0 && which == 0 && h == 0)
                record_error(err, kErrBadMetadata, i);
            continue;
        }
        const int64_t dst = (slot >> 4) * block_stride + (slot & 15) * token_stride + h * head_stride + vec;
        (which == 0 ? k_cache : v_cache)[dst] = src;
    }
}

// Staging copy (pa_copy_to_device): 16-byte vectors, up to four per thread
// per pass with every load issued before the stores, so a source in host
// memory costs one round trip over the CPU-GPU link per pass; the bytes past
// the last whole vector go one by one.  With src_ready the first pass reads
// before the wait for the preceding grid (no grid in flight writes src);
// every store still waits for it (it may read dst).
__global__ void __launch_bounds__(256) copy_to_device_kernel(uint4 *__restrict__ dst, const uint4 *__restrict__ src,
                                                             int64_t n16, uint8_t *__restrict__ dst_tail,
                                                             const uint8_t *__restrict__ src_tail, int tail,
                                                             int src_ready)
{
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    int64_t base = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    uint4 v[4];
    uint8_t t8 = 0;
    const bool tail_thread = blockIdx.x == 0 && (int)threadIdx.x < tail;
    if (src_ready) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (base + i * stride < n16)
                v[i] = src[base + i * stride];
        if (tail_thread)
            t8 = src_tail[threadIdx.x];
    }
    // programmatic stream serialization: the preceding grid may still read
    // dst (and, without src_ready, write src) until it has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (bool first = true; base < n16; base += 4 * stride, first = false) {
        if (!first || !src_ready) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (base + i * stride < n16)
                    v[i] = src[base + i * stride];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (base + i * stride < n16)
                dst[base + i * stride] = v[i];
    }
    if (tail_thread)
        dst_tail[threadIdx.x] = src_ready ? t8 : src_tail[threadIdx.x];
}

}  // namespace pa

using namespace pa;

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The attention's KV tile: 0 (the head dim's default), or a tile that head
// dim has -- 64 or 128 at head dim 128, 128 at 256, 64 at 512.
static pa_status check_kv_tile(const pa_kv_cache *c)
{
    const int t = c->kv_tile;
    if (t == 0)
        return PA_OK;
    if (t != 64 && t != 128)
        return PA_ERR_INVALID_ARG;
    const bool ok = c->head_dim == 128 || (c->head_dim == 256 && t == 128) || (c->head_dim == 512 && t == 64);
    return ok ? PA_OK : PA_ERR_UNSUPPORTED;
}

static pa_status check_cache(const pa_kv_cache *c)
{
    if (!c || !c->k || !c->v)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v))
        return PA_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (c->block_size != 16)
        return PA_ERR_UNSUPPORTED;
    if (c->head_dim != 128 && c->head_dim != 256 && c->head_dim != 512)
        return PA_ERR_UNSUPPORTED;
    if (c->block_stride <= 0 || c->token_stride <= 0 || c->head_stride <= 0)
        return PA_ERR_INVALID_ARG;
    if ((c->block_stride | c->token_stride | c->head_stride) & 7)
        return PA_ERR_INVALID_ARG;
    if (c->head_stride < c->head_dim || c->num_blocks > (int64_t)1 << 31)
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

extern "C" {

const char *pa_status_string(pa_status s)
{
    switch (s) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
    case PA_ERR_BAD_METADATA: return "PA_ERR_BAD_METADATA";
    case PA_ERR_TIMEOUT: return "PA_ERR_TIMEOUT";
    case PA_ERR_CUDA: return "PA_ERR_CUDA";
    }
    return "PA_ERR_UNKNOWN";
}

void pa_last_launch_info(char *buf, size_t n)
{
    if (!buf || !n)
        return;
    snprintf(buf, n, "%s", g_last_info);
}

pa_status pa_init(void) { return device_setup(nullptr); }

// Cache-write arguments after validation.
struct ReshapeCall {
    const void *key, *value;
    int64_t key_tok_stride, value_tok_stride, num_tokens;
    const pa_kv_cache *cache;
    const int64_t *slot_mapping;
};

static pa_status reshape_check(const ReshapeCall &c)
{
    pa_status st = check_cache(c.cache);
    if (st != PA_OK)
        return st;
    if (c.num_tokens < 0)
        return PA_ERR_INVALID_ARG;
    if (c.num_tokens == 0)
        return PA_OK;
    const int64_t row = (int64_t)c.cache->num_kv_heads * c.cache->head_dim;
    if (!c.key || !c.value || !c.slot_mapping || !aligned16(c.key) || !aligned16(c.value))
        return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(c.slot_mapping) & 7u) != 0)
        return PA_ERR_INVALID_ARG;
    if (c.key_tok_stride < row || c.value_tok_stride < row || (c.key_tok_stride & 7) || (c.value_tok_stride & 7))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

static pa_status reshape_launch(const ReshapeCall &c, ErrState *err, cudaStream_t stream, char *info,
                                size_t info_len)
{
    if (c.num_tokens == 0) {
        snprintf(info, info_len, "reshape_and_cache tokens=0 (nothing launched)");
        return PA_OK;
    }
    const pa_kv_cache *cache = c.cache;
    const int vecs = cache->head_dim / 8;
    const int64_t total = c.num_tokens * cache->num_kv_heads * 2 * vecs;
    int64_t blocks = (total + 255) / 256;
    if (blocks > 152 * 16)
        blocks = 152 * 16;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg, reshape_and_cache_kernel, static_cast<const uint4 *>(c.key), (int64_t)(c.key_tok_stride / 8),
        static_cast<const uint4 *>(c.value), (int64_t)(c.value_tok_stride / 8), c.num_tokens,
        (int32_t)cache->num_kv_heads, (int32_t)vecs, static_cast<uint4 *>(cache->k), static_cast<uint4 *>(cache->v),
        (int64_t)(cache->num_blocks * 16), (int64_t)(cache->block_stride / 8), (int64_t)(cache->token_stride / 8),
        (int64_t)(cache->head_stride / 8), c.slot_mapping, err);
    snprintf(info, info_len, "reshape_and_cache tokens=%lld grid=%lld block=256", (long long)c.num_tokens,
             (long long)blocks);
    return cuda_status(e);
}

// Validates an attention call and fills the kernel arguments and the plan.
// *empty is set when there is nothing to launch.
static pa_status attention_check(const void *q, int64_t num_q_tokens, int64_t q_tok_stride, int32_t num_q_heads,
                                 const pa_kv_cache *cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
                                 int32_t max_query_len, int32_t max_seq_len, float scale, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, AttnArgs *a, AttnPlan *pl, bool *empty)
{
    *empty = false;
    pa_status st = check_cache(cache);
    if (st != PA_OK)
        return st;
    if ((st = check_kv_tile(cache)) != PA_OK)
        return st;
    if (num_q_heads <= 0 || num_seqs < 0 || max_query_len < 0 || max_seq_len < 0 || num_q_tokens < 0 ||
        max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (num_q_heads % cache->num_kv_heads != 0 || num_q_heads / cache->num_kv_heads > 128)
        return PA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || scale == INFINITY)  // also rejects NaN
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_q_tokens == 0 || max_query_len == 0) {
        *empty = true;
        return PA_OK;
    }
    const int64_t row = (int64_t)num_q_heads * cache->head_dim;
    if (!q || !out || !block_tables || !seq_lens || !query_start_loc || !aligned16(q) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
        return PA_ERR_INVALID_ARG;
    if (q_tok_stride < row || (q_tok_stride & 7) || num_q_tokens > ((int64_t)1 << 31) - 1)
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq == 0)
        return PA_ERR_INVALID_ARG;
    if (!plan_attention(num_seqs, num_q_heads, cache->num_kv_heads, cache->head_dim, max_query_len, max_seq_len,
                        pl))
        return PA_ERR_UNSUPPORTED;
    if (cache->kv_tile != 0)
        pl->kt = cache->kv_tile;
    if (pl->ws_bytes > 0) {
        if (!workspace || workspace_bytes < pl->ws_bytes)
            return PA_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return PA_ERR_INVALID_ARG;
    }
    a->q = q;
    a->num_q_tokens = num_q_tokens;
    a->q_tok_stride = q_tok_stride;
    a->num_q_heads = num_q_heads;
    a->k = cache->k;
    a->v = cache->v;
    a->num_blocks = cache->num_blocks;
    a->num_kv_heads = cache->num_kv_heads;
    a->head_dim = cache->head_dim;
    a->block_stride = cache->block_stride;
    a->token_stride = cache->token_stride;
    a->head_stride = cache->head_stride;
    a->block_tables = block_tables;
    a->max_blocks_per_seq = max_blocks_per_seq;
    a->seq_lens = seq_lens;
    a->query_start_loc = query_start_loc;
    a->num_seqs = num_seqs;
    a->max_query_len = max_query_len;
    a->max_seq_len = max_seq_len;
    a->scale = scale;
    a->out = out;
    a->lse = lse;
    a->workspace = workspace;
    a->workspace_bytes = workspace_bytes;
    a->early_reads = false;
    return PA_OK;
}

static pa_status attention_launch(const AttnArgs &a, const AttnPlan &pl, ErrState *err, cudaStream_t stream,
                                  char *info, size_t info_len)
{
    cudaError_t e = launch_attention(a, pl, err, stream, info, info_len);
    if (e == cudaErrorNotSupported)
        return PA_ERR_UNSUPPORTED;
    return cuda_status(e);
}

// Half-open byte range [lo, hi) of a device buffer.
struct Span {
    uintptr_t lo, hi;
};

static Span span(const void *p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

static bool overlaps(const Span &x, const Span &y) { return x.lo < y.hi && y.lo < x.hi; }

// Bytes spanned by one view of the pool (K or V).
static int64_t pool_view_bytes(const pa_kv_cache *c)
{
    return ((c->num_blocks - 1) * c->block_stride + 15 * c->token_stride +
            (int64_t)(c->num_kv_heads - 1) * c->head_stride + c->head_dim) *
           2;
}

pa_status pa_reshape_and_cache(const void *key, int64_t key_tok_stride, const void *value,
                               int64_t value_tok_stride, int64_t num_tokens, const pa_kv_cache *cache,
                               const int64_t *slot_mapping, pa_stream_t stream)
{
    const ReshapeCall c{key, value, key_tok_stride, value_tok_stride, num_tokens, cache, slot_mapping};
    pa_status st = reshape_check(c);
    if (st != PA_OK)
        return st;
    ErrState *err = nullptr;
    if (num_tokens > 0 && (st = device_setup(&err)) != PA_OK)
        return st;
    return reshape_launch(c, err, reinterpret_cast<cudaStream_t>(stream), g_last_info, sizeof g_last_info);
}

pa_status pa_copy_to_device(void *dst, const void *src, size_t bytes, int32_t src_ready, pa_stream_t stream)
{
    if (bytes == 0)
        return PA_OK;
    if (!dst || !src)
        return PA_ERR_INVALID_ARG;
    const uintptr_t d = reinterpret_cast<uintptr_t>(dst), s = reinterpret_cast<uintptr_t>(src);
    if (d < s + bytes && s < d + bytes)
        return PA_ERR_INVALID_ARG;  // overlapping ranges
    if ((d | s) & 15u)
        return PA_ERR_INVALID_ARG;  // both 16-byte aligned
    ErrState *err = nullptr;
    pa_status st = device_setup(&err);
    if (st != PA_OK)
        return st;
    const int64_t n16 = (int64_t)(bytes / 16);
    const int tail = (int)(bytes % 16);
    int64_t blocks = (n16 + 4 * 256 - 1) / (4 * 256);
    if (blocks < 1)
        blocks = 1;
    if (blocks > 152 * 8)
        blocks = 152 * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, copy_to_device_kernel, static_cast<uint4 *>(dst), static_cast<const uint4 *>(src),
                           n16, static_cast<uint8_t *>(dst) + n16 * 16, static_cast<const uint8_t *>(src) + n16 * 16,
                           tail, src_ready ? 1 : 0);
    snprintf(g_last_info, sizeof g_last_info, "copy_to_device bytes=%zu grid=%lld block=256", bytes,
             (long long)blocks);
    return cuda_status(e);
}

size_t pa_paged_attention_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t max_query_len, int32_t max_seq_len)
{
    AttnPlan pl{};
    if (!plan_attention(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len, &pl))
        return 0;
    return pl.ws_bytes;
}

pa_status pa_paged_attention(const void *q, int64_t num_q_tokens, int64_t q_tok_stride, int32_t num_q_heads,
                             const pa_kv_cache *cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
                             int32_t max_query_len, int32_t max_seq_len, float scale, void *out, float *lse,
                             void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    AttnArgs a;
    AttnPlan pl{};
    bool empty = false;
    pa_status st = attention_check(q, num_q_tokens, q_tok_stride, num_q_heads, cache, block_tables,
                                   max_blocks_per_seq, seq_lens, query_start_loc, num_seqs, max_query_len,
                                   max_seq_len, scale, out, lse, workspace, workspace_bytes, &a, &pl, &empty);
    if (st != PA_OK)
        return st;
    if (empty) {
        snprintf(g_last_info, sizeof g_last_info, "attention: empty batch (nothing launched)");
        return PA_OK;
    }
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    return attention_launch(a, pl, err, reinterpret_cast<cudaStream_t>(stream), g_last_info, sizeof g_last_info);
}

pa_status pa_reshape_and_paged_attention(const void *key, int64_t key_tok_stride, const void *value,
                                         int64_t value_tok_stride, int64_t num_new_tokens,
                                         const int64_t *slot_mapping, const void *q, int64_t num_q_tokens,
                                         int64_t q_tok_stride, int32_t num_q_heads, const pa_kv_cache *cache,
                                         const int32_t *block_tables, int32_t max_blocks_per_seq,
                                         const int32_t *seq_lens, const int32_t *query_start_loc,
                                         int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len,
                                         float scale, void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, pa_stream_t stream)
{
    // Validate both calls before launching either.
    const ReshapeCall c{key, value, key_tok_stride, value_tok_stride, num_new_tokens, cache, slot_mapping};
    pa_status st = reshape_check(c);
    if (st != PA_OK)
        return st;
    AttnArgs a;
    AttnPlan pl{};
    bool empty = false;
    st = attention_check(q, num_q_tokens, q_tok_stride, num_q_heads, cache, block_tables, max_blocks_per_seq,
                         seq_lens, query_start_loc, num_seqs, max_query_len, max_seq_len, scale, out, lse,
                         workspace, workspace_bytes, &a, &pl, &empty);
    if (st != PA_OK)
        return st;
    if (!empty && num_new_tokens > 0) {
        // The attention grid reads q and the metadata, and writes out, lse
        // and the workspace, while the cache write may still run: none of
        // them may share bytes with what the cache write reads or writes.
        const int64_t kv_row = (int64_t)cache->num_kv_heads * cache->head_dim;
        const Span writes_of_write[2] = {span(cache->k, pool_view_bytes(cache)),
                                         span(cache->v, pool_view_bytes(cache))};
        const Span reads_of_write[3] = {span(key, ((num_new_tokens - 1) * key_tok_stride + kv_row) * 2),
                                        span(value, ((num_new_tokens - 1) * value_tok_stride + kv_row) * 2),
                                        span(slot_mapping, num_new_tokens * 8)};
        const Span early_reads[4] = {
            span(q, ((num_q_tokens - 1) * q_tok_stride + (int64_t)num_q_heads * cache->head_dim) * 2),
            span(block_tables, (int64_t)num_seqs * max_blocks_per_seq * 4), span(seq_lens, (int64_t)num_seqs * 4),
            span(query_start_loc, ((int64_t)num_seqs + 1) * 4)};
        const Span attn_writes[3] = {span(out, num_q_tokens * num_q_heads * (int64_t)cache->head_dim * 2),
                                     span(lse, lse ? num_q_tokens * num_q_heads * 4 : 0),
                                     span(workspace, (int64_t)pl.ws_bytes)};
        for (const Span &w : writes_of_write)
            for (const Span &r : early_reads)
                if (overlaps(w, r))
                    return PA_ERR_INVALID_ARG;
        for (const Span &w : attn_writes) {
            for (const Span &x : writes_of_write)
                if (overlaps(w, x))
                    return PA_ERR_INVALID_ARG;
            for (const Span &x : reads_of_write)
                if (overlaps(w, x))
                    return PA_ERR_INVALID_ARG;
        }
    }
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char info_w[128], info_a[192];
    if ((st = reshape_launch(c, err, s, info_w, sizeof info_w)) != PA_OK)
        return st;
    if (empty) {
        snprintf(g_last_info, sizeof g_last_info, "%.80s; attention: empty batch (nothing launched)", info_w);
        return PA_OK;
    }
    // Only a cache write launched just before makes the early reads safe;
    // the head-dim 512 kernel always waits at entry.
    a.early_reads = num_new_tokens > 0 && cache->head_dim != 512;
    st = attention_launch(a, pl, err, s, info_a, sizeof info_a);
    snprintf(g_last_info, sizeof g_last_info, "%.80s; %.160s%s", info_w, info_a, a.early_reads ? " early_reads" : "");
    return st;
}

// Scratch for pa_paged_attention_noalloc: lives in the library image, so
// every device that loads the library holds it; nothing is allocated per call.
static __device__ __align__(256) unsigned char g_noalloc_scratch[PA_NOALLOC_SCRATCH_BYTES];
static void *g_noalloc_ptr[kMaxDevices];

pa_status pa_paged_attention_noalloc(const void *q, int64_t num_q_tokens, int64_t q_tok_stride,
                                     int32_t num_q_heads, const pa_kv_cache *cache,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq,
                                     const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
                                     int32_t max_query_len, int32_t max_seq_len, float scale, void *out,
                                     float *lse, pa_stream_t stream)
{
    // Every host check of pa_paged_attention runs first, against the
    // built-in array's size, before any CUDA call: a stand-in address (256,
    // aligned and never dereferenced) takes the scratch's place until the
    // call is known to be valid.  Bounds that need more scratch than the
    // array holds fail here with PA_ERR_WORKSPACE.
    AttnArgs a;
    AttnPlan pl{};
    bool empty = false;
    pa_status st = attention_check(q, num_q_tokens, q_tok_stride, num_q_heads, cache, block_tables,
                                   max_blocks_per_seq, seq_lens, query_start_loc, num_seqs, max_query_len,
                                   max_seq_len, scale, out, lse, reinterpret_cast<void *>(uintptr_t{256}),
                                   PA_NOALLOC_SCRATCH_BYTES, &a, &pl, &empty);
    if (st != PA_OK)
        return st;
    if (empty) {
        snprintf(g_last_info, sizeof g_last_info, "attention: empty batch (nothing launched)");
        return PA_OK;
    }
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return PA_ERR_CUDA;
    void *scratch = nullptr;
    {
        // Host code cannot use the array's name as a device address: resolve
        // it once per device, with that device current.
        std::lock_guard<std::mutex> lock(g_mu);
        if (!g_noalloc_ptr[dev]) {
            void *ptr = nullptr;
            if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || !ptr)
                return PA_ERR_CUDA;
            g_noalloc_ptr[dev] = ptr;
        }
        scratch = g_noalloc_ptr[dev];
    }
    a.workspace = scratch;
    a.workspace_bytes = PA_NOALLOC_SCRATCH_BYTES;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // The arrival counters at the head of the scratch must start at zero; the
    // previous call (or an aborted one) may have left anything there.
    if (pl.ws_counter_bytes > 0 && cudaMemsetAsync(scratch, 0, pl.ws_counter_bytes, s) != cudaSuccess)
        return PA_ERR_CUDA;
    return attention_launch(a, pl, err, s, g_last_info, sizeof g_last_info);
}

uint64_t pa_set_fold_wait_limit_ns(uint64_t limit_ns) { return set_fold_wait_limit_ns(limit_ns); }

pa_status pa_check_errors(pa_stream_t stream, int64_t *first_bad_index)
{
    if (first_bad_index)
        *first_bad_index = -1;
    ErrState *err = nullptr;
    pa_status st = device_setup(&err);
    if (st != PA_OK)
        return st;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return PA_ERR_CUDA;
    ErrState h{};
    if (cudaMemcpy(&h, err, sizeof h, cudaMemcpyDeviceToHost) != cudaSuccess)
        return PA_ERR_CUDA;
    if (h.code == 0)
        return PA_OK;
    const ErrState zero{};
    if (cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
        return PA_ERR_CUDA;
    if (first_bad_index)
        *first_bad_index = h.index;
    if (h.code == kErrBudget)
        return PA_ERR_WORKSPACE;
    return h.code == kErrTimeout ? PA_ERR_TIMEOUT : PA_ERR_BAD_METADATA;
}

pa_status pa_gather_kv_head(const pa_kv_cache *cache, int32_t kv_head, const int32_t *block_tables,
                            int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs,
                            void *packed_k, void *packed_v, int64_t capacity_pages, int32_t *compact_tables,
                            int32_t *compact_offsets, pa_stream_t stream)
{
    pa_status st = check_cache(cache);
    if (st != PA_OK)
        return st;
    if (kv_head < 0 || kv_head >= cache->num_kv_heads || num_seqs < 0 || max_blocks_per_seq <= 0 ||
        capacity_pages < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > kGatherMaxSeqsHost || (int64_t)num_seqs * max_blocks_per_seq > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) {
        snprintf(g_last_info, sizeof g_last_info, "gather_kv_head: empty batch (nothing launched)");
        return PA_OK;
    }
    if (!block_tables || !seq_lens || !compact_tables || !compact_offsets)
        return PA_ERR_INVALID_ARG;
    if (capacity_pages > 0 && (!packed_k || !packed_v || !aligned16(packed_k) || !aligned16(packed_v)))
        return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(compact_tables) | reinterpret_cast<uintptr_t>(compact_offsets) |
         reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens)) &
        3u)
        return PA_ERR_INVALID_ARG;
    {
        // the kernel writes its four outputs while it reads the pool and the
        // metadata: no output may share a byte with an input or another output
        const int64_t page_bytes = (int64_t)16 * cache->head_dim * 2;
        const int64_t table_bytes = (int64_t)num_seqs * max_blocks_per_seq * 4;
        const Span reads[4] = {span(cache->k, pool_view_bytes(cache)), span(cache->v, pool_view_bytes(cache)),
                               span(block_tables, table_bytes), span(seq_lens, (int64_t)num_seqs * 4)};
        const Span writes[4] = {span(packed_k, capacity_pages * page_bytes),
                                span(packed_v, capacity_pages * page_bytes), span(compact_tables, table_bytes),
                                span(compact_offsets, ((int64_t)num_seqs + 1) * 4)};
        for (int i = 0; i < 4; ++i) {
            for (const Span &r : reads)
                if (overlaps(writes[i], r))
                    return PA_ERR_INVALID_ARG;
            for (int j = i + 1; j < 4; ++j)
                if (overlaps(writes[i], writes[j]))
                    return PA_ERR_INVALID_ARG;
        }
    }
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PA_ERR_CUDA;
    const cudaError_t e = launch_gather_kv_head(
        cache->k, cache->v, cache->num_blocks, cache->block_stride, cache->token_stride, cache->head_stride,
        kv_head, cache->head_dim, block_tables, max_blocks_per_seq, seq_lens, num_seqs, packed_k, packed_v,
        capacity_pages, compact_tables, compact_offsets, err, reinterpret_cast<cudaStream_t>(stream), nsm);
    snprintf(g_last_info, sizeof g_last_info, "gather_kv_head head=%d seqs=%d capacity_pages=%lld", kv_head,
             num_seqs, (long long)capacity_pages);
    return cuda_status(e);
}

// ------------------------------------------------------ step metadata ----
static bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

pa_status pa_build_step_metadata(const int32_t *context_lens, const int32_t *query_lens, int32_t num_seqs,
                                 int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *free_pages,
                                 int32_t num_free_pages, const int32_t *cursor_in, int32_t *cursor_out,
                                 int64_t num_blocks, int64_t *slot_mapping, int32_t *positions, int64_t num_tokens,
                                 int32_t *seq_lens, int32_t *query_start_loc, pa_stream_t stream)
{
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || num_free_pages < 0 || num_blocks <= 0 ||
        num_blocks > (int64_t)1 << 31 || num_tokens < 0 || num_tokens > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    // positions and lengths are 32-bit
    if (num_seqs > kScanMaxSeqsHost || max_blocks_per_seq > INT32_MAX / 16)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) {
        snprintf(g_last_info, sizeof g_last_info, "build_step_metadata: empty batch (nothing launched)");
        return PA_OK;
    }
    if (!context_lens || !query_lens || !block_tables || !cursor_out || !seq_lens || !query_start_loc ||
        (num_free_pages > 0 && !free_pages) || (num_tokens > 0 && (!slot_mapping || !positions)))
        return PA_ERR_INVALID_ARG;
    if (!aligned4(context_lens) || !aligned4(query_lens) || !aligned4(block_tables) || !aligned4(free_pages) ||
        !aligned4(cursor_in) || !aligned4(cursor_out) || !aligned4(seq_lens) || !aligned4(query_start_loc) ||
        !aligned4(positions) || !aligned8(slot_mapping))
        return PA_ERR_INVALID_ARG;
    {
        const int64_t n4 = (int64_t)num_seqs * 4;
        const Span reads[4] = {span(context_lens, n4), span(query_lens, n4),
                               span(free_pages, (int64_t)num_free_pages * 4), span(cursor_in, cursor_in ? 4 : 0)};
        const Span writes[6] = {span(block_tables, n4 * max_blocks_per_seq), span(seq_lens, n4),
                                span(query_start_loc, n4 + 4), span(slot_mapping, num_tokens * 8),
                                span(positions, num_tokens * 4), span(cursor_out, 4)};
        for (int i = 0; i < 6; ++i) {
            for (int j = 0; j < 4; ++j) {
                // lengths and cursor may advance in place
                if ((i == 1 && j == 0 && seq_lens == context_lens) || (i == 5 && j == 3 && cursor_out == cursor_in))
                    continue;
                if (overlaps(writes[i], reads[j]))
                    return PA_ERR_INVALID_ARG;
            }
            for (int j = i + 1; j < 6; ++j)
                if (overlaps(writes[i], writes[j]))
                    return PA_ERR_INVALID_ARG;
        }
    }
    ErrState *err = nullptr;
    int nsm = 0;
    pa_status st = device_setup(&err, &nsm);
    if (st != PA_OK)
        return st;
    const StepMetaArgs a{context_lens, query_lens, num_seqs,   block_tables, max_blocks_per_seq,
                         free_pages,   num_free_pages, cursor_in, cursor_out,   num_blocks,
                         slot_mapping, positions,  num_tokens, seq_lens,     query_start_loc};
    int grid = 0;
    const cudaError_t e = launch_step_metadata(a, err, reinterpret_cast<cudaStream_t>(stream), nsm, &grid);
    snprintf(g_last_info, sizeof g_last_info, "build_step_metadata seqs=%d tokens=%lld grid=%d", num_seqs,
             (long long)num_tokens, grid);
    return cuda_status(e);
}

// ---------------------------------------------- norm, rotation (and write) --
// num_tokens rows of `row` elements, `stride` elements apart.
struct Rows {
    const void *p;
    int64_t stride, row;
};

static Span rows_span(const Rows &r, int64_t n) { return span(r.p, ((n - 1) * r.stride + r.row) * 2); }

// Whether two row sets share bytes.  Rows of one stride that interleave
// without touching (slices of a fused projection) do not.
static bool rows_overlap(const Rows &a, const Rows &b, int64_t n)
{
    if (!overlaps(rows_span(a, n), rows_span(b, n)))
        return false;
    if (a.stride != b.stride || n <= 1)
        return true;
    const int64_t period = a.stride * 2;
    int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % period;
    if (d < 0)
        d += period;
    return d < a.row * 2 || d + b.row * 2 > period;
}

static bool bad_rows(const Rows &r) { return !r.p || !aligned16(r.p) || r.stride < r.row || (r.stride & 7); }

static pa_status rope_call(const Rows &q, int32_t hq, const Rows &k, int32_t hkv, const Rows *value, int32_t head_dim,
                           int64_t num_tokens, const int32_t *positions, const float *cos_sin, int64_t max_positions,
                           int32_t rot_dim, int32_t interleaved, const void *q_weight, const void *k_weight,
                           float weight_offset, float eps, const Rows &q_out, const Rows *k_out,
                           const pa_kv_cache *cache, const int64_t *slot_mapping, pa_stream_t stream, const char *name)
{
    if (num_tokens < 0 || num_tokens > INT32_MAX || max_positions <= 0)
        return PA_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16)
        return PA_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps == INFINITY || !std::isfinite(weight_offset))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) {
        snprintf(g_last_info, sizeof g_last_info, "%s tokens=0 (nothing launched)", name);
        return PA_OK;
    }
    if (bad_rows(q) || bad_rows(k) || bad_rows(q_out) || (value && bad_rows(*value)) || (k_out && bad_rows(*k_out)))
        return PA_ERR_INVALID_ARG;
    if (!positions || !aligned4(positions) || !cos_sin || !aligned16(cos_sin) || !aligned16(q_weight) ||
        !aligned16(k_weight) || (cache && (!slot_mapping || !aligned8(slot_mapping))))
        return PA_ERR_INVALID_ARG;
    {
        const int64_t n = num_tokens;
        // in place: the very rows that are read
        const bool q_same = q_out.p == q.p && q_out.stride == q.stride;
        const bool k_same = k_out && k_out->p == k.p && k_out->stride == k.stride;
        if ((!q_same && rows_overlap(q_out, q, n)) || rows_overlap(q_out, k, n) ||
            (value && rows_overlap(q_out, *value, n)))
            return PA_ERR_INVALID_ARG;
        if (k_out && ((!k_same && rows_overlap(*k_out, k, n)) || rows_overlap(*k_out, q, n) ||
                      rows_overlap(*k_out, q_out, n)))
            return PA_ERR_INVALID_ARG;
        const Span small[5] = {span(positions, n * 4), span(cos_sin, max_positions * rot_dim * 4),
                               span(q_weight, q_weight ? head_dim * 2 : 0), span(k_weight, k_weight ? head_dim * 2 : 0),
                               span(slot_mapping, cache ? n * 8 : 0)};
        const Span pool[2] = {cache ? span(cache->k, pool_view_bytes(cache)) : Span{0, 0},
                              cache ? span(cache->v, pool_view_bytes(cache)) : Span{0, 0}};
        for (const Span &x : small)
            if (overlaps(x, rows_span(q_out, n)) || (k_out && overlaps(x, rows_span(*k_out, n))) || overlaps(x, pool[0]) ||
                overlaps(x, pool[1]))
                return PA_ERR_INVALID_ARG;
        for (const Span &x : pool)
            if (overlaps(x, rows_span(q, n)) || overlaps(x, rows_span(k, n)) || overlaps(x, rows_span(q_out, n)) ||
                (value && overlaps(x, rows_span(*value, n))))
                return PA_ERR_INVALID_ARG;
    }
    ErrState *err = nullptr;
    int nsm = 0;
    const pa_status st = device_setup(&err, &nsm);
    if (st != PA_OK)
        return st;
    RopeArgs a{};
    a.q = static_cast<const uint4 *>(q.p);
    a.k = static_cast<const uint4 *>(k.p);
    a.q_stride = q.stride / 8;
    a.k_stride = k.stride / 8;
    if (value) {
        a.v = static_cast<const uint4 *>(value->p);
        a.v_stride = value->stride / 8;
    }
    a.num_q_heads = hq;
    a.num_kv_heads = hkv;
    a.head_dim = head_dim;
    a.num_tokens = num_tokens;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.max_positions = max_positions;
    a.rot_dim = rot_dim;
    a.interleaved = interleaved != 0;
    a.q_weight = static_cast<const uint4 *>(q_weight);
    a.k_weight = static_cast<const uint4 *>(k_weight);
    a.weight_offset = weight_offset;
    a.eps = eps;
    a.q_out = static_cast<uint4 *>(const_cast<void *>(q_out.p));
    a.q_out_stride = q_out.stride / 8;
    if (k_out) {
        a.k_out = static_cast<uint4 *>(const_cast<void *>(k_out->p));
        a.k_out_stride = k_out->stride / 8;
    }
    if (cache) {
        a.k_cache = static_cast<uint4 *>(cache->k);
        a.v_cache = static_cast<uint4 *>(cache->v);
        a.num_slots = cache->num_blocks * 16;
        a.block_stride = cache->block_stride / 8;
        a.token_stride = cache->token_stride / 8;
        a.head_stride = cache->head_stride / 8;
        a.slot_mapping = slot_mapping;
    }
    int64_t grid = 0;
    const cudaError_t e = launch_qk_norm_rope(a, err, reinterpret_cast<cudaStream_t>(stream), nsm, &grid);
    snprintf(g_last_info, sizeof g_last_info, "%s tokens=%lld grid=%lld", name, (long long)num_tokens, (long long)grid);
    return cuda_status(e);
}

pa_status pa_qk_norm_rope(const void *q, int64_t q_tok_stride, int32_t num_q_heads, const void *k,
                          int64_t k_tok_stride, int32_t num_kv_heads, int32_t head_dim, int64_t num_tokens,
                          const int32_t *positions, const float *cos_sin, int64_t max_positions, int32_t rot_dim,
                          int32_t interleaved, const void *q_weight, const void *k_weight, float weight_offset,
                          float eps, void *q_out, int64_t q_out_tok_stride, void *k_out, int64_t k_out_tok_stride,
                          pa_stream_t stream)
{
    if (num_q_heads <= 0 || num_kv_heads <= 0)
        return PA_ERR_INVALID_ARG;
    if (head_dim != 128 && head_dim != 256 && head_dim != 512)
        return PA_ERR_UNSUPPORTED;
    const int64_t qr = (int64_t)num_q_heads * head_dim, kr = (int64_t)num_kv_heads * head_dim;
    const Rows ko{k_out, k_out_tok_stride, kr};
    return rope_call(Rows{q, q_tok_stride, qr}, num_q_heads, Rows{k, k_tok_stride, kr}, num_kv_heads, nullptr, head_dim,
                     num_tokens, positions, cos_sin, max_positions, rot_dim, interleaved, q_weight, k_weight,
                     weight_offset, eps, Rows{q_out, q_out_tok_stride, qr}, &ko, nullptr, nullptr, stream,
                     "qk_norm_rope");
}

pa_status pa_qk_norm_rope_and_cache(const void *q, int64_t q_tok_stride, int32_t num_q_heads, const void *k,
                                    int64_t k_tok_stride, const void *value, int64_t value_tok_stride,
                                    int64_t num_tokens, const int32_t *positions, const float *cos_sin,
                                    int64_t max_positions, int32_t rot_dim, int32_t interleaved, const void *q_weight,
                                    const void *k_weight, float weight_offset, float eps, void *q_out,
                                    int64_t q_out_tok_stride, const pa_kv_cache *cache, const int64_t *slot_mapping,
                                    pa_stream_t stream)
{
    const pa_status st = check_cache(cache);
    if (st != PA_OK)
        return st;
    if (num_q_heads <= 0)
        return PA_ERR_INVALID_ARG;
    const int32_t hkv = cache->num_kv_heads, dh = cache->head_dim;
    const int64_t qr = (int64_t)num_q_heads * dh, kr = (int64_t)hkv * dh;
    const Rows v{value, value_tok_stride, kr};
    return rope_call(Rows{q, q_tok_stride, qr}, num_q_heads, Rows{k, k_tok_stride, kr}, hkv, &v, dh, num_tokens,
                     positions, cos_sin, max_positions, rot_dim, interleaved, q_weight, k_weight, weight_offset, eps,
                     Rows{q_out, q_out_tok_stride, qr}, nullptr, cache, slot_mapping, stream,
                     "qk_norm_rope_and_cache");
}

// --------------------------------------------------------- 4-bit cache ----
// A power of two in [2^-32, 2^32].
static bool tensor_scale_ok(float s)
{
    int e = 0;
    return s > 0.f && std::isfinite(s) && std::frexp(s, &e) == 0.5f && e - 1 >= -32 && e - 1 <= 32;
}

static pa_status check_quant_cache(const pa_quant_cache *c)
{
    if (!c || !c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))
        return PA_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->num_blocks > (int64_t)1 << 31 || c->num_kv_heads <= 0 || c->head_dim <= 0 ||
        c->reserved != 0)
        return PA_ERR_INVALID_ARG;
    if (c->block_size != 16 || (c->head_dim != 128 && c->head_dim != 256 && c->head_dim != 512))
        return PA_ERR_UNSUPPORTED;
    if (c->block_stride <= 0 || c->head_stride < (int64_t)9 * c->head_dim || ((c->block_stride | c->head_stride) & 15))
        return PA_ERR_INVALID_ARG;
    if (c->block_stride > UINT32_MAX || c->head_stride > UINT32_MAX)
        return PA_ERR_UNSUPPORTED;
    return tensor_scale_ok(c->k_scale) && tensor_scale_ok(c->v_scale) ? PA_OK : PA_ERR_INVALID_ARG;
}

static QuantPool quant_pool(const pa_quant_cache *c)
{
    return QuantPool{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->num_blocks, c->block_stride,
                     c->head_stride,               c->num_kv_heads,              c->head_dim,   c->k_scale,
                     c->v_scale};
}

static int64_t quant_view_bytes(const pa_quant_cache *c)
{
    return (c->num_blocks - 1) * c->block_stride + (int64_t)(c->num_kv_heads - 1) * c->head_stride + 9 * c->head_dim;
}

pa_status pa_reshape_and_cache_quant(const void *key, int64_t key_tok_stride, const void *value,
                                     int64_t value_tok_stride, int64_t num_tokens, const pa_quant_cache *cache,
                                     const int64_t *slot_mapping, pa_stream_t stream)
{
    pa_status st = check_quant_cache(cache);
    if (st != PA_OK)
        return st;
    if (num_tokens < 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) {
        snprintf(g_last_info, sizeof g_last_info, "reshape_and_cache_quant tokens=0 (nothing launched)");
        return PA_OK;
    }
    const int64_t row = (int64_t)cache->num_kv_heads * cache->head_dim;
    const Rows k{key, key_tok_stride, row}, v{value, value_tok_stride, row};
    if (bad_rows(k) || bad_rows(v) || !slot_mapping || !aligned8(slot_mapping))
        return PA_ERR_INVALID_ARG;
    const Span pool[2] = {span(cache->k, quant_view_bytes(cache)), span(cache->v, quant_view_bytes(cache))};
    for (const Span &x : pool)
        if (overlaps(x, rows_span(k, num_tokens)) || overlaps(x, rows_span(v, num_tokens)) ||
            overlaps(x, span(slot_mapping, num_tokens * 8)))
            return PA_ERR_INVALID_ARG;
    ErrState *err = nullptr;
    int nsm = 0;
    if ((st = device_setup(&err, &nsm)) != PA_OK)
        return st;
    int64_t grid = 0;
    const cudaError_t e = launch_quant_write(key, key_tok_stride, value, value_tok_stride, num_tokens,
                                             quant_pool(cache), slot_mapping, err,
                                             reinterpret_cast<cudaStream_t>(stream), nsm, &grid);
    snprintf(g_last_info, sizeof g_last_info, "reshape_and_cache_quant tokens=%lld grid=%lld", (long long)num_tokens,
             (long long)grid);
    return cuda_status(e);
}

pa_status pa_dequantize_kv(const pa_quant_cache *cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                           const int32_t *seq_lens, int32_t num_seqs, void *k_out, void *v_out,
                           int64_t capacity_pages, int32_t *compact_tables, int32_t *compact_offsets,
                           pa_stream_t stream)
{
    pa_status st = check_quant_cache(cache);
    if (st != PA_OK)
        return st;
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || capacity_pages < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > kScanMaxSeqsHost || (int64_t)num_seqs * max_blocks_per_seq > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) {
        snprintf(g_last_info, sizeof g_last_info, "dequantize_kv: empty batch (nothing launched)");
        return PA_OK;
    }
    if (!block_tables || !seq_lens || !compact_tables || !compact_offsets || !aligned4(block_tables) ||
        !aligned4(seq_lens) || !aligned4(compact_tables) || !aligned4(compact_offsets))
        return PA_ERR_INVALID_ARG;
    if (capacity_pages > 0 && (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)))
        return PA_ERR_INVALID_ARG;
    {
        const int64_t out_bytes = capacity_pages * 16 * cache->num_kv_heads * cache->head_dim * 2;
        const int64_t table_bytes = (int64_t)num_seqs * max_blocks_per_seq * 4;
        const Span reads[4] = {span(cache->k, quant_view_bytes(cache)), span(cache->v, quant_view_bytes(cache)),
                               span(block_tables, table_bytes), span(seq_lens, (int64_t)num_seqs * 4)};
        const Span writes[4] = {span(k_out, out_bytes), span(v_out, out_bytes), span(compact_tables, table_bytes),
                                span(compact_offsets, ((int64_t)num_seqs + 1) * 4)};
        for (int i = 0; i < 4; ++i) {
            for (const Span &r : reads)
                if (overlaps(writes[i], r))
                    return PA_ERR_INVALID_ARG;
            for (int j = i + 1; j < 4; ++j)
                if (overlaps(writes[i], writes[j]))
                    return PA_ERR_INVALID_ARG;
        }
    }
    ErrState *err = nullptr;
    int nsm = 0;
    if ((st = device_setup(&err, &nsm)) != PA_OK)
        return st;
    int64_t grid = 0;
    const cudaError_t e = launch_dequantize_kv(quant_pool(cache), block_tables, max_blocks_per_seq, seq_lens, num_seqs,
                                               k_out, v_out, capacity_pages, compact_tables, max_blocks_per_seq,
                                               compact_offsets, false, nullptr, 0, err,
                                               reinterpret_cast<cudaStream_t>(stream), nsm, &grid);
    snprintf(g_last_info, sizeof g_last_info, "dequantize_kv seqs=%d capacity_pages=%lld grid=%lld", num_seqs,
             (long long)capacity_pages, (long long)grid);
    return cuda_status(e);
}

// The workspace of an attention call over a 4-bit cache.  Nothing in it has to
// outlast a call: the direct kernels write what they read, and the counters of
// the BF16 attention over read-back pages are cleared by the read-back.
struct QuantPlan {
    bool direct;
    int64_t pages;                      // not direct: read-back pages,
    int32_t cols;                       // compact table columns,
    size_t v, tables, inner, bytes;     // and offsets (K at 0)
    AttnPlan attn;
};

constexpr int kQuantMaxSeqs = 2048;
constexpr int64_t kQuantMaxPages = int64_t(1) << 28;  // sums of the chunks' weights stay below 2^31
static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

static pa_status plan_quant(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t dh, int32_t max_query_len,
                            int32_t max_seq_len, int64_t max_pages, QuantPlan *pl)
{
    *pl = QuantPlan{};
    if (max_pages < 0)
        return PA_ERR_INVALID_ARG;
    if (!plan_attention(num_seqs, hq, hkv, dh, max_query_len, max_seq_len, &pl->attn))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs > kQuantMaxSeqs || (int64_t)num_seqs * (((int64_t)max_seq_len + 15) / 16) > kQuantMaxPages ||
        (int64_t)num_seqs * 2 * hkv > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    // The direct kernels take up to two tiles of a request's tokens whatever
    // the batch.  Measured against the read-back path: 8 requests of 3345 keys,
    // 40 rows 12 us to 30; 16 of up to 7168 keys with 2 KV heads, 64 rows 46 to
    // 137; 64 of them with 8 KV heads, 64 rows 567 to 613, so twice the rows
    // would lose there: they take more only in small calls.
    const int tiles = quant_attn_tiles(num_seqs, hkv, dh, hq / hkv, max_query_len, max_seq_len);
    pl->direct = tiles > 0;
    if (pl->direct) {
        const int rows = (max_query_len + tiles - 1) / tiles * (hq / hkv);
        pl->bytes = quant_attn_bytes(num_seqs, tiles, hkv, dh, rows, max_seq_len, max_pages);
        return PA_OK;
    }
    // The BF16 attention gives the same bits with the keys split over CTAs or
    // not.  Split, it writes and folds a record per (tile, 256-key chunk), whose
    // cost grows with the rows; measured, read-back included, 7168 keys, 8
    // query and 2 KV heads, split against not: 4 tiles of 128 rows 64 us to 94,
    // 8 tiles of 36 rows 68 to 118, of 68 rows 162 to 118, of 128 rows 547 to
    // 95; 2048 keys, 8 tiles of 68 rows 29 to 44, 16 of 128 rows 42 to 37.
    if (pl->attn.split && (int64_t)num_seqs * hkv * pl->attn.qtiles * pl->attn.nch * pl->attn.ws_rows > 96 * 152)
        plan_attention(num_seqs, hq, hkv, dh, max_query_len, max_seq_len, &pl->attn, false);
    pl->cols = (int32_t)(((int64_t)max_seq_len + 15) / 16);
    if (pl->cols < 1)
        pl->cols = 1;
    pl->pages = (int64_t)num_seqs * pl->cols;
    if (max_pages > 0 && max_pages < pl->pages)
        pl->pages = max_pages;
    const size_t view = (size_t)pl->pages * 16 * hkv * dh * 2;
    pl->v = round256(view);
    pl->tables = pl->v + round256(view);
    pl->inner = pl->tables + round256((size_t)num_seqs * pl->cols * 4);
    pl->bytes = pl->inner + pl->attn.ws_bytes;
    return PA_OK;
}

size_t pa_paged_attention_quant_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t head_dim, int32_t max_query_len, int32_t max_seq_len,
                                               int64_t max_pages)
{
    QuantPlan pl;
    return plan_quant(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len, max_pages, &pl) == PA_OK
               ? pl.bytes
               : 0;
}

pa_status pa_paged_attention_quant(const void *q, int64_t num_q_tokens, int64_t q_tok_stride, int32_t num_q_heads,
                                   const pa_quant_cache *cache, const int32_t *block_tables,
                                   int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *query_start_loc,
                                   int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len, int64_t max_pages,
                                   float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   pa_stream_t stream)
{
    pa_status st = check_quant_cache(cache);
    if (st != PA_OK)
        return st;
    if (num_q_heads <= 0 || num_seqs < 0 || max_query_len < 0 || max_seq_len < 0 || num_q_tokens < 0 ||
        max_blocks_per_seq < 0 || max_pages < 0 || num_q_tokens > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    const int32_t hkv = cache->num_kv_heads, dh = cache->head_dim;
    if (num_q_heads % hkv != 0 || num_q_heads / hkv > 128)
        return PA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || scale == INFINITY)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_q_tokens == 0 || max_query_len == 0) {
        snprintf(g_last_info, sizeof g_last_info, "quant attention: empty batch (nothing launched)");
        return PA_OK;
    }
    const int64_t row = (int64_t)num_q_heads * dh;
    if (!q || !out || !block_tables || !seq_lens || !query_start_loc || !aligned16(q) || !aligned16(out) ||
        !aligned4(lse) || !aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(query_start_loc))
        return PA_ERR_INVALID_ARG;
    if (q_tok_stride < row || (q_tok_stride & 7) || max_blocks_per_seq == 0)
        return PA_ERR_INVALID_ARG;
    QuantPlan pl;
    if ((st = plan_quant(num_seqs, num_q_heads, hkv, dh, max_query_len, max_seq_len, max_pages, &pl)) != PA_OK)
        return st;
    if (!workspace || workspace_bytes < pl.bytes)
        return PA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return PA_ERR_INVALID_ARG;
    {
        const Span reads[6] = {rows_span(Rows{q, q_tok_stride, row}, num_q_tokens),
                               span(cache->k, quant_view_bytes(cache)),
                               span(cache->v, quant_view_bytes(cache)),
                               span(block_tables, (int64_t)num_seqs * max_blocks_per_seq * 4),
                               span(seq_lens, (int64_t)num_seqs * 4),
                               span(query_start_loc, (int64_t)num_seqs * 4 + 4)};
        const Span writes[3] = {span(out, num_q_tokens * row * 2),
                                span(lse, lse ? num_q_tokens * num_q_heads * 4 : 0),
                                span(workspace, (int64_t)pl.bytes)};
        for (int i = 0; i < 3; ++i) {
            for (const Span &r : reads)
                if (overlaps(writes[i], r))
                    return PA_ERR_INVALID_ARG;
            for (int j = i + 1; j < 3; ++j)
                if (overlaps(writes[i], writes[j]))
                    return PA_ERR_INVALID_ARG;
        }
    }
    ErrState *err = nullptr;
    int nsm = 0;
    if ((st = device_setup(&err, &nsm)) != PA_OK)
        return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (pl.direct) {
        QuantAttnArgs a{};
        a.q = q;
        a.num_q_tokens = num_q_tokens;
        a.q_tok_stride = q_tok_stride;
        a.num_q_heads = num_q_heads;
        a.pool = quant_pool(cache);
        a.block_tables = block_tables;
        a.max_blocks = max_blocks_per_seq;
        a.seq_lens = seq_lens;
        a.query_start_loc = query_start_loc;
        a.num_seqs = num_seqs;
        a.max_query_len = max_query_len;
        a.max_seq_len = max_seq_len;
        a.scale = scale;
        a.out = out;
        a.lse = lse;
        a.max_pages = max_pages;
        a.workspace = ws;
        return cuda_status(launch_quant_attention(a, err, s, g_last_info, sizeof g_last_info));
    }
    // read the selected pages back, then the BF16 attention over them
    const int32_t cols = pl.cols < max_blocks_per_seq ? pl.cols : max_blocks_per_seq;
    int32_t *tables = reinterpret_cast<int32_t *>(ws + pl.tables);
    int64_t grid = 0;
    cudaError_t e = launch_dequantize_kv(quant_pool(cache), block_tables, max_blocks_per_seq, seq_lens, num_seqs,
                                         ws, ws + pl.v, pl.pages, tables, cols, nullptr, true, ws + pl.inner,
                                         pl.attn.ws_counter_bytes, err, s, nsm, &grid);
    if (e != cudaSuccess)
        return cuda_status(e);
    AttnArgs a{};
    a.q = q;
    a.num_q_tokens = num_q_tokens;
    a.q_tok_stride = q_tok_stride;
    a.num_q_heads = num_q_heads;
    a.k = ws;
    a.v = ws + pl.v;
    a.num_blocks = pl.pages;
    a.num_kv_heads = hkv;
    a.head_dim = dh;
    a.block_stride = (int64_t)16 * hkv * dh;
    a.token_stride = (int64_t)hkv * dh;
    a.head_stride = dh;
    a.block_tables = tables;
    a.max_blocks_per_seq = cols;
    a.seq_lens = seq_lens;
    a.query_start_loc = query_start_loc;
    a.num_seqs = num_seqs;
    a.max_query_len = max_query_len;
    a.max_seq_len = max_seq_len;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.workspace = ws + pl.inner;
    a.workspace_bytes = workspace_bytes - pl.inner;
    char info[192];
    st = attention_launch(a, pl.attn, err, s, info, sizeof info);
    snprintf(g_last_info, sizeof g_last_info, "quant attention read-back grid=%lld; %.180s", (long long)grid, info);
    return st;
}

// ------------------------------------------------------------ page copies --
// pa_copy_pages and pa_copy_pages_quant after the checks of the caches:
// geometry of a view's page in 16-byte units, first cache's strides for all.
static pa_status copy_call(CopyArgs &a, const int32_t *src_pages, const int32_t *dst_pages, int64_t num_pairs,
                           const Span *views, const char *name, pa_stream_t stream)
{
    if (num_pairs < 0 || num_pairs > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    if (num_pairs == 0 || a.num_caches == 0) {
        snprintf(g_last_info, sizeof g_last_info, "%s pairs=0 (nothing launched)", name);
        return PA_OK;
    }
    if (!src_pages || !dst_pages || !aligned4(src_pages) || !aligned4(dst_pages))
        return PA_ERR_INVALID_ARG;
    for (int i = 0; i < 2 * a.num_caches; ++i)
        if (overlaps(views[i], span(src_pages, num_pairs * 4)) || overlaps(views[i], span(dst_pages, num_pairs * 4)))
            return PA_ERR_INVALID_ARG;
    a.num_pairs = (int32_t)num_pairs;
    a.src = src_pages;
    a.dst = dst_pages;
    ErrState *err = nullptr;
    int nsm = 0;
    const pa_status st = device_setup(&err, &nsm);
    if (st != PA_OK)
        return st;
    int64_t grid = 0;
    const cudaError_t e = launch_copy_pages(a, err, reinterpret_cast<cudaStream_t>(stream), nsm, &grid);
    snprintf(g_last_info, sizeof g_last_info, "%s caches=%d pairs=%lld grid=%lld", name, a.num_caches,
             (long long)num_pairs, (long long)grid);
    return cuda_status(e);
}

pa_status pa_copy_pages(const pa_kv_cache *caches, int32_t num_caches, const int32_t *src_pages,
                        const int32_t *dst_pages, int64_t num_pairs, pa_stream_t stream)
{
    if (num_caches < 0 || (num_caches > 0 && !caches))
        return PA_ERR_INVALID_ARG;
    if (num_caches > kCopyMaxCachesHost)
        return PA_ERR_UNSUPPORTED;
    CopyArgs a{};
    a.num_caches = num_caches;
    Span views[2 * kCopyMaxCachesHost];
    for (int i = 0; i < num_caches; ++i) {
        const pa_kv_cache &c = caches[i], &f = caches[0];
        const pa_status st = check_cache(&c);
        if (st != PA_OK)
            return st;
        if (c.num_blocks != f.num_blocks || c.num_kv_heads != f.num_kv_heads || c.head_dim != f.head_dim ||
            c.block_stride != f.block_stride || c.token_stride != f.token_stride || c.head_stride != f.head_stride)
            return PA_ERR_INVALID_ARG;
        a.k[i] = static_cast<uint4 *>(c.k);
        a.v[i] = static_cast<uint4 *>(c.v);
        views[2 * i] = span(c.k, pool_view_bytes(&c));
        views[2 * i + 1] = span(c.v, pool_view_bytes(&c));
    }
    if (num_caches > 0) {
        const pa_kv_cache &f = caches[0];
        const int64_t dh = f.head_dim, hkv = f.num_kv_heads;
        if (2 * hkv * dh > INT32_MAX / 4)
            return PA_ERR_UNSUPPORTED;
        a.num_blocks = f.num_blocks;
        a.block_stride = f.block_stride / 8;
        a.page_vecs = (int32_t)(2 * hkv * dh);
        // the longest runs of neighbouring bytes; one head has no head stride
        if (hkv == 1 ? f.token_stride == dh : f.head_stride == dh && f.token_stride == hkv * dh) {
            a.run_vecs = a.page_vecs;
        } else if (f.token_stride == dh) {
            a.run_vecs = f.head_stride == 16 * dh ? a.page_vecs : (int32_t)(2 * dh);
            a.c1 = (int32_t)hkv;
            a.s1 = f.head_stride / 8;
        } else if (hkv == 1 || f.head_stride == dh) {
            a.run_vecs = (int32_t)(hkv * dh / 8);
            a.c1 = 16;
            a.s1 = f.token_stride / 8;
        } else {
            a.run_vecs = (int32_t)(dh / 8);
            a.c1 = (int32_t)hkv;
            a.s1 = f.head_stride / 8;
            a.s0 = f.token_stride / 8;
        }
    }
    return copy_call(a, src_pages, dst_pages, num_pairs, views, "copy_pages", stream);
}

pa_status pa_copy_pages_quant(const pa_quant_cache *caches, int32_t num_caches, const int32_t *src_pages,
                              const int32_t *dst_pages, int64_t num_pairs, pa_stream_t stream)
{
    if (num_caches < 0 || (num_caches > 0 && !caches))
        return PA_ERR_INVALID_ARG;
    if (num_caches > kCopyMaxCachesHost)
        return PA_ERR_UNSUPPORTED;
    CopyArgs a{};
    a.num_caches = num_caches;
    Span views[2 * kCopyMaxCachesHost];
    for (int i = 0; i < num_caches; ++i) {
        const pa_quant_cache &c = caches[i], &f = caches[0];
        const pa_status st = check_quant_cache(&c);
        if (st != PA_OK)
            return st;
        if (c.num_blocks != f.num_blocks || c.num_kv_heads != f.num_kv_heads || c.head_dim != f.head_dim ||
            c.block_stride != f.block_stride || c.head_stride != f.head_stride)
            return PA_ERR_INVALID_ARG;
        a.k[i] = static_cast<uint4 *>(c.k);
        a.v[i] = static_cast<uint4 *>(c.v);
        views[2 * i] = span(c.k, quant_view_bytes(&c));
        views[2 * i + 1] = span(c.v, quant_view_bytes(&c));
    }
    if (num_caches > 0) {
        const pa_quant_cache &f = caches[0];
        const int64_t record = 9 * (int64_t)f.head_dim / 16, hkv = f.num_kv_heads;
        if (record * hkv > INT32_MAX / 4)
            return PA_ERR_UNSUPPORTED;
        a.num_blocks = f.num_blocks;
        a.block_stride = f.block_stride / 16;
        a.page_vecs = (int32_t)(record * hkv);
        a.run_vecs = hkv == 1 || f.head_stride == record * 16 ? a.page_vecs : (int32_t)record;
        a.c1 = (int32_t)hkv;
        a.s1 = f.head_stride / 16;
    }
    return copy_call(a, src_pages, dst_pages, num_pairs, views, "copy_pages_quant", stream);
}

// ------------------------------------------------- fork, release, compact --
// Whether a write shares bytes with a read or another write.  same[i] >= 0:
// write i may be read same[i] itself (in place), bytes 0 on.
static bool any_overlap(const Span *writes, const int *same, int nw, const Span *reads, int nr)
{
    for (int i = 0; i < nw; ++i) {
        for (int j = 0; j < nr; ++j)
            if (!(same[i] == j && writes[i].lo == reads[j].lo) && overlaps(writes[i], reads[j]))
                return true;
        for (int j = i + 1; j < nw; ++j)
            if (overlaps(writes[i], writes[j]))
                return true;
    }
    return false;
}

static bool bad_i32(const void *p) { return !p || !aligned4(p); }

static pa_status page_limits(int32_t num_seqs, int32_t max_blocks_per_seq, int64_t num_blocks, int32_t num_free_pages)
{
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || num_blocks > (int64_t)1 << 31 ||
        num_free_pages < 0)
        return PA_ERR_INVALID_ARG;
    // lengths are 32-bit, and so is the number of a table entry
    if (num_seqs > kPageMaxSeqsHost || max_blocks_per_seq > INT32_MAX / 16 ||
        (int64_t)num_seqs * max_blocks_per_seq > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

pa_status pa_fork_requests(const int32_t *parents, const int32_t *children, const int32_t *fork_lens,
                           int32_t num_forks, const int32_t *context_lens, int32_t num_seqs, int32_t *block_tables,
                           int32_t max_blocks_per_seq, const int32_t *shares_in, int32_t *shares_out,
                           int64_t num_blocks, const int32_t *free_pages, int32_t num_free_pages,
                           const int32_t *cursor_in, int32_t *cursor_out, int32_t *seq_lens, int32_t *copy_src,
                           int32_t *copy_dst, pa_stream_t stream)
{
    pa_status st = page_limits(num_seqs, max_blocks_per_seq, num_blocks, num_free_pages);
    if (st != PA_OK)
        return st;
    if (num_forks < 0)
        return PA_ERR_INVALID_ARG;
    if (num_forks > kPageMaxSeqsHost)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) {
        snprintf(g_last_info, sizeof g_last_info, "fork_requests: empty batch (nothing launched)");
        return num_forks == 0 ? PA_OK : PA_ERR_INVALID_ARG;
    }
    if ((num_forks > 0 && (bad_i32(parents) || bad_i32(children) || bad_i32(copy_src) || bad_i32(copy_dst))) ||
        !aligned4(fork_lens) || bad_i32(context_lens) || bad_i32(block_tables) || bad_i32(shares_in) ||
        bad_i32(shares_out) || (num_free_pages > 0 && bad_i32(free_pages)) || bad_i32(cursor_in) ||
        bad_i32(cursor_out) || bad_i32(seq_lens))
        return PA_ERR_INVALID_ARG;
    const int64_t f4 = (int64_t)num_forks * 4, n4 = (int64_t)num_seqs * 4;
    const Span reads[7] = {span(context_lens, n4), span(shares_in, num_blocks * 4), span(cursor_in, 4),
                           span(parents, f4),      span(children, f4),              span(fork_lens, fork_lens ? f4 : 0),
                           span(free_pages, (int64_t)num_free_pages * 4)};
    const Span writes[6] = {span(seq_lens, n4), span(shares_out, num_blocks * 4), span(cursor_out, 4),
                            span(block_tables, n4 * max_blocks_per_seq), span(copy_src, f4), span(copy_dst, f4)};
    const int same[6] = {0, 1, 2, -1, -1, -1};
    if (any_overlap(writes, same, 6, reads, 7))
        return PA_ERR_INVALID_ARG;
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    PageArgs a{};
    a.parents = parents, a.children = children, a.fork_lens = fork_lens, a.num_forks = num_forks;
    a.context_lens = context_lens, a.num_seqs = num_seqs, a.block_tables = block_tables, a.max_blocks = max_blocks_per_seq;
    a.shares_in = shares_in, a.shares_out = shares_out, a.num_blocks = num_blocks;
    a.free_pages = const_cast<int32_t *>(free_pages), a.num_free = num_free_pages;
    a.cursor_in = cursor_in, a.cursor_out = cursor_out, a.seq_lens = seq_lens, a.copy_src = copy_src, a.copy_dst = copy_dst;
    int grid = 0;
    const cudaError_t e = launch_fork_requests(a, err, reinterpret_cast<cudaStream_t>(stream), &grid);
    snprintf(g_last_info, sizeof g_last_info, "fork_requests forks=%d seqs=%d grid=%d", num_forks, num_seqs, grid);
    return cuda_status(e);
}

pa_status pa_release_pages(const int32_t *context_lens, const int32_t *keep_lens, int32_t num_seqs,
                           const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *shares_in,
                           int32_t *shares_out, int64_t num_blocks, int32_t *free_pages, int32_t num_free_pages,
                           const int32_t *cursor_in, int32_t *cursor_out, int32_t *seq_lens, pa_stream_t stream)
{
    pa_status st = page_limits(num_seqs, max_blocks_per_seq, num_blocks, num_free_pages);
    if (st != PA_OK)
        return st;
    if (num_seqs == 0) {
        snprintf(g_last_info, sizeof g_last_info, "release_pages: empty batch (nothing launched)");
        return PA_OK;
    }
    if (bad_i32(context_lens) || bad_i32(keep_lens) || bad_i32(block_tables) || bad_i32(shares_in) ||
        bad_i32(shares_out) || (num_free_pages > 0 && bad_i32(free_pages)) || bad_i32(cursor_in) ||
        bad_i32(cursor_out) || bad_i32(seq_lens))
        return PA_ERR_INVALID_ARG;
    const int64_t n4 = (int64_t)num_seqs * 4;
    const Span reads[5] = {span(context_lens, n4), span(shares_in, num_blocks * 4), span(cursor_in, 4),
                           span(keep_lens, n4), span(block_tables, n4 * max_blocks_per_seq)};
    const Span writes[4] = {span(seq_lens, n4), span(shares_out, num_blocks * 4), span(cursor_out, 4),
                            span(free_pages, (int64_t)num_free_pages * 4)};
    const int same[4] = {0, 1, 2, -1};
    if (any_overlap(writes, same, 4, reads, 5))
        return PA_ERR_INVALID_ARG;
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    PageArgs a{};
    a.context_lens = context_lens, a.keep_lens = keep_lens, a.num_seqs = num_seqs;
    a.block_tables = const_cast<int32_t *>(block_tables), a.max_blocks = max_blocks_per_seq;
    a.shares_in = shares_in, a.shares_out = shares_out, a.num_blocks = num_blocks;
    a.free_pages = free_pages, a.num_free = num_free_pages, a.cursor_in = cursor_in, a.cursor_out = cursor_out;
    a.seq_lens = seq_lens;
    int grid = 0;
    const cudaError_t e = launch_release_pages(a, err, reinterpret_cast<cudaStream_t>(stream), &grid);
    snprintf(g_last_info, sizeof g_last_info, "release_pages seqs=%d grid=%d", num_seqs, grid);
    return cuda_status(e);
}

size_t pa_compact_pages_workspace_size(int64_t num_blocks)
{
    return num_blocks <= 0 || num_blocks > kPageMaxBlocksHost ? 0 : round256(((size_t)num_blocks + 31) / 32 * 4);
}

pa_status pa_compact_pages(const int32_t *context_lens, int32_t num_seqs, const int32_t *block_tables,
                           int32_t *tables_out, int32_t max_blocks_per_seq, const int32_t *shares_in,
                           int32_t *shares_out, int64_t num_blocks, int32_t *free_pages, int32_t num_free_pages,
                           const int32_t *cursor_in, int32_t *cursor_out, int32_t *copy_src, int32_t *copy_dst,
                           int32_t max_moves, int32_t *counts, void *workspace, size_t workspace_bytes,
                           pa_stream_t stream)
{
    pa_status st = page_limits(num_seqs, max_blocks_per_seq, num_blocks, num_free_pages);
    if (st != PA_OK)
        return st;
    if (max_moves < 0 || (int64_t)num_free_pages < num_blocks)
        return PA_ERR_INVALID_ARG;
    if (num_blocks > kPageMaxBlocksHost)
        return PA_ERR_UNSUPPORTED;
    if ((num_seqs > 0 && (bad_i32(context_lens) || bad_i32(block_tables) || bad_i32(tables_out))) || bad_i32(shares_in) ||
        bad_i32(shares_out) || bad_i32(free_pages) || bad_i32(cursor_in) || bad_i32(cursor_out) ||
        (max_moves > 0 && (bad_i32(copy_src) || bad_i32(copy_dst))) || bad_i32(counts))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa_compact_pages_workspace_size(num_blocks);
    if (!workspace || workspace_bytes < need)
        return PA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return PA_ERR_INVALID_ARG;
    const int64_t n4 = (int64_t)num_seqs * 4, m4 = (int64_t)max_moves * 4, t4 = n4 * max_blocks_per_seq;
    const Span reads[4] = {span(block_tables, t4), span(shares_in, num_blocks * 4), span(cursor_in, 4),
                           span(context_lens, n4)};
    const Span writes[8] = {span(tables_out, t4), span(shares_out, num_blocks * 4), span(cursor_out, 4),
                            span(free_pages, (int64_t)num_free_pages * 4), span(copy_src, m4), span(copy_dst, m4),
                            span(counts, 8), span(workspace, (int64_t)need)};
    const int same[8] = {0, 1, 2, -1, -1, -1, -1, -1};
    if (any_overlap(writes, same, 8, reads, 4))
        return PA_ERR_INVALID_ARG;
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    PageArgs a{};
    a.context_lens = context_lens, a.num_seqs = num_seqs, a.block_tables = const_cast<int32_t *>(block_tables);
    a.tables_out = tables_out, a.max_blocks = max_blocks_per_seq;
    a.shares_in = shares_in, a.shares_out = shares_out, a.num_blocks = num_blocks;
    a.free_pages = free_pages, a.num_free = num_free_pages, a.cursor_in = cursor_in, a.cursor_out = cursor_out;
    a.copy_src = copy_src, a.copy_dst = copy_dst, a.max_moves = max_moves, a.counts = counts;
    a.bitmap = static_cast<uint32_t *>(workspace);
    int grid = 0;
    const cudaError_t e = launch_compact_pages(a, err, reinterpret_cast<cudaStream_t>(stream), &grid);
    snprintf(g_last_info, sizeof g_last_info, "compact_pages seqs=%d blocks=%lld grid=%d", num_seqs, (long long)num_blocks,
             grid);
    return cuda_status(e);
}

// -------------------------------------------------------- scored attention --
constexpr int kScoredMaxSeqs = 8192;

static bool scored_sizes_ok(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t dh, int32_t max_query_len,
                            int32_t max_seq_len, int64_t num_q_tokens)
{
    return num_seqs > 0 && num_seqs <= kScoredMaxSeqs && hkv > 0 && hq > 0 && hq % hkv == 0 && hq / hkv <= 128 &&
           (dh == 128 || dh == 256 || dh == 512) && max_query_len > 0 && max_seq_len >= 0 &&
           max_seq_len <= INT32_MAX - 4096 && (int64_t)num_seqs * max_query_len * hq <= INT32_MAX &&
           scored_supported(num_seqs, hq, hkv, dh, max_query_len, max_seq_len, num_q_tokens);
}

size_t pa_paged_attention_scored_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                int32_t head_dim, int32_t max_query_len, int32_t max_seq_len)
{
    if (!scored_sizes_ok(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len, -1))
        return 0;
    return scored_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len);
}

pa_status pa_paged_attention_scored(const void *q, int64_t num_q_tokens, int64_t q_tok_stride, int32_t num_q_heads,
                                    const pa_kv_cache *cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    const int32_t *seq_lens, const int32_t *query_start_loc, int32_t num_seqs,
                                    int32_t max_query_len, int32_t max_seq_len, float scale,
                                    const pa_score_rules *rules, void *out, float *lse, void *workspace,
                                    size_t workspace_bytes, pa_stream_t stream)
{
    pa_status st = check_cache(cache);
    if (st != PA_OK)
        return st;
    if (num_q_heads <= 0 || num_seqs < 0 || max_query_len < 0 || max_seq_len < 0 || num_q_tokens < 0 ||
        max_blocks_per_seq < 0 || num_q_tokens > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    const int32_t hkv = cache->num_kv_heads, dh = cache->head_dim;
    if (num_q_heads % hkv != 0 || num_q_heads / hkv > 128)
        return PA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || scale == INFINITY)
        return PA_ERR_INVALID_ARG;
    const pa_score_rules none{};
    const pa_score_rules &r = rules ? *rules : none;
    if (!(r.soft_cap == 0.f || (r.soft_cap >= 0x1p-20f && r.soft_cap <= 0x1p20f)) || r.window < 0 ||
        !aligned4(r.slopes) || !aligned4(r.prefix_lens) || !aligned4(r.first_keys))
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale * 4.f) || (r.soft_cap > 0.f && !std::isfinite(4.f * scale / r.soft_cap)))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_q_tokens == 0 || max_query_len == 0) {
        snprintf(g_last_info, sizeof g_last_info, "scored attention: empty batch (nothing launched)");
        return PA_OK;
    }
    const int64_t row = (int64_t)num_q_heads * dh;
    if (!q || !out || !aligned16(q) || !aligned16(out) || !aligned4(lse) || bad_i32(block_tables) || bad_i32(seq_lens) ||
        bad_i32(query_start_loc))
        return PA_ERR_INVALID_ARG;
    if (q_tok_stride < row || (q_tok_stride & 7) || max_blocks_per_seq == 0)
        return PA_ERR_INVALID_ARG;
    if (!scored_sizes_ok(num_seqs, num_q_heads, hkv, dh, max_query_len, max_seq_len, num_q_tokens))
        return PA_ERR_UNSUPPORTED;
    const size_t need = scored_workspace_bytes(num_seqs, num_q_heads, hkv, dh, max_query_len, max_seq_len);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return PA_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return PA_ERR_INVALID_ARG;
    }
    const int64_t n4 = (int64_t)num_seqs * 4;
    const Span reads[9] = {rows_span(Rows{q, q_tok_stride, row}, num_q_tokens),
                           span(cache->k, pool_view_bytes(cache)),
                           span(cache->v, pool_view_bytes(cache)),
                           span(block_tables, n4 * max_blocks_per_seq),
                           span(seq_lens, n4),
                           span(query_start_loc, n4 + 4),
                           span(r.slopes, r.slopes ? (int64_t)num_q_heads * 4 : 0),
                           span(r.prefix_lens, r.prefix_lens ? n4 : 0),
                           span(r.first_keys, r.first_keys ? num_q_tokens * 4 : 0)};
    const Span writes[3] = {span(out, num_q_tokens * row * 2), span(lse, lse ? num_q_tokens * num_q_heads * 4 : 0),
                            span(workspace, (int64_t)need)};
    const int same[3] = {-1, -1, -1};
    if (any_overlap(writes, same, 3, reads, 9))
        return PA_ERR_INVALID_ARG;
    ErrState *err = nullptr;
    if ((st = device_setup(&err)) != PA_OK)
        return st;
    AttnArgs a{};
    a.q = q;
    a.num_q_tokens = num_q_tokens;
    a.q_tok_stride = q_tok_stride;
    a.num_q_heads = num_q_heads;
    a.k = cache->k;
    a.v = cache->v;
    a.num_blocks = cache->num_blocks;
    a.num_kv_heads = hkv;
    a.head_dim = dh;
    a.block_stride = cache->block_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.block_tables = block_tables;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.seq_lens = seq_lens;
    a.query_start_loc = query_start_loc;
    a.num_seqs = num_seqs;
    a.max_query_len = max_query_len;
    a.max_seq_len = max_seq_len;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    const ScoreRules sr{r.soft_cap, r.window, r.slopes, r.prefix_lens, r.first_keys};
    return cuda_status(launch_scored_attention(a, sr, err, reinterpret_cast<cudaStream_t>(stream), g_last_info,
                                               sizeof g_last_info));
}

}  // extern "C"

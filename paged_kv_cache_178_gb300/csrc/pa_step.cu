// The step's preparation around the cache write: metadata built from request
// lengths (pa_build_step_metadata), and the norm and rotation of queries and
// keys (pa_qk_norm_rope, with or without the cache write).
#include <cuda_bf16.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_scan.cuh"

namespace pa {

// ------------------------------------------------------- step metadata ----
// Two exclusive sums over the requests (new tokens, new pages), then one
// binary search per token and per new page.  A few KB are read and 12 bytes
// per token written: launch and latency bound, so one kernel does all of it.
// Every CTA repeats the sums (from L2) rather than passing them on through
// memory.  The inputs may be the outputs (lengths and cursor advance in
// place), so nothing is written before every CTA has read them: the grid is
// one cluster, and a cluster barrier stands between.
constexpr int kMetaThreads = 1024;
constexpr int kMetaClusterMax = 8;  // the portable cluster size

__global__ void __launch_bounds__(kMetaThreads, 1) step_metadata_kernel(StepMetaArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int32_t s_meta[];
    __shared__ long long s_sums[kMetaThreads / 32];
    int32_t *s_tok = s_meta;                    // [n + 1] first token of a request
    int32_t *s_page = s_tok + a.num_seqs + 1;   // [n + 1] first new page
    int32_t *s_ctx = s_page + a.num_seqs + 1;   // [n] cached tokens (0: bad)
    const int tid = threadIdx.x, n = a.num_seqs;
    const int64_t gtid = (int64_t)blockIdx.x * kMetaThreads + tid, gsize = (int64_t)gridDim.x * kMetaThreads;
    const int64_t limit = (int64_t)a.max_blocks * 16;
    auto tokens_of = [&](int b, int &ctx) -> int {
        const int c = a.context_lens[b], q = a.query_lens[b];
        const bool c_ok = c >= 0 && (int64_t)c <= limit;
        ctx = c_ok ? c : 0;
        if (c_ok && q >= 0 && (int64_t)c + q <= limit)
            return q;
        if (blockIdx.x == 0)
            record_error(err, kErrBadMetadata, b);
        return 0;
    };
    const int cursor = a.cursor_in ? *a.cursor_in : 0;
    // s_ctx is filled by the first sum and read by the second from the same
    // thread (both give request b to thread b % kMetaThreads)
    const long long tokens = block_exclusive_sums<kMetaThreads>(n, s_tok, s_sums, [&](int b) {
        int ctx;
        const int q = tokens_of(b, ctx);
        s_ctx[b] = ctx;
        s_page[b] = q;
        return q;
    });
    const long long pages = block_exclusive_sums<kMetaThreads>(n, s_page, s_sums, [&](int b) {
        const int64_t c = s_ctx[b], q = s_page[b];
        return (c + q + 15) / 16 - (c + 15) / 16;
    });
    const bool bad_cursor = cursor < 0 || cursor > a.num_free;
    const bool short_pages = !bad_cursor && pages > (long long)a.num_free - cursor;
    const bool empty = bad_cursor || short_pages || tokens > a.num_tokens;
    if (gridDim.x > 1)
        cluster_sync_all();  // every CTA has read the inputs
    if (gtid == 0) {
        if (short_pages)
            record_error(err, kErrBudget, pages);
        else if (empty)
            record_error(err, kErrBadMetadata, n);
        *a.cursor_out = empty ? cursor : cursor + (int)pages;
    }
    for (int64_t b = gtid; b <= n; b += gsize) {
        a.query_start_loc[b] = empty ? 0 : s_tok[b];
        if (b < n)
            a.seq_lens[b] = s_ctx[b] + (empty ? 0 : s_tok[b + 1] - s_tok[b]);
    }
    auto id_ok = [&](int id) { return id >= 0 && (int64_t)id < a.num_blocks; };
    if (!empty) {
        for (int64_t x = gtid; x < pages; x += gsize) {
            const int b = owner_of(s_page, n, (int)x);
            const int col = (s_ctx[b] + 15) / 16 + (int)x - s_page[b];
            a.block_tables[(int64_t)b * a.max_blocks + col] = a.free_pages[cursor + x];
        }
    }
    for (int64_t t = gtid; t < a.num_tokens; t += gsize) {
        int64_t slot = -1;
        int pos = -1;
        if (!empty && t < tokens) {
            const int b = owner_of(s_tok, n, (int)t);
            const int ctx = s_ctx[b], have = (ctx + 15) / 16;
            pos = ctx + (int)t - s_tok[b];
            // a new page's id comes from the free list: its table entry may
            // be written by another thread just now
            const int p = pos / 16;
            const int id = p < have ? a.block_tables[(int64_t)b * a.max_blocks + p]
                                    : a.free_pages[cursor + s_page[b] + p - have];
            if (id_ok(id))
                slot = (int64_t)id * 16 + pos % 16;
            else
                record_error(err, kErrBadMetadata, b);
        }
        a.slot_mapping[t] = slot;
        a.positions[t] = pos;
    }
}

static size_t meta_smem(int num_seqs) { return (size_t)(3 * num_seqs + 2) * 4; }

cudaError_t launch_step_metadata(const StepMetaArgs &a, ErrState *err, cudaStream_t stream, int *grid)
{
    // One CTA until a second one would have work (about one item per thread);
    // eight of them write 12 bytes a token at about 8 x 64 bytes a clock.
    const int64_t items = a.num_tokens + a.num_seqs;
    int ctas = 1;
    while (ctas < kMetaClusterMax && (int64_t)ctas * kMetaThreads < items)
        ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kMetaThreads);
    cfg.dynamicSmemBytes = meta_smem(a.num_seqs);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *grid = ctas;
    return cudaLaunchKernelEx(&cfg, step_metadata_kernel, a, err);
}

// ------------------------------------------- norm, rotation, cache write --
// Memory bound: each row is read once and written once (plus the token's
// cos/sin row, shared by all its heads through L1).  A row of DH elements is
// DH/8 vectors of 16 bytes; a group of DH/16 lanes owns it, two vectors a
// lane.  With pairs (i, i + rot/2) lane j < rot/16 takes vectors j and
// j + rot/16, whose elements are each other's partners; with pairs
// (2i, 2i+1) any two vectors do.  So the rotation needs no exchange between
// lanes, and the norm one butterfly over the group.
constexpr int kRopeThreads = 256;

template <int DH>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = DH / 32; o >= 1; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
}

// Sum of squares of a lane's sixteen elements, in a fixed order.
__device__ __forceinline__ float sum_squares(const float (&a)[8], const float (&b)[8])
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s = __fmaf_rn(a[i], a[i], s);
        s = __fmaf_rn(b[i], b[i], s);
    }
    return s;
}

template <int DH, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int LANES = DH / 16;  // lanes of a row
    const int lane = threadIdx.x % LANES;
    const int hk = a.num_kv_heads, hq = a.num_q_heads;
    const int rows_tok = hq + hk * (a.k_cache ? 2 : 1);
    const int64_t rows = a.num_tokens * rows_tok;
    const int64_t step = (int64_t)gridDim.x * (kRopeThreads / LANES);
    // vectors of this lane, and the pairs of the first one
    const int rv = a.rot_dim / 16;  // vectors of half the rotated part
    const bool turned = lane < rv;
    const int v0 = turned ? (INTERLEAVED ? 2 * lane : lane) : 2 * lane;
    const int v1 = turned && !INTERLEAVED ? lane + rv : v0 + 1;
    // Every lane of a warp runs the same number of passes (the butterflies
    // name all 32); a group past the last row works on row 0 and stores
    // nothing.
    const int64_t first = (int64_t)blockIdx.x * (kRopeThreads / LANES) + threadIdx.x / LANES;
    const int64_t warp_first = (int64_t)blockIdx.x * (kRopeThreads / LANES) + (threadIdx.x & ~31) / LANES;
    for (int64_t r0 = warp_first, row = first; r0 < rows; r0 += step, row += step) {
        const bool live = row < rows;
        const int64_t t = !live ? 0 : rows <= 0xffffffffll ? (int64_t)((uint32_t)row / (uint32_t)rows_tok) : row / rows_tok;
        const int h = live ? (int)(row - t * rows_tok) : 0;
        const int kind = h < hq ? 0 : (h < hq + hk ? 1 : 2);  // q, k, v
        const int head = kind == 0 ? h : (kind == 1 ? h - hq : h - hq - hk);
        const uint4 *src = (kind == 0   ? a.q + t * a.q_stride
                            : kind == 1 ? a.k + t * a.k_stride
                                        : a.v + t * a.v_stride) +
                           (int64_t)head * (DH / 8);
        uint4 x0 = src[v0], x1 = src[v1];
        const int pos = __ldg(a.positions + t);
        int64_t slot = -1;
        if (kind != 0 && a.k_cache)
            slot = __ldg(a.slot_mapping + t);
        const bool bad_pos = (int64_t)pos >= a.max_positions;
        const uint4 *wv = kind == 0 ? a.q_weight : (kind == 1 ? a.k_weight : nullptr);
        float p[8], q[8];
        unpack8(x0, p);
        unpack8(x1, q);
        // the whole warp takes part in the sums, whatever its rows are
        float ss = group_sum<DH>(sum_squares(p, q));
        float eps = a.eps;
        const bool large = !(ss < 1e36f), tiny = ss < 1e-30f && eps < 1e-20f;
        if (__any_sync(0xffffffffu, wv && (large || tiny))) {
            // squares past fp32's range: the row times a power of two, eps
            // times its square (the norm cancels it)
            const float g = !wv ? 1.f : (large ? 0x1p-96f : (!tiny ? 1.f : (eps < 1e-38f ? 0x1p96f : 0x1p64f)));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] *= g;
                q[i] *= g;
            }
            ss = group_sum<DH>(sum_squares(p, q));
            eps = eps * g * g;
        }
        if (kind != 2) {
            if (wv) {
                const float r = __frsqrt_rn(ss * (1.f / DH) + eps);
                float w0[8], w1[8];
                unpack8(__ldg(wv + v0), w0);
                unpack8(__ldg(wv + v1), w1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = p[i] * r * (w0[i] + a.weight_offset);
                    q[i] = q[i] * r * (w1[i] + a.weight_offset);
                }
            }
            if (turned && pos >= 0 && !bad_pos) {
                // the angles of this lane's eight pairs
                const float4 *c = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim + 8 * lane);
                const float4 *s = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim +
                                                                   a.rot_dim / 2 + 8 * lane);
                const float4 ca = __ldg(c), cb = __ldg(c + 1), sa = __ldg(s), sb = __ldg(s + 1);
                const float co[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
                const float si[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
                if (INTERLEAVED) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = p[2 * i], v = p[2 * i + 1], m = q[2 * i], o = q[2 * i + 1];
                        p[2 * i] = __fmaf_rn(u, co[i], -(v * si[i]));
                        p[2 * i + 1] = __fmaf_rn(v, co[i], u * si[i]);
                        q[2 * i] = __fmaf_rn(m, co[4 + i], -(o * si[4 + i]));
                        q[2 * i + 1] = __fmaf_rn(o, co[4 + i], m * si[4 + i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float u = p[i], v = q[i];
                        p[i] = __fmaf_rn(u, co[i], -(v * si[i]));
                        q[i] = __fmaf_rn(v, co[i], u * si[i]);
                    }
                }
            }
            x0 = pack8(p);
            x1 = pack8(q);
            if (bad_pos) {
                x0 = x1 = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
                if (live && lane == 0)
                    record_error(err, kErrBadMetadata, t);
            }
        }
        if (!live || pos < 0)
            continue;
        uint4 *dst = nullptr;
        if (kind == 0) {
            dst = a.q_out + t * a.q_out_stride + (int64_t)head * (DH / 8);
        } else if (!a.k_cache) {
            dst = a.k_out + t * a.k_out_stride + (int64_t)head * (DH / 8);
        } else if (slot >= a.num_slots) {
            if (lane == 0 && head == 0 && kind == 1)
                record_error(err, kErrBadMetadata, t);
        } else if (slot >= 0 && !bad_pos) {
            dst = (kind == 1 ? a.k_cache : a.v_cache) + (slot >> 4) * a.block_stride + (slot & 15) * a.token_stride +
                  (int64_t)head * a.head_stride;
        }
        if (dst) {
            dst[v0] = x0;
            dst[v1] = x1;
        }
    }
}

cudaError_t launch_qk_norm_rope(const RopeArgs &a, ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid)
{
    const int64_t rows = a.num_tokens * (a.num_q_heads + a.num_kv_heads * (a.k_cache ? 2 : 1));
    const int per_cta = kRopeThreads / (a.head_dim / 16);
    int64_t blocks = (rows + per_cta - 1) / per_cta;
    // four waves of the eight CTAs that fit an SM
    if (blocks > (int64_t)num_sms * 32)
        blocks = (int64_t)num_sms * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *grid = blocks;
    void (*kern)(const RopeArgs, ErrState *) =
        a.head_dim == 128   ? (a.interleaved ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>)
        : a.head_dim == 256 ? (a.interleaved ? qk_norm_rope_kernel<256, true> : qk_norm_rope_kernel<256, false>)
                            : (a.interleaved ? qk_norm_rope_kernel<512, true> : qk_norm_rope_kernel<512, false>);
    return cudaLaunchKernelEx(&cfg, kern, a, err);
}

cudaError_t init_step_attributes()
{
    return cudaFuncSetAttribute(step_metadata_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)meta_smem(kScanMaxSeqs));
}

}  // namespace pa

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
// per token written: launch and latency bound, so one kernel does all of it,
// with the two sums in one pass and four tokens a thread in flight.  Every CTA
// repeats the sums (from L2) rather than passing them on through memory.
// Where lengths or cursor advance in place, nothing may be written before
// every CTA has read them: the grid is then one cluster with a barrier of its
// own in between (up to eight CTAs); otherwise it takes as many CTAs as there
// is work.
constexpr int kMetaThreads = 256;
constexpr int kMetaClusterMax = 8;  // the portable cluster size
constexpr int kMetaUnroll = 4;

__global__ void __launch_bounds__(kMetaThreads) step_metadata_kernel(StepMetaArgs a, bool in_place, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int32_t s_meta[];
    __shared__ longlong2 s_sums[kMetaThreads / 32];
    int32_t *s_tok = s_meta;                   // [n + 1] first token of a request
    int32_t *s_page = s_tok + a.num_seqs + 1;  // [n + 1] first new page
    int32_t *s_ctx = s_page + a.num_seqs + 1;  // [n] cached tokens (0: bad)
    const int tid = threadIdx.x, n = a.num_seqs;
    const int gtid = blockIdx.x * kMetaThreads + tid, gsize = gridDim.x * kMetaThreads;
    const int64_t limit = (int64_t)a.max_blocks * 16;
    const int cursor = a.cursor_in ? *a.cursor_in : 0;
    longlong2 total;
    block_exclusive_sums2<kMetaThreads>(n, s_tok, s_page, s_sums, total, [&](int b, int &tokens, int &pages) {
        const int c = a.context_lens[b], q = a.query_lens[b];
        const bool c_ok = c >= 0 && (int64_t)c <= limit;
        const int ctx = c_ok ? c : 0;
        s_ctx[b] = ctx;
        if (c_ok && q >= 0 && (int64_t)c + q <= limit) {
            tokens = q;
            pages = (int)(((int64_t)ctx + q + 15) / 16) - (ctx + 15) / 16;  // limit is below 2^31
        } else if (blockIdx.x == 0) {
            record_error(err, kErrBadMetadata, b);
        }
    });
    const long long tokens = total.x, pages = total.y;
    const bool bad_cursor = cursor < 0 || cursor > a.num_free;
    const bool short_pages = !bad_cursor && pages > (long long)a.num_free - cursor;
    const bool empty = bad_cursor || short_pages || tokens > a.num_tokens;
    if (in_place && gridDim.x > 1)
        cluster_sync_all();  // every CTA has read the inputs
    if (gtid == 0) {
        if (short_pages)
            record_error(err, kErrBudget, pages);
        else if (empty)
            record_error(err, kErrBadMetadata, n);
        *a.cursor_out = empty ? cursor : cursor + (int)pages;
    }
    for (int b = gtid; b <= n; b += gsize) {
        a.query_start_loc[b] = empty ? 0 : s_tok[b];
        if (b < n)
            a.seq_lens[b] = s_ctx[b] + (empty ? 0 : s_tok[b + 1] - s_tok[b]);
    }
    const int np = empty ? 0 : (int)pages, nt = empty ? 0 : (int)tokens;
    for (int64_t x0 = gtid; x0 < np; x0 += gsize) {
        const int x = (int)x0, b = owner_of(s_page, n, x);
        const int col = (s_ctx[b] + 15) / 16 + x - s_page[b];
        a.block_tables[(int64_t)b * a.max_blocks + col] = a.free_pages[cursor + x];
    }
    for (int64_t t0 = gtid; t0 < a.num_tokens; t0 += (int64_t)kMetaUnroll * gsize) {
        int pos[kMetaUnroll], id[kMetaUnroll], req[kMetaUnroll];
#pragma unroll
        for (int u = 0; u < kMetaUnroll; ++u) {
            const int64_t t = t0 + (int64_t)u * gsize;
            pos[u] = -1;
            id[u] = req[u] = 0;
            if (t < nt) {
                const int b = owner_of(s_tok, n, (int)t), ctx = s_ctx[b], have = (ctx + 15) / 16;
                req[u] = b;
                pos[u] = ctx + (int)t - s_tok[b];
                // a new page's id comes from the free list: its table entry
                // may be written by another thread just now
                const int p = pos[u] / 16;
                id[u] = p < have ? a.block_tables[(int64_t)b * a.max_blocks + p]
                                 : a.free_pages[cursor + s_page[b] + p - have];
            }
        }
#pragma unroll
        for (int u = 0; u < kMetaUnroll; ++u) {
            const int64_t t = t0 + (int64_t)u * gsize;
            if (t >= a.num_tokens)
                break;
            int64_t slot = -1;
            if (pos[u] >= 0) {
                if (id[u] >= 0 && (int64_t)id[u] < a.num_blocks)
                    slot = (int64_t)id[u] * 16 + pos[u] % 16;
                else
                    record_error(err, kErrBadMetadata, req[u]);
            }
            a.slot_mapping[t] = slot;
            a.positions[t] = pos[u];
        }
    }
}

static size_t meta_smem(int num_seqs) { return (size_t)(3 * num_seqs + 2) * 4; }

cudaError_t launch_step_metadata(const StepMetaArgs &a, ErrState *err, cudaStream_t stream, int num_sms, int *grid)
{
    const bool in_place = a.seq_lens == a.context_lens || a.cursor_out == a.cursor_in;
    const int64_t items = a.num_tokens + a.num_seqs;
    const int64_t want = (items + kMetaThreads * kMetaUnroll - 1) / (kMetaThreads * kMetaUnroll);
    const int64_t most = in_place ? kMetaClusterMax : num_sms;
    int ctas = (int)(want < 1 ? 1 : (want < most ? want : most));
    if (in_place)
        while (ctas & (ctas - 1))
            ++ctas;  // a cluster size: a power of two
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kMetaThreads);
    cfg.dynamicSmemBytes = meta_smem(a.num_seqs);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = in_place ? (unsigned)ctas : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *grid = ctas;
    return cudaLaunchKernelEx(&cfg, step_metadata_kernel, a, in_place, err);
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
constexpr int kRopeBatch = 4;  // rows in flight

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

// A warp takes one token and a part of its rows, neighbouring groups
// neighbouring rows, so that its loads and stores are contiguous; a group's
// rows_per_task rows go one after another: the angles stay in registers, the
// weights until the kind of row changes, and the loads of several rows are in
// flight together.
template <int DH, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int LANES = DH / 16;  // lanes of a row
    constexpr int VEC = DH / 8;     // vectors of a row
    const int lane = threadIdx.x % LANES;
    const int hk = a.num_kv_heads, hq = a.num_q_heads;
    const int rows_tok = hq + hk * (a.k_cache ? 2 : 1);
    const int per = a.rows_per_task;
    constexpr int GPW = 32 / LANES;  // groups of a warp
    const uint32_t parts = (uint32_t)(rows_tok + GPW * per - 1) / (uint32_t)(GPW * per);
    // vectors of this lane, and the pairs of the first one
    const int rv = a.rot_dim / 16;  // vectors of half the rotated part
    const bool turned = lane < rv;
    const int v0 = turned && !INTERLEAVED ? lane : 2 * lane;
    const int v1 = turned && !INTERLEAVED ? lane + rv : v0 + 1;
    // Every lane of a warp runs the same passes (the butterflies name all
    // 32); a group without a row computes on zeros and stores nothing.
    const int64_t tasks = a.num_tokens * parts, step = (int64_t)gridDim.x * (kRopeThreads / 32);
    const int group = (threadIdx.x & 31) / LANES;
    for (int64_t task = (int64_t)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32; task < tasks; task += step) {
        const int64_t t = tasks <= 0xffffffffll ? (int64_t)((uint32_t)task / parts) : task / parts;
        // the group's rows: h0, h0 + GPW, ..
        const int part0 = (int)(task - t * parts) * GPW * per, h0 = part0 + group;
        const int nrows = h0 < rows_tok ? min(per, (rows_tok - h0 + GPW - 1) / GPW) : 0;
        const int pos = __ldg(a.positions + t);
        const bool bad_pos = (int64_t)pos >= a.max_positions;
        const int64_t slot = a.k_cache ? __ldg(a.slot_mapping + t) : 0;
        const bool store = nrows > 0 && pos >= 0;
        const bool slot_bad = a.k_cache && slot >= a.num_slots;
        const bool cached = slot >= 0 && !slot_bad && !bad_pos;
        if (pos >= 0 && (threadIdx.x & 31) == 0 && part0 == 0 && (bad_pos || slot_bad))
            record_error(err, kErrBadMetadata, t);
        float co[8], si[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            co[i] = 1.f;
            si[i] = 0.f;
        }
        if (turned && store && !bad_pos) {
            // the angles of this lane's eight pairs
            const float4 *c = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim + 8 * lane);
            const float4 *s = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim + a.rot_dim / 2 + 8 * lane);
            const float4 ca = __ldg(c), cb = __ldg(c + 1), sa = __ldg(s), sb = __ldg(s + 1);
            co[0] = ca.x, co[1] = ca.y, co[2] = ca.z, co[3] = ca.w, co[4] = cb.x, co[5] = cb.y, co[6] = cb.z, co[7] = cb.w;
            si[0] = sa.x, si[1] = sa.y, si[2] = sa.z, si[3] = sa.w, si[4] = sb.x, si[5] = sb.y, si[6] = sb.z, si[7] = sb.w;
        }
        auto source = [&](int h) {
            return h < hq        ? a.q + t * a.q_stride + (int64_t)h * VEC
                   : h < hq + hk ? a.k + t * a.k_stride + (int64_t)(h - hq) * VEC
                                 : a.v + t * a.v_stride + (int64_t)(h - hq - hk) * VEC;
        };
        const uint4 *w_now = nullptr;  // whose weights w0, w1 hold
        float w0[8], w1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w0[i] = w1[i] = 1.f;
        for (int r0 = 0; r0 < per; r0 += kRopeBatch) {
        uint4 x0[kRopeBatch], x1[kRopeBatch];
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
            x0[u] = x1[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r0 + u < nrows) {
                const uint4 *src = source(h0 + GPW * (r0 + u));
                x0[u] = src[v0];
                x1[u] = src[v1];
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
            if (r0 + u >= per)
                break;
            const int h = h0 + GPW * (r0 + u);
            const bool on = r0 + u < nrows;
            float p[8], q[8];
            unpack8(x0[u], p);
            unpack8(x1[u], q);
            uint4 y0 = x0[u], y1 = x1[u];
            const uint4 *wv = !on || h >= hq + hk ? nullptr : (h < hq ? a.q_weight : a.k_weight);
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
            if (on && h < hq + hk) {
                if (wv) {
                    if (wv != w_now) {
                        w_now = wv;
                        unpack8(__ldg(wv + v0), w0);
                        unpack8(__ldg(wv + v1), w1);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            w0[i] += a.weight_offset;
                            w1[i] += a.weight_offset;
                        }
                    }
                    const float rs = __frsqrt_rn(ss * (1.f / DH) + eps);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p[i] = p[i] * rs * w0[i];
                        q[i] = q[i] * rs * w1[i];
                    }
                }
                if (turned) {
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
                y0 = pack8(p);
                y1 = pack8(q);
                if (bad_pos)
                    y0 = y1 = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
            }
            if (!on || !store)
                continue;
            uint4 *dst = nullptr;
            if (h < hq)
                dst = a.q_out + t * a.q_out_stride + (int64_t)h * VEC;
            else if (!a.k_cache)
                dst = a.k_out + t * a.k_out_stride + (int64_t)(h - hq) * VEC;
            else if (cached)
                dst = (h < hq + hk ? a.k_cache : a.v_cache) + (slot >> 4) * a.block_stride + (slot & 15) * a.token_stride +
                      (int64_t)(h < hq + hk ? h - hq : h - hq - hk) * a.head_stride;
            if (dst) {
                dst[v0] = y0;
                dst[v1] = y1;
            }
        }
        }
    }
}

cudaError_t launch_qk_norm_rope(const RopeArgs &args, ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid)
{
    RopeArgs a = args;
    const int rows_tok = a.num_q_heads + a.num_kv_heads * (a.k_cache ? 2 : 1);
    const int gpw = 512 / a.head_dim;  // groups of a warp
    // Rows of a group: one while that leaves warps idle, more (their shared
    // loads then count once) as long as 24 warps per SM have some.
    const int64_t steps = (rows_tok + gpw - 1) / gpw;  // rows of a group that had the whole token
    int64_t per = a.num_tokens * steps / ((int64_t)num_sms * 24);
    per = per < 1 ? 1 : (per > 16 ? 16 : per);
    if (per > steps)
        per = steps;
    const int64_t parts = (steps + per - 1) / per;
    a.rows_per_task = (int)((steps + parts - 1) / parts);  // parts of about one size
    const int64_t tasks = a.num_tokens * ((steps + a.rows_per_task - 1) / a.rows_per_task);
    int64_t blocks = (tasks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (blocks > (int64_t)num_sms * 64)
        blocks = (int64_t)num_sms * 64;
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

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
// is work.  In a CUDA graph 64 decoding requests take 2.6 us, 240 requests with
// 62 thousand tokens 4.2 us (with the sums one after the other and a token a
// thread, 5.2 and 12); issued one by one 2.8 and 4.4, of which the host's part
// is most.
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
constexpr int kRopeCtas = 4;   // per SM
constexpr int kRopeBatch = 2;  // steps loaded together

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

// A warp takes one token and a part of its steps: a step is 32*16/DH
// neighbouring rows of q, of k or of v, a row to a group, so that loads and
// stores are contiguous.  The angles stay in registers, the weights (offset
// added) in shared memory, the rows' addresses advance by one addition, and
// kRopeBatch steps are loaded before the first is computed.  A step of 1 KB
// takes about 130 instructions.  Times in a CUDA graph: 16384 tokens of 32
// query and 8 KV heads at head dim 128, with the cache write (411 MB): 69 us,
// 6.0 TB/s, bound by the memory; 4099 tokens of 16 and 2 heads of 256 elements,
// 64 of them rotated (77 MB): 16.4 us, 4.7 TB/s, bound by latency (half of the
// issue slots and 28% of the DRAM's rate: less than one wave of CTAs, two steps
// in flight, the position and then its angles before the first store); 64 tokens
// 2.6 us.
// Loads and stores are marked as streaming (neither: 70.5 and 17.4 us; the
// loads alone 71.8 and 17.6): every row passes once.  The
// first case took 88 us with 16-byte vectors that were not neighbours in a
// load, 81 to 90 with the rows staged through shared memory, 106 with a token to
// each group of lanes.
template <int DH, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) qk_norm_rope_kernel(const RopeArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int LANES = DH / 16;   // lanes of a row
    constexpr int VEC = DH / 8;      // vectors of a row
    constexpr int GPW = 32 / LANES;  // groups of a warp: rows of a step
    __shared__ __align__(16) float s_w[2 * DH];  // weights of q and k, offset added
    const int wl = threadIdx.x & 31, lane = threadIdx.x % LANES, group = wl / LANES;
    const int hk = a.num_kv_heads, hq = a.num_q_heads;
    // steps of a token: of q, of k, of v
    const int jq = (hq + GPW - 1) / GPW, jk = (hk + GPW - 1) / GPW, jall = jq + jk + (a.k_cache ? jk : 0);
    const int per = a.steps_per_task;
    const uint32_t parts = (uint32_t)(jall + per - 1) / (uint32_t)per;
    // Vectors of this lane: neighbouring lanes have neighbouring ones in both
    // loads.  With pairs (i, i + rot/2) lanes below rv hold partners.
    const int rv = a.rot_dim / 16;  // vectors of half the rotated part
    const int v0 = INTERLEAVED || lane < rv ? lane : lane + rv;
    const int v1 = INTERLEAVED || lane >= rv ? lane + LANES : lane + rv;
    const bool turned = INTERLEAVED ? lane < 2 * rv : lane < rv;
    for (int i = threadIdx.x; i < 2 * DH; i += kRopeThreads) {
        const __nv_bfloat16 *w = reinterpret_cast<const __nv_bfloat16 *>(i < DH ? a.q_weight : a.k_weight);
        s_w[i] = w ? __bfloat162float(w[i % DH]) + a.weight_offset : 1.f;
    }
    __syncthreads();
    const int64_t tasks = a.num_tokens * parts;
    auto token_of = [&](int64_t task) {
        return tasks <= 0xffffffffll ? (int64_t)((uint32_t)task / parts) : task / parts;
    };
    // positions and slots are loaded a task ahead; a task's first rows before
    // anything waits for its position
    int64_t task = (int64_t)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;
    const int64_t step = (int64_t)gridDim.x * (kRopeThreads / 32);
    int64_t t_next = task < tasks ? token_of(task) : 0;
    int pos_next = 0;
    int64_t slot_next = 0;
    auto load_next = [&]() {
        pos_next = __ldg(a.positions + t_next);
        slot_next = a.k_cache ? __ldg(a.slot_mapping + t_next) : 0;
    };
    if (task < tasks)
        load_next();
    for (; task < tasks; task += step) {
        const int64_t t = t_next, slot = slot_next;
        const int pos = pos_next, part = (int)(task - t * parts), j0 = part * per, j1 = min(j0 + per, jall);
        if (task + step < tasks) {
            t_next = token_of(task + step);
            load_next();
        }
        const bool bad_pos = (int64_t)pos >= a.max_positions;
        const bool slot_bad = a.k_cache && slot >= a.num_slots;
        if (pos >= 0 && wl == 0 && part == 0 && (bad_pos || slot_bad))
            record_error(err, kErrBadMetadata, t);
        float co[8], si[8];
        bool have_angles = false;
        auto load_angles = [&]() {
            if (have_angles)
                return;
            have_angles = true;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                co[i] = 1.f;  // (for rows without an angle: not stored, or NaN)
                si[i] = 0.f;
            }
            if (turned && pos >= 0 && !bad_pos) {
                // the angles of this lane's eight pairs (interleaved: four of
                // v0, and of v1 where that is rotated)
                const float4 *c = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim);
                const int i0 = INTERLEAVED ? v0 : 2 * lane, i1 = INTERLEAVED ? v1 : 2 * lane + 1, sin0 = 2 * rv;
                const bool both = !INTERLEAVED || v1 < 2 * rv;
                const float4 ca = __ldg(c + i0), sa = __ldg(c + sin0 + i0);
                const float4 cb = both ? __ldg(c + i1) : make_float4(1.f, 1.f, 1.f, 1.f);
                const float4 sb = both ? __ldg(c + sin0 + i1) : make_float4(0.f, 0.f, 0.f, 0.f);
                co[0] = ca.x, co[1] = ca.y, co[2] = ca.z, co[3] = ca.w, co[4] = cb.x, co[5] = cb.y, co[6] = cb.z, co[7] = cb.w;
                si[0] = sa.x, si[1] = sa.y, si[2] = sa.z, si[3] = sa.w, si[4] = sb.x, si[5] = sb.y, si[6] = sb.z, si[7] = sb.w;
            }
        };
        // One row: norm and rotation.  The whole warp takes part in the sums.
        auto row = [&](uint4 &x0, uint4 &x1, bool norm, const float4 *w) {
            float p[8], q[8];
            unpack8(x0, p);
            unpack8(x1, q);
            if (norm) {
                float ss = group_sum<DH>(sum_squares(p, q)), eps = a.eps;
                const bool large = !(ss < 1e36f), tiny = ss < 1e-30f && eps < 1e-20f;
                if (__any_sync(0xffffffffu, large || tiny)) {
                    // squares past fp32's range: the row times a power of two,
                    // eps times its square (the norm cancels it)
                    const float g = large ? 0x1p-96f : (!tiny ? 1.f : (eps < 1e-38f ? 0x1p96f : 0x1p64f));
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p[i] *= g;
                        q[i] *= g;
                    }
                    ss = group_sum<DH>(sum_squares(p, q));
                    eps = eps * g * g;
                }
                const float rs = rsqrtf(ss * (1.f / DH) + eps);
                const float4 wa = w[2 * v0], wb = w[2 * v0 + 1], wc = w[2 * v1], wd = w[2 * v1 + 1];
                const float w0[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
                const float w1[8] = {wc.x, wc.y, wc.z, wc.w, wd.x, wd.y, wd.z, wd.w};
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
                        const float u = p[2 * i], v = p[2 * i + 1];
                        p[2 * i] = __fmaf_rn(u, co[i], -(v * si[i]));
                        p[2 * i + 1] = __fmaf_rn(v, co[i], u * si[i]);
                    }
                    // (cos 1 and sin 0 would not do: infinities, NaN and -0
                    // of unrotated elements would change their neighbours)
                    if (v1 < 2 * rv)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float m = q[2 * i], o = q[2 * i + 1];
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
            if (bad_pos)
                x0 = x1 = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        };
        // steps [ja, jb) of one kind: src, dst of its first row; dst null: not stored
        auto run = [&](int ja, int jb, int heads, const uint4 *src, uint4 *dst, int64_t dst_row, bool compute, bool norm,
                       const float4 *w) {
            int h = ja * GPW + group;
            src += (int64_t)h * VEC;
            dst += h * dst_row;
            const int64_t dst_step = GPW * dst_row;
            for (int j = ja; j < jb; j += kRopeBatch) {
                uint4 x0[kRopeBatch], x1[kRopeBatch];
#pragma unroll
                for (int u = 0; u < kRopeBatch; ++u) {
                    x0[u] = x1[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (j + u < jb && h + u * GPW < heads) {
                        x0[u] = __ldcs(src + u * GPW * VEC + v0);
                        x1[u] = __ldcs(src + u * GPW * VEC + v1);
                    }
                }
                if (compute)
                    load_angles();
#pragma unroll
                for (int u = 0; u < kRopeBatch; ++u) {
                    if (j + u >= jb)
                        break;
                    if (compute)
                        row(x0[u], x1[u], norm, w);
                    if (h + u * GPW < heads && pos >= 0) {
                        __stcs(dst + v0, x0[u]);
                        __stcs(dst + v1, x1[u]);
                    }
                    dst += dst_step;
                }
                src += kRopeBatch * GPW * VEC;
                h += kRopeBatch * GPW;
            }
        };
        if (j0 < jq)
            run(j0, min(j1, jq), hq, a.q + t * a.q_stride, a.q_out + t * a.q_out_stride, VEC, true, a.q_weight != nullptr,
                reinterpret_cast<const float4 *>(s_w));
        const int64_t at = a.k_cache ? (slot >> 4) * a.block_stride + (slot & 15) * a.token_stride : 0;
        const bool cached = pos >= 0 && slot >= 0 && !slot_bad && !bad_pos;
        if (j1 > jq && j0 < jq + jk && (cached || !a.k_cache))
            run(max(j0 - jq, 0), min(j1 - jq, jk), hk, a.k + t * a.k_stride,
                a.k_cache ? a.k_cache + at : a.k_out + t * a.k_out_stride, a.k_cache ? a.head_stride : VEC, true,
                a.k_weight != nullptr, reinterpret_cast<const float4 *>(s_w + DH));
        if (j1 > jq + jk && cached)
            run(max(j0 - jq - jk, 0), j1 - jq - jk, hk, a.v + t * a.v_stride, a.v_cache + at, a.head_stride, false, false,
                nullptr);
    }
}

cudaError_t launch_qk_norm_rope(const RopeArgs &args, ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid)
{
    RopeArgs a = args;
    const int gpw = 512 / a.head_dim;  // rows of a step
    const int64_t jk = (a.num_kv_heads + gpw - 1) / gpw;
    const int64_t steps = (a.num_q_heads + gpw - 1) / gpw + jk * (a.k_cache ? 2 : 1);
    // Steps of a warp: one while that leaves warps idle, more (the token's
    // angles and addresses then count once) as long as 16 warps per SM have some.
    int64_t per = a.num_tokens * steps / ((int64_t)num_sms * 16);
    per = per < 1 ? 1 : (per > steps ? steps : per);
    const int64_t parts = (steps + per - 1) / per;
    a.steps_per_task = (int)((steps + parts - 1) / parts);  // parts of about one size
    const int64_t tasks = a.num_tokens * ((steps + a.steps_per_task - 1) / a.steps_per_task);
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

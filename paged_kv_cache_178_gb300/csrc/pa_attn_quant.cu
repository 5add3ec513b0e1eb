// Attention of few query rows over a 4-bit cache (pa_quant_common.cuh): decode
// steps and drafted tokens.  S = Q.K^T, P = softmax(S), O = P.V with K and V
// dequantised on the way into the matrix instructions.
//
// What bounds it: a 16-token page of one KV head at head dim 128 is 2304
// bytes (K and V), 98 clocks of an SM's share of the memory bandwidth.  Its
// 4096 elements need 2048 conversions (two elements each) and as many scale
// products; both issue at two warp instructions per clock and SM, about 64
// clocks together with the regrouping of V.  Passing dequantised tiles
// through shared memory (as operands of tcgen05) would add 16 KB of writes and
// 16 KB of operand reads per page, 256 clocks at 128 bytes per clock; so the
// fragments of mma.sync are built in registers, straight from the codes, and
// nothing dequantised is ever stored.
//
// The keys (then the head-dim elements) are the M = 16 dimension of
// mma.m16n8k16 and the query rows its N = 8: one page is one M tile, and up to
// eight rows cost one instruction.  Everything is f16 with fp32 accumulation:
// codes times scales are exact there; q is scaled per row by a power of two
// to [1, 2) at its largest element (elements below 2^-14 of it lose bits, at
// most 2^-25 of the largest); p is scaled by 2^15 (11 bits down to
// 2^-29 of the row's largest probability).
//
// Fixed arithmetic (a row's results do not depend on the batch or the grid):
//   tiles of 128 keys from key 0, one page per warp; the running maximum is
//   exact per tile; chunks of 256 keys start fresh; a chunk's row sum is, per
//   warp, a butterfly over the keys, then the eight warps' sums pairwise;
//   chunk states fold left to right (fold_coef, fold_elem).
//
// A CTA (8 warps): per tile, warp w scores page w, the warps exchange row
// maxima (barrier), write P to shared memory in fragment order (barrier), and
// warp w multiplies P by head-dim elements 16w..16w+15 (of each 128) of all
// pages: O needs no exchange between warps.  Each warp's lane 0 copies page w
// of the tiles ahead (cp.async.bulk, one mbarrier per tile).  The chunks of
// all (request, KV head) groups are dealt out as equal contiguous ranges; a
// group inside one range is folded in registers, the chunks of a group cut by
// a range end become records, folded by the last CTA to arrive.
#include <cstdio>

#include "pa_attn_common.cuh"
#include "pa_quant_common.cuh"
#include "pa_scan.cuh"
#include "pa_split.cuh"

namespace pa {

namespace qa {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kTile = 128;   // keys per tile: one page per warp
constexpr int kChunk = 256;  // keys per chunk
constexpr int kTilesPerChunk = kChunk / kTile;
constexpr int kPagesPerChunk = kChunk / 16;
constexpr float kShift = 15.f;  // p is scaled by 2^kShift (largest f16: 2^16)

template <int DH>
constexpr int stages() { return DH == 512 ? 2 : 3; }
template <int DH>
constexpr int stage_bytes() { return 2 * kWarps * quant_record_bytes(DH); }
// CTAs per SM that registers (256 threads) and shared memory are sized for
template <int DH, int NT>
constexpr int ctas_per_sm()
{
    return DH == 128 ? (NT == 1 ? 3 : NT <= 4 ? 2 : 1) : (DH == 256 && NT <= 2 ? 2 : 1);
}

// Shared-memory layout in bytes.
template <int DH, int NT>
struct Layout {
    static constexpr int R = 8 * NT;
    static constexpr int q = stages<DH>() * stage_bytes<DH>();
    static constexpr int p = q + NT * DH * 16;
    static constexpr int max = p + kWarps * NT * 256;
    static constexpr int sum = max + R * kWarps * 4;
    static constexpr int cq = sum + R * kWarps * 4;
    static constexpr int bars = cq + R * 4;
    static constexpr int bad = bars + 8 * 4;
    static constexpr int flags = bad + 8 * 4;
    static constexpr int sums = flags + 16;
    static constexpr int pre = sums + kWarps * 8;  // [num_seqs + 1] int32
    static_assert(stages<DH>() <= 4 && q % 16 == 0 && bars % 8 == 0 && sums % 8 == 0, "layout");
    static_assert(pre + (kScanMaxSeqs + 1) * 4 <= (int)kMaxSmemPerBlock, "shared memory");
    static size_t bytes(int num_seqs) { return (size_t)pre + 4 * ((size_t)num_seqs + 1); }
};

struct Params {
    const uint8_t *k, *v;
    int64_t block_stride, head_stride, num_blocks;
    const __nv_bfloat16 *q;
    int64_t q_tok_stride, num_q_tokens;
    const int32_t *block_tables, *seq_lens, *qsl;
    int32_t max_blocks, num_seqs, hq, hkv, group, max_query_len, max_seq_len;
    int32_t rows;     // rows of a record
    int64_t nch;      // records of a group
    float score_scale;  // scale * log2(e) * k_scale
    float v_scale;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *counters;
    float *records;
    ErrState *err;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
                 "%4;" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar), "l"(policy)
                 : "memory");
}

struct Meta {
    int qs, qn, L;
    bool sane, ok;  // as ReqMeta
};

__device__ __forceinline__ Meta meta_of(const Params &p, int b)
{
    Meta m;
    const int qs = __ldg(p.qsl + b), qe = __ldg(p.qsl + b + 1);
    m.L = __ldg(p.seq_lens + b);
    m.qs = qs;
    m.sane = qs >= 0 && qe >= qs && (int64_t)qe <= p.num_q_tokens;
    m.qn = m.sane ? qe - qs : 0;
    m.ok = m.sane && m.L >= m.qn && (int64_t)m.L <= (int64_t)p.max_blocks * 16 && m.qn <= p.max_query_len &&
           m.L <= p.max_seq_len;
    return m;
}

// A chunk of the dealt sequence: chunk lc of group (b, kvh), request-major.
struct Chunk {
    int b, kvh, lc, nch;
    int qs, qn, L;

    __device__ __forceinline__ void load(const Params &p, const int32_t *pre)
    {
        const Meta m = meta_of(p, b);
        qs = m.qs;
        qn = m.qn;
        L = m.L;
        nch = pre[b + 1] - pre[b];
    }
    __device__ __forceinline__ void at(const Params &p, const int32_t *pre, int64_t x)
    {
        b = owner_of(pre, p.num_seqs, (int)(x / p.hkv));
        load(p, pre);
        const int r = (int)(x - (int64_t)p.hkv * pre[b]);
        kvh = r / nch;
        lc = r % nch;
    }
    // the chunk after this one (there is one)
    __device__ __forceinline__ void next(const Params &p, const int32_t *pre)
    {
        if (++lc < nch)
            return;
        lc = 0;
        if (++kvh < p.hkv)
            return;
        kvh = 0;
        do
            ++b;
        while (pre[b + 1] == pre[b]);
        load(p, pre);
    }
    __device__ __forceinline__ int tiles() const
    {
        return min(kTilesPerChunk, (L - lc * kChunk + kTile - 1) / kTile);
    }
    // block id of the chunk's page `lane` (lanes 0..15; 0 where there is none)
    __device__ __forceinline__ int id(const Params &p, int lane) const
    {
        const int pg = lc * kPagesPerChunk + lane;
        return lane < kPagesPerChunk && pg < (L + 15) / 16 ? __ldg(p.block_tables + (int64_t)b * p.max_blocks + pg) : 0;
    }
};

// Left-to-right fold of a group's records by the whole CTA, and its output.
template <int DH>
__device__ __forceinline__ void merge_group(const Params &p, const float *rec0, int nch, int rv, int64_t tok, int kvh)
{
    const int64_t hdr = part_header_floats(p.rows), stride = part_record_floats(p.rows, DH);
    for (int e = threadIdx.x; e < rv * (DH / 4); e += kThreads) {
        const int n = e / (DH / 4), d = e % (DH / 4) * 4;
        const float *base = rec0 + n;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < nch; c0 += 4) {
            float mc[4], lc[4];
            float4 oc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = min(c0 + i, nch - 1);
                mc[i] = __ldcg(base + c * stride);
                lc[i] = __ldcg(base + c * stride + p.rows);
                oc[i] = __ldcg(reinterpret_cast<const float4 *>(rec0 + c * stride + hdr + (int64_t)n * DH + d));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c0 + i < nch) {
                    const Fold f = fold_coef(m, l, mc[i], lc[i]);
                    m = f.m;
                    l = f.l;
                    o.x = fold_elem(o.x, oc[i].x, f);
                    o.y = fold_elem(o.y, oc[i].y, f);
                    o.z = fold_elem(o.z, oc[i].z, f);
                    o.w = fold_elem(o.w, oc[i].w, f);
                }
            }
        }
        const int64_t row = (tok + n / p.group) * p.hq + kvh * p.group + n % p.group;
        const float r = __frcp_rn(l) * p.v_scale;
        *reinterpret_cast<uint2 *>(p.out + row * DH + d) =
            make_uint2(pack_bf16x2(o.x * r, o.y * r), pack_bf16x2(o.z * r, o.w * r));
        if (d == 0 && p.lse)
            p.lse[row] = lse_of(m, l * 0x1p-15f);
    }
}

template <int DH, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<DH, NT>()) quant_attn_kernel(const Params p)
{
    using Lay = Layout<DH, NT>;
    constexpr int R = 8 * NT;            // query rows
    constexpr int NB = DH / 128;         // 128-element blocks of the head dim
    constexpr int NST = stages<DH>();
    constexpr int REC = quant_record_bytes(DH), CODES = quant_code_bytes(DH);
    constexpr bool kQRegs = NT * DH <= 256;  // Q fragments in registers (else read from shared memory)
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const s_stage = smem;
    uint2 *const s_q = reinterpret_cast<uint2 *>(smem + Lay::q);   // [NT][DH/16][32]
    uint2 *const s_p = reinterpret_cast<uint2 *>(smem + Lay::p);   // [8 pages][NT][32]
    float *const s_max = reinterpret_cast<float *>(smem + Lay::max);  // [R][8 warps]
    float *const s_sum = reinterpret_cast<float *>(smem + Lay::sum);  // [R][8 warps]
    float *const s_cq = reinterpret_cast<float *>(smem + Lay::cq);    // [R] raw score -> log2 units
    uint64_t *const s_bars = reinterpret_cast<uint64_t *>(smem + Lay::bars);
    uint8_t *const s_bad = smem + Lay::bad;                           // [stage][8 warps]
    volatile int *const s_flags = reinterpret_cast<int *>(smem + Lay::flags);  // [0] abort [1] fold
    int32_t *const s_pre = reinterpret_cast<int32_t *>(smem + Lay::pre);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int G = p.group, hkv = p.hkv;

    // the work: chunks of the valid requests
    if (tid == 0) {
        for (int i = 0; i < NST; ++i)
            mbar_init(smem_addr(s_bars + i), kWarps);
        s_flags[0] = 0;
        fence_barrier_init();
    }
    const long long tot = block_exclusive_sums<kThreads>(
        p.num_seqs, s_pre, reinterpret_cast<long long *>(smem + Lay::sums), [&](int b) {
            const Meta m = meta_of(p, b);
            if (!m.ok && blockIdx.x == 0)
                record_error(p.err, kErrBadMetadata, b);
            return m.ok && m.qn > 0 ? (m.L + kChunk - 1) / kChunk : 0;
        });
    for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x) {
        if (s_pre[b + 1] != s_pre[b])
            continue;
        const Meta m = meta_of(p, b);
        if (m.sane && !m.ok) {  // bad lengths: NaN rows
            const int64_t first = (int64_t)m.qs * p.hq, n = (int64_t)m.qn * p.hq;
            for (int64_t i = tid; i < n * DH; i += kThreads)
                p.out[first * DH + i] = __ushort_as_bfloat16(0x7FC0);
            if (p.lse)
                for (int64_t i = tid; i < n; i += kThreads)
                    p.lse[first + i] = __int_as_float(0x7FC00000);
        }
    }
    const int64_t T = tot * hkv;
    const int64_t ctas = T < (int64_t)gridDim.x ? T : (int64_t)gridDim.x;
    if ((int64_t)blockIdx.x >= ctas)
        return;
    const int64_t lo = blockIdx.x * T / ctas, hi = (blockIdx.x + 1) * T / ctas;
    auto cta_of = [&](int64_t x) { return (int)(((x + 1) * ctas + T - 1) / T - 1); };

    // producer state: every warp copies its page of each tile
    const uint64_t policy = l2_policy_evict_first();
    Chunk pc;
    pc.at(p, s_pre, lo);
    int64_t px = lo;      // the chunk being issued
    int ptile = 0;        // its next tile
    int issued = 0;       // tiles issued so far
    int ids = pc.id(p, lane);
    auto issue = [&]() {
        if (px >= hi)
            return;
        const int in_chunk = ptile * kWarps + warp;
        const int id = __shfl_sync(0xffffffffu, ids, in_chunk);
        const bool exists = pc.lc * kPagesPerChunk + in_chunk < (pc.L + 15) / 16;
        const int st = issued % NST;
        if (lane == 0) {
            const uint32_t bar = smem_addr(s_bars + st);
            const bool bad = exists && (id < 0 || (int64_t)id >= p.num_blocks);
            s_bad[st * 8 + warp] = bad;
            if (bad)
                record_error(p.err, kErrBadMetadata, pc.b);
            if (exists && !bad) {
                const int64_t off = (int64_t)id * p.block_stride + pc.kvh * p.head_stride;
                const uint32_t dst = smem_addr(s_stage + st * stage_bytes<DH>() + warp * REC);
                mbar_arrive_expect_tx(bar, 2 * REC);
                bulk_copy(dst, p.k + off, REC, bar, policy);
                bulk_copy(dst + kWarps * REC, p.v + off, REC, bar, policy);
            } else {
                mbar_arrive(bar);
            }
        }
        ++issued;
        if (++ptile >= pc.tiles()) {
            ptile = 0;
            if (++px < hi) {
                pc.next(p, s_pre);
                ids = pc.id(p, lane);
            }
        }
    };
    for (int i = 0; i < NST; ++i)
        issue();

    Chunk c;
    c.at(p, s_pre, lo);
    int tile_no = 0;
    uint2 qf[kQRegs ? NT * (DH / 16) : 1];
    float cq[2 * NT];
    int lim[2 * NT];  // last key of the row
    // rows 8nt + 2t, +1 of this thread: folded state of a whole group
    float acc_m[2 * NT], acc_l[2 * NT], acc_o[NB][NT][4];
    bool whole = false;
    int64_t seg_first = 0;
    for (int64_t x = lo; x < hi; ++x) {
        if (x > lo)
            c.next(p, s_pre);
        const int64_t gs = x - c.lc;  // the group's first chunk
        if (x == lo || c.lc == 0) {
            // a new group: its rows, scaled to [1, 2) by a power of two, in
            // fragment order (the previous group's readers are past a barrier)
            seg_first = x;
            whole = gs >= lo && gs + c.nch <= hi;
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                const int r = 8 * k + warp;
                const bool valid = r < c.qn * G;
                const uint2 *src = reinterpret_cast<const uint2 *>(p.q + (int64_t)(c.qs + (valid ? r / G : 0)) * p.q_tok_stride +
                                                                   (int64_t)(c.kvh * G + (valid ? r % G : 0)) * DH);
                uint2 w[NB];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    w[i] = valid ? __ldg(src + 32 * i + lane) : make_uint2(0u, 0u);
                    top = max(top, max(max(w[i].x & 0x7fffu, (w[i].x >> 16) & 0x7fffu),
                                       max(w[i].y & 0x7fffu, (w[i].y >> 16) & 0x7fffu)));
                }
                top = __reduce_max_sync(0xffffffffu, top);
                int e = (int)(top >> 7) - 127;
                e = top == 0 || top >= 0x7F80u ? 0 : max(-100, min(126, e));
                const float f = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const float a0 = __uint_as_float(w[i].x << 16) * f, a1 = __uint_as_float(w[i].x & 0xffff0000u) * f;
                    const float a2 = __uint_as_float(w[i].y << 16) * f, a3 = __uint_as_float(w[i].y & 0xffff0000u) * f;
                    // lane holds elements 4*lane..+3 of block i: thread lane/8, step lane%8
                    s_q[(k * (DH / 16) + 8 * i + lane % 8) * 32 + warp * 4 + lane / 8] =
                        make_uint2(pack_f16x2(a0, a1), pack_f16x2(a2, a3));
                }
                if (lane == 0)
                    s_cq[r] = p.score_scale * __int_as_float((127 + e) << 23);
            }
            __syncthreads();
            if constexpr (kQRegs) {
#pragma unroll
                for (int i = 0; i < NT * (DH / 16); ++i)
                    qf[i] = s_q[i * 32 + lane];
            }
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const int r = 8 * (i / 2) + 2 * t + i % 2;
                cq[i] = s_cq[r];
                lim[i] = c.L - c.qn + min(r / G, c.qn - 1);
                acc_m[i] = -INFINITY;
                acc_l[i] = 0.f;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc_o[b][n][i] = 0.f;
        }

        // ------------------------------------------------------ one chunk --
        float m[2 * NT], l[2 * NT], o[NB][NT][4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[b][n][i] = 0.f;
        const int tiles = c.tiles();
        for (int tile = 0; tile < tiles; ++tile, ++tile_no) {
            const int st = tile_no % NST;
            const int key0 = c.lc * kChunk + tile * kTile;
            const int npages = min(kWarps, (c.L - key0 + 15) / 16);
            const bool masked = key0 + kTile > c.L - c.qn + 1;  // some row does not see some key
            wait_bar(smem_addr(s_bars + st), (tile_no / NST) & 1, s_flags, p.err, st);
            const uint8_t *stage = s_stage + st * stage_bytes<DH>();

            // S = K . Q^T of page `warp`: rows are keys, columns query rows
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[n][i] = 0.f;
            const int r0 = 4 * (g >> 1) + (g & 1);  // token of fragment row g; row g + 8 is token r0 + 2
            if (warp < npages) {
                const uint8_t *kr = stage + warp * REC + r0 * (DH / 2) + 16 * t;
                const uint8_t *ks = stage + warp * REC + CODES + r0 * (DH / 16) + 2 * t;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint4 ka = *reinterpret_cast<const uint4 *>(kr + 64 * b);
                    const uint4 kb = *reinterpret_cast<const uint4 *>(kr + DH + 64 * b);
                    const uint32_t sa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(ks + 8 * b));
                    const uint32_t sb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(ks + DH / 8 + 8 * b));
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // words 0, 1 are the thread's first 16 elements, 2, 3 the next
                        const uint32_t fa = __byte_perm(sa, 0u, i < 2 ? 0x1010 : 0x3232);
                        const uint32_t fb = __byte_perm(sb, 0u, i < 2 ? 0x1010 : 0x3232);
                        uint32_t a[4], bb[4];
                        e2m1x8_to_f16x2(wa[i], a);
                        e2m1x8_to_f16x2(wb[i], bb);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[j] = mul_f16x2(a[j], fa);
                            bb[j] = mul_f16x2(bb[j], fb);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int step = n * (DH / 16) + 8 * b + 2 * i + j;
                                const uint2 q = kQRegs ? qf[kQRegs ? step : 0] : s_q[step * 32 + lane];
                                mma_f16(s[n], a[2 * j], bb[2 * j], a[2 * j + 1], bb[2 * j + 1], q.x, q.y);
                            }
                    }
                }
            }
            // raw scores to log2 units; keys a row does not see are left out
            const int key = key0 + 16 * warp + r0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[n][i] = s[n][i] * cq[2 * n + i % 2];
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key + (i < 2 ? 0 : 2) > lim[2 * n + i % 2])
                            s[n][i] = -INFINITY;
                }
                float x0 = fmaxf(s[n][0], s[n][2]), x1 = fmaxf(s[n][1], s[n][3]);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
                }
                if (g == 0) {
                    s_max[(8 * n + 2 * t) * kWarps + warp] = x0;
                    s_max[(8 * n + 2 * t + 1) * kWarps + warp] = x1;
                }
            }
            __syncthreads();  // A: maxima written; the previous tile is consumed
            if (s_flags[0]) {
                // a wait ran out of time: let the copies in flight land, give up
                for (int k = tile_no; k < issued; ++k)
                    wait_bar_drain(smem_addr(s_bars + k % NST), (k / NST) & 1);
                return;
            }
            if (tile_no > 0)
                issue();
            bad |= *reinterpret_cast<const uint64_t *>(s_bad + 8 * st) != 0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p4[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 u = *reinterpret_cast<const float4 *>(s_max + (8 * n + 2 * t + i) * kWarps);
                    const float4 v = *reinterpret_cast<const float4 *>(s_max + (8 * n + 2 * t + i) * kWarps + 4);
                    const float mx = fmaxf(fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)), fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
                    const float mo = m[2 * n + i], mn = fmaxf(mo, mx);
                    const float f = mo == mn ? 1.f : ex2(mo - mn);
                    m[2 * n + i] = mn;
                    l[2 * n + i] *= f;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        o[b][n][i] *= f;
                        o[b][n][2 + i] *= f;
                    }
                    const float ref = (mn == -INFINITY ? 0.f : mn) - kShift;
                    p4[i] = ex2(s[n][i] - ref);  // 0 for keys left out
                    p4[2 + i] = ex2(s[n][2 + i] - ref);
                    l[2 * n + i] += p4[i] + p4[2 + i];
                }
                // P^T fragment of the second product: keys in pairs
                s_p[(warp * NT + n) * 32 + lane] =
                    make_uint2(movmatrix(pack_f16x2(p4[0], p4[1])), movmatrix(pack_f16x2(p4[2], p4[3])));
            }
            __syncthreads();  // B: P written

            // O^T += V^T . P^T: rows are head-dim elements 16*(warp + 8b)..+15
            int nan_key[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
                nan_key[b] = 0x7fffffff;
            const uint8_t *vr = stage + kWarps * REC + (warp * 8 + g) * 16 + 4 * t;
            const uint8_t *vs = stage + kWarps * REC + CODES + warp * 16 + 4 * t;
#pragma unroll 2
            for (int j = 0; j < npages; ++j) {
                uint2 pf[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    pf[n] = s_p[(j * NT + n) * 32 + lane];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(vr + j * REC + b * 1024);
                    const uint32_t sw = *reinterpret_cast<const uint32_t *>(vs + j * REC + b * 128);
                    uint32_t s01 = e4m3x2_to_f16x2(sw), s23 = e4m3x2_to_f16x2(sw >> 16);
                    if (masked) {
                        // tokens no row sees count as zero whatever their
                        // bytes; a NaN that only some rows see is added to
                        // those rows below
                        const int k0 = key0 + 16 * j + 4 * t;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool gone = k0 + i >= c.L;
                            const bool nan = ((sw >> (8 * i)) & 0x7fu) == 0x7fu;
                            if (gone || (nan && k0 + i > c.L - c.qn)) {
                                uint32_t &sp = i < 2 ? s01 : s23;
                                sp &= i % 2 ? 0x0000ffffu : 0xffff0000u;
                                if (!gone)
                                    nan_key[b] = min(nan_key[b], k0 + i);
                            }
                        }
                    }
                    uint32_t e[4];
                    e2m1x8_to_f16x2(w, e);  // token 4t + i: elements 2g (low), 2g + 1
                    const uint32_t a0 = mul_f16x2(__byte_perm(e[0], e[1], 0x5410), s01);
                    const uint32_t a1 = mul_f16x2(__byte_perm(e[0], e[1], 0x7632), s01);
                    const uint32_t a2 = mul_f16x2(__byte_perm(e[2], e[3], 0x5410), s23);
                    const uint32_t a3 = mul_f16x2(__byte_perm(e[2], e[3], 0x7632), s23);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(o[b][n], a0, a1, a2, a3, pf[n].x, pf[n].y);
                }
            }
            if (masked) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int k = __reduce_min_sync(0xffffffffu, nan_key[b]);
                    if (k != 0x7fffffff) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (lim[2 * n + i % 2] >= k)
                                    o[b][n][i] = __int_as_float(0x7FC00000);
                    }
                }
            }
        }

        // ------------------------------------------------ the chunk's state --
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1)
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
            if (g == 0)
                s_sum[(8 * (i / 2) + 2 * t + i % 2) * kWarps + warp] = l[i];
        }
        __syncthreads();  // C: sums written
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            const float *ss = s_sum + (8 * (i / 2) + 2 * t + i % 2) * kWarps;
            const float4 u = *reinterpret_cast<const float4 *>(ss), v = *reinterpret_cast<const float4 *>(ss + 4);
            l[i] = ((u.x + u.y) + (u.z + u.w)) + ((v.x + v.y) + (v.z + v.w));
            if (bad)
                l[i] = __int_as_float(0x7FC00000);
            if (l[i] != l[i] && m[i] == -INFINITY)
                m[i] = 0.f;  // a NaN state must not pass for an empty one
        }
        const int rv = c.qn * G;
        const bool last = c.lc + 1 == c.nch;
        const int64_t group = (int64_t)c.b * hkv + c.kvh;
        if (whole) {
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const Fold f = fold_coef(acc_m[i], acc_l[i], m[i], l[i]);
                acc_m[i] = f.m;
                acc_l[i] = f.l;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        acc_o[b][i / 2][i % 2 + 2 * k] = fold_elem(acc_o[b][i / 2][i % 2 + 2 * k], o[b][i / 2][i % 2 + 2 * k], f);
                const int r = 8 * (i / 2) + 2 * t + i % 2;
                if (last && r < rv) {
                    const int64_t row = (int64_t)(c.qs + r / G) * p.hq + c.kvh * G + r % G;
                    const float rl = __frcp_rn(acc_l[i]) * p.v_scale;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        *reinterpret_cast<uint32_t *>(p.out + row * DH + 16 * (warp + 8 * b) + 2 * g) =
                            pack_bf16x2(acc_o[b][i / 2][i % 2] * rl, acc_o[b][i / 2][i % 2 + 2] * rl);
                    if (p.lse && warp == 0 && g == 0)
                        p.lse[row] = lse_of(acc_m[i], acc_l[i] * 0x1p-15f);
                }
            }
        } else {
            float *rec = p.records + (group * p.nch + c.lc) * part_record_floats(p.rows, DH);
            float *ro = rec + part_header_floats(p.rows);
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const int r = 8 * (i / 2) + 2 * t + i % 2;
                if (r < rv) {
                    if (warp == 0 && g == 0) {
                        __stcg(rec + r, m[i]);
                        __stcg(rec + p.rows + r, l[i]);
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        __stcg(reinterpret_cast<float2 *>(ro + (int64_t)r * DH + 16 * (warp + 8 * b) + 2 * g),
                               make_float2(o[b][i / 2][i % 2], o[b][i / 2][i % 2 + 2]));
                }
            }
            if (last || x + 1 == hi) {
                // the group's chunks of this range are written: arrive; the
                // last CTA folds them all
                const int arrivals = cta_of(gs + c.nch - 1) - cta_of(gs) + 1;
                __syncthreads();
                if (tid == 0) {
                    uint32_t old;
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                 : "=r"(old)
                                 : "l"(p.counters + group)
                                 : "memory");
                    const bool fold = old == (uint32_t)(arrivals - 1);
                    if (fold)
                        p.counters[group] = 0u;  // ready for the next call
                    s_flags[1] = fold;
                }
                __syncthreads();
                if (s_flags[1])
                    merge_group<DH>(p, p.records + group * p.nch * part_record_floats(p.rows, DH), c.nch, rv, c.qs,
                                    c.kvh);
            }
        }
    }
    (void)seg_first;
}

template <int DH, int NT>
cudaError_t set_attributes()
{
    return cudaFuncSetAttribute(quant_attn_kernel<DH, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Layout<DH, NT>::bytes(kScanMaxSeqs));
}

template <int DH, int NT>
cudaError_t launch(const Params &p, cudaStream_t stream, int num_sms, int64_t max_chunks, int64_t *grid)
{
    const size_t smem = Layout<DH, NT>::bytes(p.num_seqs);
    // CTAs resident at once: registers allow ctas_per_sm, shared memory (228 KB
    // per SM, 1 KB of it reserved per CTA) may allow fewer
    int64_t per_sm = (int64_t)(228 * 1024 / (smem + 1024));
    per_sm = per_sm < 1 ? 1 : (per_sm > ctas_per_sm<DH, NT>() ? ctas_per_sm<DH, NT>() : per_sm);
    *grid = per_sm * num_sms < max_chunks ? per_sm * num_sms : max_chunks;
    if (*grid < 1)
        *grid = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)*grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, quant_attn_kernel<DH, NT>, p);
}

static int64_t chunks_of(int32_t len) { return ((int64_t)len + kChunk - 1) / kChunk; }

}  // namespace qa

size_t quant_attn_record_bytes(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int rows, int32_t max_seq_len)
{
    return (size_t)num_seqs * num_kv_heads * qa::chunks_of(max_seq_len) * (size_t)part_record_floats(rows, head_dim) * 4;
}

cudaError_t launch_quant_attention(const QuantAttnArgs &a, ErrState *err, cudaStream_t stream, int num_sms, char *info,
                                   size_t info_len)
{
    qa::Params p{};
    p.k = a.pool.k;
    p.v = a.pool.v;
    p.block_stride = a.pool.block_stride;
    p.head_stride = a.pool.head_stride;
    p.num_blocks = a.pool.num_blocks;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.q_tok_stride = a.q_tok_stride;
    p.num_q_tokens = a.num_q_tokens;
    p.block_tables = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.qsl = a.query_start_loc;
    p.max_blocks = a.max_blocks;
    p.num_seqs = a.num_seqs;
    p.hq = a.num_q_heads;
    p.hkv = a.pool.num_kv_heads;
    p.group = p.hq / p.hkv;
    p.max_query_len = a.max_query_len;
    p.max_seq_len = a.max_seq_len;
    p.rows = a.max_query_len * p.group;
    p.nch = qa::chunks_of(a.max_seq_len);
    p.score_scale = a.scale * 1.4426950408889634f * a.pool.k_scale;
    p.v_scale = a.pool.v_scale;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.counters = a.counters;
    p.records = a.records;
    p.err = err;
    const int64_t max_chunks = (int64_t)p.num_seqs * p.hkv * p.nch;
    const int nt = p.rows <= 8 ? 1 : p.rows <= 16 ? 2 : p.rows <= 32 ? 4 : 8;
    int64_t grid = 0;
    cudaError_t e = cudaErrorNotSupported;
    auto go = [&](auto fn) { e = fn(p, stream, num_sms, max_chunks, &grid); };
    switch (a.pool.head_dim) {
    case 128:
        go(nt == 1 ? qa::launch<128, 1> : nt == 2 ? qa::launch<128, 2> : nt == 4 ? qa::launch<128, 4> : qa::launch<128, 8>);
        break;
    case 256:
        go(nt == 1 ? qa::launch<256, 1> : nt == 2 ? qa::launch<256, 2> : qa::launch<256, 4>);
        break;
    case 512:
        go(nt == 1 ? qa::launch<512, 1> : nt == 2 ? qa::launch<512, 2> : qa::launch<512, 4>);
        break;
    }
    snprintf(info, info_len, "quant attention direct dh=%d rows=%d grid=%lld chunks<=%lld", a.pool.head_dim, p.rows,
             (long long)grid, (long long)max_chunks);
    return e;
}

cudaError_t init_quant_attention_attributes()
{
    cudaError_t e;
    if ((e = qa::set_attributes<128, 1>()) != cudaSuccess || (e = qa::set_attributes<128, 2>()) != cudaSuccess ||
        (e = qa::set_attributes<128, 4>()) != cudaSuccess || (e = qa::set_attributes<128, 8>()) != cudaSuccess ||
        (e = qa::set_attributes<256, 1>()) != cudaSuccess || (e = qa::set_attributes<256, 2>()) != cudaSuccess ||
        (e = qa::set_attributes<256, 4>()) != cudaSuccess || (e = qa::set_attributes<512, 1>()) != cudaSuccess ||
        (e = qa::set_attributes<512, 2>()) != cudaSuccess)
        return e;
    return qa::set_attributes<512, 4>();
}

}  // namespace pa

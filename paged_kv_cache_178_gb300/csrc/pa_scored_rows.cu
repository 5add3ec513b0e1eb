// pa_paged_attention_scored for few rows: decode steps and drafted tokens.
//
// Bound by the memory: every K and V byte that some row sees is read once, and
// 16 or 32 rows do not fill an M = 128 tensor-memory tile, so the products run
// on mma.m16n8k16, whose rate is many times what the bytes ask for.
//
// Work: a group is one (request, KV head), at most 32 rows, its items the blocks of
// kKeys keys that some row sees.  The items of all groups are dealt
// out as one wave of equal contiguous ranges, one to a CTA.  What a CTA has of a
// group becomes a record (maximum, sum, unnormalised output) in the workspace; a
// second kernel folds a group's records, in order.
//
// In a CTA a fifth warp copies blocks with TMA page boxes into a ring of stages;
// four warps compute.  Scores: a warp takes a quarter of the block's keys and
// all of the head dim.  Output: a warp takes all keys and a quarter of the head
// dim.  So nothing is computed twice, the output needs no join between warps, and
// maxima and probabilities cross through shared memory (two barriers a block).
//
// Measured, heads of 8 and 2 by 128: a token of each of 64 requests, 312 MB of K
// and V, capped: 56 us, 5.6 TB/s (a plain copy: 6.8); 4 and 8 tokens of each (16 and
// 32 rows) 61 and 84 us: two m16 tiles a block and three special-function operations a
// score are then more than the bytes; of 4 requests behind a
// window of 1024, 3.7 MB: 8.7 us, two launches and the chain of lengths, table,
// copy, products and fold.  With 64-bit divisions in the ranges of items the first
// and last took 59 and 15.9 us.
#include <cstdio>

#include "pa_scan.cuh"
#include "pa_score.cuh"
#include "pa_scored.h"

namespace pa {

constexpr int kRowsWarps = 4;  // computing warps
constexpr int kRowsThreads = (kRowsWarps + 1) * 32;

template <int DH, int MT>
struct RowsCfg {
    static constexpr int kKeys = DH == 128 ? 64 : 32;  // of a block: two or four pages
    // (with three stages of head dim 256 and 32 rows an SM holds one CTA: 115 us
    // instead of 74 for 32 requests of 4096 keys)
    static constexpr int kStages = DH == 512 || (DH == 256 && MT == 2) ? 2 : 3;
    static constexpr int kCtas = DH == 512 ? 1 : 2;  // per SM
    static constexpr int kView = kKeys * DH * 2;     // bytes of K (or V) of a block
};

template <int DH, int MT>
constexpr size_t rows_smem(int num_seqs)
{
    using C = RowsCfg<DH, MT>;
    return 1024 + (size_t)C::kStages * 2 * C::kView + 16 * MT * DH * 2 + 16 * MT * (C::kKeys * 2 + 16) +
           2 * kRowsWarps * 16 * MT * 4 + 256 + (size_t)(num_seqs + 1) * 4;
}
static_assert(2 * (rows_smem<256, 2>(64) + 1024) <= kMaxSmemPerBlock + 1024, "two CTAs to an SM");
static_assert(rows_smem<512, 2>(kScanMaxSeqs) <= kMaxSmemPerBlock, "shared-memory layout");
static_assert(rows_smem<256, 2>(kScanMaxSeqs) <= kMaxSmemPerBlock, "shared-memory layout");
static_assert(rows_smem<128, 2>(kScanMaxSeqs) <= kMaxSmemPerBlock, "shared-memory layout");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t &r0, uint32_t &r1)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Workspace: where each group's parts are, then the records.
struct RowsWork {
    int2 *groups;      // [num_groups] (first CTA * 4 + its record (record_slot), CTAs that have a part)
    float *records;    // [2 * ctas + num_groups] of record_floats
    int64_t record_floats;
    int32_t ctas, rows;  // rows that any request can fill
};

// Record of the part that a CTA (items [clo, chi)) has of a group (items [g0, g1)):
// the group's own (2) where that is all of it, else the CTA's first (0) or second.
__device__ __forceinline__ int record_slot(int g0, int g1, int clo, int chi)
{
    return g0 >= clo && g1 <= chi ? 2 : (g0 <= clo ? 0 : 1);
}
__device__ __forceinline__ int64_t record_index(int slot, int g, int c, int max_ctas)
{
    return 2 * (int64_t)(slot == 2 ? max_ctas : c) + (slot == 2 ? g : slot);
}

// Entry of RowsWork::groups for items [g0, g1) of all.
__device__ __forceinline__ int2 group_parts(int total, int g0, int g1, int ctas)
{
    const int c = range_owner(total, g0, ctas), last = range_owner(total, g1 - 1, ctas);
    return make_int2(c * 4 + record_slot(g0, g1, (int)range_lo(total, c, ctas), (int)range_lo(total, c + 1, ctas)),
                     last - c + 1);
}

template <int DH, int MT>
__global__ void __launch_bounds__(kRowsThreads, RowsCfg<DH, MT>::kCtas)
    scored_rows_kernel(const __grid_constant__ ScoreParams p, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const RowsWork w)
{
    using C = RowsCfg<DH, MT>;
    constexpr int KB = C::kKeys, R = 16 * MT, NS = C::kStages;
    constexpr int KW = KB / kRowsWarps, NT = KW / 8;  // keys of a warp's scores, in n-tiles
    constexpr int DW = DH / kRowsWarps, OT = DW / 8;  // output columns of a warp, in n-tiles
    constexpr int PSTRIDE = KB * 2 + 16;              // bytes; eight rows hit eight bank groups
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *s_kv = smem;                                          // [NS][K, V][DH/64][KB][128 bytes]
    uint8_t *s_q = s_kv + NS * 2 * C::kView;                       // [R][DH], 16-byte chunks XOR row % 8
    uint8_t *s_p = s_q + R * DH * 2;                               // [R][PSTRIDE]
    float *s_max = reinterpret_cast<float *>(s_p + R * PSTRIDE);   // [warps][R]
    float *s_sum = s_max + kRowsWarps * R;                         // [warps][R]
    uint64_t *bars = reinterpret_cast<uint64_t *>(s_sum + kRowsWarps * R);  // full[NS], empty[NS]
    volatile int *s_abort = reinterpret_cast<volatile int *>(bars + 2 * NS);
    uint32_t *s_bad = reinterpret_cast<uint32_t *>(bars + 2 * NS + 1);      // [NS] bad pages of a stage
    int32_t *s_off = reinterpret_cast<int32_t *>(reinterpret_cast<uint8_t *>(bars) + 256);  // [num_seqs + 1]
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto full = [&](int s) { return smem_addr(bars + s); };
    auto empty = [&](int s) { return smem_addr(bars + NS + s); };

    // -------------------------------------------- items before each request --
    int *scratch = reinterpret_cast<int *>(s_max);  // (all sums fit: at most INT32_MAX items)
    static_assert(2 * kRowsWarps * 16 >= kRowsWarps + 1, "scan scratch");
    const int per_head = block_exclusive_sums<kRowsThreads>(p.num_seqs, s_off, scratch, [&](int b) {
        const ReqMeta m = score_meta(p, b);
        if (!m.ok) {
            if (blockIdx.x == 0)
                record_error(p.err, kErrBadMetadata, b);
            return 0;
        }
        return tile_blocks(tile_view(p, b, m, 0, m.qn * p.group), KB).count;
    });
    const int total = per_head * p.hkv, ctas = min(w.ctas, total), c = blockIdx.x;
    // where the fold finds a group's parts
    auto write_groups = [&](int at, int step) {
        for (int g = at; g < p.num_seqs * p.hkv; g += step) {
            const int b = g / p.hkv, n = s_off[b + 1] - s_off[b];
            const int first = s_off[b] * p.hkv + (g - b * p.hkv) * n;
            w.groups[g] = n ? group_parts(total, first, first + n, ctas) : make_int2(0, 0);
        }
    };
    if (c >= ctas) {
        if (warp == kRowsWarps)
            write_groups(c * 32 + lane, w.ctas * 32);
        return;
    }
    const int lo = (int)range_lo(total, c, ctas), hi = (int)range_lo(total, c + 1, ctas);
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kRowsWarps);
        }
        *s_abort = 0;
        fence_barrier_init();
    }
    __syncthreads();

    // the group of an item, as both sides walk through the range
    struct Group {
        int b, kvh, g, rows;
        int g0, g1;
        ReqMeta m;
        TileView v;
        TileBlocks t;
    };
    auto group_of = [&](int item) {
        Group x;
        x.b = owner_of(s_off, p.num_seqs, item / p.hkv);  // no request's items before that are past the item
        const int n = s_off[x.b + 1] - s_off[x.b], first = s_off[x.b] * p.hkv;
        x.kvh = (item - first) / n;
        x.g = x.b * p.hkv + x.kvh;
        x.g0 = first + x.kvh * n;
        x.g1 = x.g0 + n;
        x.m = score_meta(p, x.b);
        x.rows = x.m.qn * p.group;
        x.v = tile_view(p, x.b, x.m, 0, x.rows);
        x.t = tile_blocks(x.v, KB);
        return x;
    };
    auto block_key = [&](const Group &x, int i) { return (i < x.t.np ? i : x.t.b0 + i - x.t.np) * KB; };

    if (warp == kRowsWarps) {
        // ---------------------------------------------------------- producer --
        constexpr int NB = (KB / 16) * (DH / 64);  // boxes of a view: (page, 64 columns) a lane
        static_assert(NB <= 32, "a lane per box");
        const int pg = lane % (KB / 16), cb = lane / (KB / 16);
        const uint64_t policy = l2_policy_evict_first();
        int stage = 0, round = 0, issued = 0;
        bool ok = true;
        for (int item = lo; ok && item < hi;) {
            const Group x = group_of(item);
            const int32_t *bt = p.block_tables + (int64_t)x.b * p.max_blocks;
            const int end = min(hi, x.g1);
            for (; item < end; ++item) {
                const int k0 = block_key(x, item - x.g0) + pg * 16;
                // pages that hold no key which some row sees are not read
                const bool need = page_needed(p, x.m, x.v, 0, x.rows, k0);
                int id = need ? __ldg(bt + k0 / 16) : -1;
                const bool bad = need && (id < 0 || (int64_t)id >= p.num_blocks);
                if (bad)
                    id = -1;
                const uint32_t bad_pages = __ballot_sync(0xffffffffu, bad && cb == 0);
                if (round > 0)
                    ok = wait_bar(empty(stage), (round - 1) & 1, s_abort, p.err, NS + stage);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                if (lane == 0) {
                    s_bad[stage] = bad_pages;
                    if (bad_pages)
                        record_error(p.err, kErrBadMetadata, x.b);
                    mbar_arrive_expect_tx(full(stage), 2 * C::kView);
                }
                __syncwarp();
                if (lane < NB) {
                    // (block -1 lies outside the pool: zeros, no bytes read)
                    const uint32_t at = smem_addr(s_kv + stage * 2 * C::kView + cb * KB * 128 + pg * 2048);
                    tma_load_4d_hint(at, &tm_k, full(stage), cb * 64, x.kvh, 0, id, policy);
                    tma_load_4d_hint(at + C::kView, &tm_v, full(stage), cb * 64, x.kvh, 0, id, policy);
                }
                ++issued;
                if (++stage == NS)
                    stage = 0, ++round;
            }
        }
        // after a timeout: no copy may land in memory that the CTA has left
        if (!ok && lane == 0)
            for (int i = max(0, issued - NS); i < issued; ++i)
                wait_bar_drain(full(i % NS), (i / NS) & 1);
        write_groups(c * 32 + lane, w.ctas * 32);
        return;
    }

    // ------------------------------------------------------------- compute --
    const int g8 = lane / 4, t4 = lane % 4;
    // (a wide cap has a pass of its own, and leaves nothing to do here)
    const bool wide = p.cap_log2 > kCapNarrow;
    const float c1 = wide ? 1.f : p.scale_log2, cap = wide ? 0.f : p.cap_log2;
    int stage = 0, parity = 0;
    bool ok = true;
    for (int item = lo; item < hi;) {
        const Group x = group_of(item);
        const int end = min(hi, x.g1);
        const int rows = x.rows;
        named_sync(1, kRowsWarps * 32);  // Q and the sums of the group before have been read
        // Q into shared memory; rows past the request's are zero
        for (int i = tid; i < R * (DH / 8); i += kRowsWarps * 32) {
            const int r = i / (DH / 8), ch = i % (DH / 8);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
                const int tok = r / p.group, h = x.kvh * p.group + r - tok * p.group;
                v = __ldg(reinterpret_cast<const uint4 *>(p.q + ((int64_t)x.m.qs + tok) * p.q_tok_stride + (int64_t)h * DH) + ch);
            }
            *reinterpret_cast<uint4 *>(s_q + r * DH * 2 + (ch ^ (r & 7)) * 16) = v;
        }
        // what this lane's rows see: 2 * MT of them
        int r_lo[2 * MT], r_len[2 * MT], r_near[2 * MT], r_pos[2 * MT];
        float slope[2 * MT];
        int lo_max = 0, pos_min = INT32_MAX;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int r = 8 * i + g8;
            r_lo[i] = r_len[i] = r_near[i] = r_pos[i] = 0;
            slope[i] = 0.f;
            if (r < rows) {
                const int tok = r / p.group, pos = x.m.L - x.m.qn + tok;
                r_pos[i] = pos;
                r_lo[i] = score_low(p, (int64_t)x.m.qs + tok, pos);
                r_len[i] = pos - r_lo[i] + 1;
                r_near[i] = score_nearest(r_lo[i], pos, x.v.prefix);
                if (p.slopes)
                    slope[i] = __ldg(p.slopes + x.kvh * p.group + r - tok * p.group) * kLog2e;
                lo_max = max(lo_max, r_lo[i]);
                pos_min = min(pos_min, pos);
            }
        }
        lo_max = __reduce_max_sync(0xffffffffu, lo_max);
        pos_min = __reduce_min_sync(0xffffffffu, pos_min);
        float m[2 * MT], l[2 * MT], o[MT][OT][4];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < OT; ++j)
                o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
        named_sync(1, kRowsWarps * 32);
        for (; item < end; ++item) {
            const int k0 = block_key(x, item - x.g0);
            if (ok)
                ok = wait_bar(full(stage), parity, s_abort, p.err, stage);
            const uint32_t kb = smem_addr(s_kv + stage * 2 * C::kView), vb = kb + C::kView;
            const uint32_t bad_pages = s_bad[stage];
            // scores of this warp's keys
            float s[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                uint32_t bf[4];
                // matrices: keys 0-7 and, with two n-tiles, 8-15; columns 0-7 and 8-15 of the step
                const int key = warp * KW + (NT == 2 ? (lane / 16) * 8 : 0) + lane % 8;
                const int ch = ks * 2 + (lane / 8) % 2;
                const uint32_t ka = kb + (ch / 8) * KB * 128 + key * 128 + (((ch % 8) ^ (key & 7)) << 4);
                if (NT == 2)
                    ldsm4(ka, bf);
                else
                    ldsm2(ka, bf[0], bf[1]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t af[4];
                    const int r = i * 16 + lane % 16, qc = ks * 2 + lane / 16;
                    ldsm4(smem_addr(s_q + r * DH * 2 + (qc ^ (r & 7)) * 16), af);
                    mma16816(s[i][0], af, bf[0], bf[1]);
                    if (NT == 2)
                        mma16816(s[i][NT - 1], af, bf[2], bf[3]);
                }
            }
            // scores in log2 units, what is hidden at -inf; their row maxima
            if (wide) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[i][j][e] = capped_wide(s[i][j][e], p.scale_log2, p.cap_log2);
            }
            const bool all = (k0 >= lo_max && k0 + KB - 1 <= pos_min) || k0 + KB <= x.v.prefix;
            float mx[2 * MT];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                mx[i] = -INFINITY;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &z = s[i / 2][j][(i % 2) * 2 + e];
                        const int key = k0 + warp * KW + j * 8 + t4 * 2 + e;
                        z = cap > 0.f ? capped(z, c1, cap) : z * c1;
                        if (p.slopes)
                            z -= slope[i] * (float)(abs(r_pos[i] - key) - r_near[i]);
                        if (bad_pages && (bad_pages >> ((key - k0) / 16) & 1u))
                            z = __int_as_float(0x7FC00000);
                        if (!all || bad_pages)
                            z = key < x.v.prefix || (uint32_t)(key - r_lo[i]) < (uint32_t)r_len[i] ? z : -INFINITY;
                        mx[i] = fmaxf(mx[i], z);
                    }
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                if (t4 == 0)
                    s_max[warp * R + 8 * i + g8] = mx[i];
            }
            named_sync(1, kRowsWarps * 32);
            float alpha[2 * MT];
            bool scale_o = false;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                float top = m[i];
#pragma unroll
                for (int k = 0; k < kRowsWarps; ++k)
                    top = fmaxf(top, s_max[k * R + 8 * i + g8]);
                alpha[i] = top == m[i] ? 1.f : ex2(m[i] - top);
                scale_o |= alpha[i] != 1.f;
                m[i] = top;
                const float base = top == -INFINITY ? 0.f : top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float *z = &s[i / 2][j][(i % 2) * 2];
                    const float p0 = ex2(z[0] - base), p1 = ex2(z[1] - base);
                    sum += p0 + p1;
                    *reinterpret_cast<uint32_t *>(s_p + (8 * i + g8) * PSTRIDE + (warp * KW + j * 8 + t4 * 2) * 2) =
                        pack_bf16x2(p0, p1);
                }
                l[i] = l[i] * alpha[i] + sum;
            }
            if (__any_sync(0xffffffffu, scale_o)) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < OT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][j][e] *= alpha[2 * i + e / 2];
            }
            named_sync(1, kRowsWarps * 32);
            // output: V rows that no row sees become zeros (they may
            // hold anything, and 0 * NaN is NaN)
            const bool whole = (k0 >= x.v.lo && k0 + KB <= x.v.hi) || k0 + KB <= x.v.prefix;
#pragma unroll
            for (int ks = 0; ks < KB / 16; ++ks) {
                uint32_t af[MT][4], keep[2];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    ldsm4(smem_addr(s_p + (i * 16 + lane % 16) * PSTRIDE + (ks * 2 + lane / 16) * 16), af[i]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = k0 + ks * 16 + i * 8 + t4 * 2;
                    auto seen = [&](int j) { return j < x.v.prefix || (j >= x.v.lo && j < x.v.hi); };
                    keep[i] = whole ? 0xffffffffu : (seen(key) ? 0xffffu : 0u) | (seen(key + 1) ? 0xffff0000u : 0u);
                }
#pragma unroll
                for (int j = 0; j < OT; j += 2) {
                    uint32_t bf[4];
                    const int key = ks * 16 + lane % 16, ch = (warp * DW + j * 8) / 8 + lane / 16;
                    ldsm4t(vb + (ch / 8) * KB * 128 + key * 128 + (((ch % 8) ^ (key & 7)) << 4), bf);
                    if (!whole) {
                        bf[0] &= keep[0], bf[1] &= keep[1];
                        bf[2] &= keep[0], bf[3] &= keep[1];
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        mma16816(o[i][j], af[i], bf[0], bf[1]);
                        mma16816(o[i][j + 1], af[i], bf[2], bf[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(stage));
            if (++stage == NS)
                stage = 0, parity ^= 1;
        }
        // the record: a row's sum over the lanes and warps that share it
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (t4 == 0)
                s_sum[warp * R + 8 * i + g8] = ok ? l[i] : __int_as_float(0x7FC00000);
        }
        named_sync(1, kRowsWarps * 32);
        float *rec = w.records + record_index(record_slot(x.g0, x.g1, lo, hi), x.g, c, w.ctas) * w.record_floats;
        if (warp == 0 && t4 == 0)
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                const int r = 8 * i + g8;
                if (r < rows) {
                    rec[r] = m[i];
                    rec[R + r] = (s_sum[r] + s_sum[R + r]) + (s_sum[2 * R + r] + s_sum[3 * R + r]);
                }
            }
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int r = 8 * i + g8;
            if (r < rows) {
                float *dst = rec + 2 * R + (int64_t)r * DH + warp * DW + t4 * 2;
#pragma unroll
                for (int j = 0; j < OT; ++j)
                    *reinterpret_cast<float2 *>(dst + j * 8) =
                        make_float2(o[i / 2][j][(i % 2) * 2], o[i / 2][j][(i % 2) * 2 + 1]);
            }
        }
    }
}

// Folds a row's records: a CTA per (group, row).  A row whose result is not
// finite is computed again key by key: a key that only other rows of the request
// see may have met a zero probability with an infinity or a NaN.
constexpr int kFoldThreads = 256;
constexpr int kFoldWarps = kFoldThreads / 32;

template <int DH>
__global__ void __launch_bounds__(kFoldThreads) scored_fold_kernel(const ScoreParams p, const RowsWork w, int tile_rows)
{
    constexpr int E = DH / 128;  // 16-byte vectors of a lane
    __shared__ float s_part[kFoldWarps][DH];
    __shared__ float s_ml[2][kFoldWarps];
    const int g = blockIdx.x / w.rows, r = blockIdx.x - g * w.rows;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int b = g / p.hkv, kvh = g - b * p.hkv;
    // (the caller's inputs were there before the first kernel read them)
    const ReqMeta m = score_meta(p, b);
    griddep_wait();
    griddep_launch_dependents();
    const int2 parts = w.groups[g];
    if (!m.ok) {
        // every row of the request, whatever its number: the grid goes by the bounds
        if (m.sane && kvh == 0 && r == 0) {
            const int64_t first = (int64_t)m.qs * p.hq, n = (int64_t)m.qn * p.hq;
            for (int64_t i = tid; i < n * DH; i += kFoldThreads)
                p.out[first * DH + i] = __ushort_as_bfloat16(0x7FC0);
            if (p.lse)
                for (int64_t i = tid; i < n; i += kFoldThreads)
                    p.lse[first + i] = __int_as_float(0x7FC00000);
        }
        return;
    }
    const int tok = r / p.group, h = kvh * p.group + r - tok * p.group;
    if (tok >= m.qn)
        return;
    // a warp takes every eighth part
    float mx = -INFINITY, l = 0.f;
    float4 o[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = warp; i < parts.y; i += kFoldWarps) {
        const float *rec = w.records + record_index(i == 0 ? parts.x & 3 : 0, g, (parts.x >> 2) + i, w.ctas) * w.record_floats;
        const float mr = __ldcg(rec + r), lr = __ldcg(rec + tile_rows + r);
        const float top = fmaxf(mx, mr);
        const float a = mx == top ? 1.f : ex2(mx - top), k = mr == top ? 1.f : ex2(mr - top);
        l = l * a + lr * k;
        mx = top;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(rec + 2 * tile_rows + (int64_t)r * DH) + e * 32 + lane);
            o[e].x = o[e].x * a + v.x * k;
            o[e].y = o[e].y * a + v.y * k;
            o[e].z = o[e].z * a + v.z * k;
            o[e].w = o[e].w * a + v.w * k;
        }
    }
    if (lane == 0) {
        s_ml[0][warp] = mx;
        s_ml[1][warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        *reinterpret_cast<float4 *>(&s_part[warp][(e * 32 + lane) * 4]) = o[e];
    __syncthreads();
    float top = -INFINITY, sum = 0.f, k[kFoldWarps];
#pragma unroll
    for (int i = 0; i < kFoldWarps; ++i)
        top = fmaxf(top, s_ml[0][i]);
#pragma unroll
    for (int i = 0; i < kFoldWarps; ++i) {
        k[i] = s_ml[0][i] == top ? 1.f : ex2(s_ml[0][i] - top);
        sum += s_ml[1][i] * k[i];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t at = ((int64_t)m.qs + tok) * p.hq + h;
    bool odd = !(fabsf(sum) < INFINITY);
    for (int d = tid * 2; d < DH; d += 2 * kFoldThreads) {
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < kFoldWarps; ++i) {
            a += s_part[i][d] * k[i];
            c += s_part[i][d + 1] * k[i];
        }
        a *= inv, c *= inv;
        odd |= !(fabsf(a) < INFINITY && fabsf(c) < INFINITY);
        *reinterpret_cast<uint32_t *>(p.out + at * DH + d) = pack_bf16x2(a, c);
    }
    if (tid == 0 && p.lse) {
        const int pos = m.L - m.qn + tok;
        const int near = score_nearest(score_low(p, (int64_t)m.qs + tok, pos), pos, score_prefix(p, b, m.L));
        const float slope = p.slopes ? __ldg(p.slopes + h) : 0.f;
        p.lse[at] = score_lse(top, sum, slope * (float)near);
    }
    if (__syncthreads_or(odd) && warp == 0)
        scored_row<DH>(p, b, m, tok, h, 0, DH, !(fabsf(sum) < INFINITY));
}

// --------------------------------------------------------------------- host --
static int rows_of(int32_t max_query_len, int group) { return max_query_len * group <= 16 ? 16 : 32; }

static int rows_keys(int dh) { return dh == 128 ? 64 : 32; }

bool scored_rows_fits(int32_t num_seqs, int32_t hkv, int32_t head_dim, int32_t max_seq_len)
{
    const int64_t groups = (int64_t)num_seqs * hkv;
    return groups * 32 <= INT32_MAX &&
           groups * (((int64_t)max_seq_len + rows_keys(head_dim) - 1) / rows_keys(head_dim) + 1) <= INT32_MAX;
}

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The CTAs of a wave, or fewer where the bounds allow fewer items.
static int rows_ctas(int64_t groups, int head_dim, int32_t max_seq_len)
{
    const int64_t items = groups * (((int64_t)max_seq_len + rows_keys(head_dim) - 1) / rows_keys(head_dim) + 1);
    const int64_t wave = (int64_t)kScoredSms * (head_dim == 512 ? 1 : 2);
    return (int)(items < wave ? items : wave);
}

size_t scored_rows_bytes(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len,
                         int32_t max_seq_len)
{
    const int64_t groups = (int64_t)num_seqs * hkv;
    const int r = rows_of(max_query_len, group);
    return align256((size_t)groups * 8) +
           (size_t)(2 * rows_ctas(groups, head_dim, max_seq_len) + groups) * r * (head_dim + 2) * 4;
}

template <int DH, int MT>
static cudaError_t launch_rows(const ScoreParams &p, const CUtensorMap &k, const CUtensorMap &v, const RowsWork &w,
                               int64_t groups, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)w.ctas);
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = rows_smem<DH, MT>(p.num_seqs);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, scored_rows_kernel<DH, MT>, p, k, v, w);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3((unsigned)(groups * w.rows));
    cfg.blockDim = dim3(kFoldThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, scored_fold_kernel<DH>, p, w, 16 * MT);
}

cudaError_t launch_scored_rows(const ScoreParams &p, int32_t head_dim, void *workspace, cudaStream_t stream, char *info,
                               size_t info_len)
{
    CUtensorMap tm[2];
    if (!scored_pool_maps(p, head_dim, tm))
        return cudaErrorInvalidValue;
    RowsWork w{};
    const int r = rows_of(p.max_query_len, p.group);
    const int64_t groups = (int64_t)p.num_seqs * p.hkv;
    w.ctas = rows_ctas(groups, head_dim, p.max_seq_len);
    w.rows = p.max_query_len * p.group;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    w.groups = reinterpret_cast<int2 *>(ws);
    w.records = reinterpret_cast<float *>(ws + align256((size_t)groups * 8));
    w.record_floats = (int64_t)r * (head_dim + 2);
    snprintf(info, info_len, "scored attention dh=%d kernel=rows-r%d grid=%d", head_dim, r, w.ctas);
    const bool two = r == 32;
    switch (head_dim) {
    case 128: return two ? launch_rows<128, 2>(p, tm[0], tm[1], w, groups, stream) : launch_rows<128, 1>(p, tm[0], tm[1], w, groups, stream);
    case 256: return two ? launch_rows<256, 2>(p, tm[0], tm[1], w, groups, stream) : launch_rows<256, 1>(p, tm[0], tm[1], w, groups, stream);
    default: return two ? launch_rows<512, 2>(p, tm[0], tm[1], w, groups, stream) : launch_rows<512, 1>(p, tm[0], tm[1], w, groups, stream);
    }
}

template <int DH, int MT>
static cudaError_t rows_attribute()
{
    return cudaFuncSetAttribute(scored_rows_kernel<DH, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)rows_smem<DH, MT>(kScanMaxSeqs));
}

cudaError_t init_scored_rows_attributes()
{
    cudaError_t e;
    if ((e = rows_attribute<128, 1>()) != cudaSuccess || (e = rows_attribute<128, 2>()) != cudaSuccess ||
        (e = rows_attribute<256, 1>()) != cudaSuccess || (e = rows_attribute<256, 2>()) != cudaSuccess ||
        (e = rows_attribute<512, 1>()) != cudaSuccess)
        return e;
    return rows_attribute<512, 2>();
}

}  // namespace pa

// Attention of few query rows over a 4-bit cache (pa_quant_common.cuh): decode
// steps and drafted tokens.  S = Q.K^T, P = softmax(S), O = P.V with K and V
// dequantised on the way into the matrix instructions.
//
// What bounds it: a 16-token page of one KV head at head dim 128 is 2304
// bytes (K and V), 98 clocks of an SM's share of the memory bandwidth.  Its
// 4096 elements need 2048 conversions (two elements each) and as many scale
// products, which issue at two warp instructions per clock and SM: 64 clocks.
// So the instruction count decides.  Passing dequantised tiles through shared
// memory (as operands of tcgen05) would add 16 KB of writes and 16 KB of operand
// reads per page, 256 clocks at 128 bytes per clock; the fragments of mma.sync
// are built in registers, straight from the codes, and nothing dequantised is
// ever stored.
//
// The products are mma.m16n8k16, f16 with fp32 accumulation.  Codes times
// scales are exact in f16; q is scaled per row by a power of two to [1, 2) at
// its largest element (what is below 2^-14 of it loses bits, at most 2^-25 of
// the largest); p is scaled by 2^15 (11 bits down to 2^-29 of the row's largest
// probability).  Both are the matrix instruction's operand type; p's rounding
// adds less than 1% to the error that the rounding of the result leaves.
//   S^T = K.Q^T: M = the 16 tokens of a page, N = 8 query rows, K = head dim.
//   O^T = V^T.P^T: M = the head dim, N = 8 query rows, K = the 16 tokens.  A V
//     byte holds two neighbouring elements of one token; permutes regroup the
//     converted pairs by element, and the scales come as pairs of tokens.
//     (Taking the pair as two K indices instead, with (p, 0) and (0, p) as
//     columns of P, saves the permutes but needs each scale twice: 56 clocks of
//     shared-memory reads per page against 32.)
//
// Fixed arithmetic (a row's results do not depend on the batch or the grid):
//   chunks of 512 keys (256 at head dim 256, 128 at 512) from key 0, each with
//   its own exact maximum; a chunk's row sum is, per warp, a butterfly over its
//   keys, then the eight warps' sums pairwise; the states of a span of 16 chunks
//   are added with their exact maximum (the outputs in order, the sums as a
//   tree of fixed shape), and the spans fold left to right (State::fold).
//
// A CTA (8 warps) per chunk: each warp scores its pages; row maxima are
// exchanged (barrier); P goes to shared memory in fragment order, the V scales
// as one f16 pair each (barrier); each warp multiplies P by 32 head-dim
// elements of the pages (at head dim 128 of half of the pages, the halves are
// added through shared memory, with the row sums; barrier).  A ninth warp
// copies the next chunk (cp.async.bulk): K during the second product, V during
// the first one.  The chunks of all (token tile, KV head) groups are dealt out as
// contiguous ranges of about equal weight; the state of a chunk becomes a
// record, unless it is its group's only one, and a second kernel folds the
// records.  (Folded by the last CTA to arrive instead, 32 records of eight rows
// took that CTA 5 us, 17 of twenty rows at head dim 256 13 us.)
//
// Measured in a CUDA graph (as all times in this file; issued one by one they
// are 0.4 to 0.9 us longer), head dim 128 unless said: 64 requests of 7168,
// 7168, 4171 and 513 keys with 8 query and 2 KV heads (88 MB) 29.8 us, of which
// the metadata and the shares take 2, the first chunk 7, three more 4.2 each
// (5.3 TB/s, two CTAs per SM), uneven ends 4 and the fold 3; four of them 8.6
// us; 131072 keys and 32 query and 4 KV heads 29.9 us; 16 requests of up to 5000
// keys with five new tokens at head dim 256 24.3 us, 4.8 a chunk of 256 keys,
// bound by latency: one CTA per SM goes from product to exchange to product (a
// quarter of the issue slots, 18% of the tensor pipe, 13% of the DRAM's rate).
#include <cstdio>
#include <type_traits>

#include "pa_attn_common.cuh"
#include "pa_quant_common.cuh"
#include "pa_scan.cuh"
#include "pa_split.cuh"

namespace pa {

namespace qa {

// Computing warps.  (Sixteen of them at head dim 256, a page each, took 43 us
// for five new tokens instead of 24.6: each reads all of Q and all maxima and
// sums from shared memory, which is then busy.)
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;       // computing threads
constexpr int kAllThreads = kThreads + 32;  // and the copying warp
// pages per warp of a chunk: as many as shared memory holds (at head dim 128
// for two CTAs), since a chunk's exchanges and bookkeeping cost the same
__host__ __device__ constexpr int pages_per_warp(int dh) { return dh == 128 ? 4 : dh == 256 ? 2 : 1; }
__host__ __device__ constexpr int chunk_pages(int dh) { return kWarps * pages_per_warp(dh); }
__host__ __device__ constexpr int chunk_keys(int dh) { return 16 * chunk_pages(dh); }
constexpr int kSpan = 16;           // chunks per span of the fold
// What a chunk costs without its pages, in pages, when the chunks are dealt out:
// 64 requests 31.5 us at 8, 30.5 at 18, 32.4 at 32.
constexpr int kChunkCost = 18;
// A tile's weight is at most 1 + kChunkCost / 8 times its pages, and kChunkCost:
// sums stay below 2^31 for two tiles of requests of 2^28 pages.  (More tiles to
// a request: each chunk of a tile has a record of nine rows or more, so the
// sums pass 2^31 only where the records pass the memory of a GPU, or the pages
// max_pages, and then differences alone are used.)
static_assert(2.0 * (1 << 28) * (1 + kChunkCost / 8.0) + kQuantMaxTiles * kChunkCost < 2147483648.0, "weights");
constexpr float kShift = 15.f;      // p is scaled by 2^kShift (largest f16: 2^16)
constexpr int kGridSms = 152;       // SMs the grid is sized for

// CTAs per SM that registers and shared memory are sized for: two where a
// thread's share of the state fits in half of the registers (64 requests at head
// dim 256 54 us with one, 48 with two; at head dim 512 59 and 53, with 12 rows
// 157 and 149; but 12 rows at head dim 256 79 and 85).
__host__ __device__ constexpr int ctas_per_sm(int dh, int rn) { return rn <= 8 || dh == 512 ? 2 : 1; }
// Shared memory that keeps a second CTA off an SM.
constexpr int kSmemAlone = 118 * 1024;
// Shared-memory layout in bytes.  RN: query rows (8, 16, 24 or 32).
template <int DH, int RN>
struct Layout {
    static constexpr int kPages = chunk_pages(DH);
    static constexpr int NQ = RN / 8;                               // N tiles
    static constexpr int NCF = DH == 128 ? RN / 2 : 0;              // floats a thread hands to the other half
    static constexpr int q = 2 * kPages * quant_record_bytes(DH);  // after the K and the V records
    static constexpr int p = q + NQ * DH * 16;
    static constexpr int spread = p + kPages * NQ * 256;            // V scales as f16
    static constexpr int half = spread + kPages * DH * 2;
    static constexpr int max = half + kThreads * NCF * 4;
    static constexpr int sum = max + NQ * 8 * kWarps * 4;
    static constexpr int cq = sum + NQ * 8 * kWarps * 4;
    static constexpr int lim = cq + NQ * 8 * 4;
    static constexpr int nan = lim + NQ * 8 * 4;
    static constexpr int bad = nan + 2 * (DH / 16) * 4;
    static constexpr int flags = bad + 16;
    static constexpr int bars = flags + 16;         // full and empty, of K and of V
    static constexpr int sums = bars + 32;           // 16 bytes for each of nine warps
    static constexpr int pre = sums + (kWarps + 2) * 16;  // two arrays [num_tiles + 1] int32
    static_assert(q % 16 == 0 && spread % 16 == 0 && max % 16 == 0 && bad % 8 == 0 && bars % 16 == 0, "layout");
    static_assert(pre + (kQuantMaxTiles + 1) * 8 <= (int)kMaxSmemPerBlock, "shared memory");
    static size_t bytes(int num_tiles) { return (size_t)pre + 8 * ((size_t)num_tiles + 1); }
};

struct Params {
    const uint8_t *k, *v;
    uint32_t block_stride, head_stride;  // bytes (the host refuses larger ones)
    int64_t num_blocks;
    const __nv_bfloat16 *q;
    int64_t q_tok_stride, num_q_tokens;
    const int32_t *block_tables, *seq_lens, *qsl;
    int32_t max_blocks, hq, hkv, group, max_query_len, max_seq_len;
    int32_t tile_shift, tile_tokens;  // a request's tokens form 1 << tile_shift tiles of tile_tokens
    int32_t num_tiles;  // of all requests
    int32_t per_group;  // a CTA for each of so many chunks of every group (0: the chunks are dealt out)
    int32_t rows;       // rows of a record (of a tile)
    int64_t max_pages;  // pages of all requests together
    float score_scale;  // scale * log2(e) * k_scale
    float v_scale;
    __nv_bfloat16 *out;
    float *lse;
    float *records;     // [chunk]: m, l, O
    int32_t *offsets;   // [num_tiles + 1]: chunks of a KV head before each tile
    uint64_t wait_ns;   // limit of a wait
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

// Arrives at a named barrier without waiting.
__device__ __forceinline__ void bar_arrive(int id, int nthreads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
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

// A tile of a request's tokens: the rows one CTA holds at a time.
struct Meta {
    int qs, qn;     // first token and tokens of the tile
    int L;          // keys of the request
    int seen;       // last key that the tile's first token sees
    bool sane, ok;  // as ReqMeta
};

__device__ __forceinline__ Meta meta_of(const Params &p, int tile)
{
    Meta m;
    const int b = tile >> p.tile_shift, first = (tile - (b << p.tile_shift)) * p.tile_tokens;
    const int qs = __ldg(p.qsl + b), qe = __ldg(p.qsl + b + 1);
    m.L = __ldg(p.seq_lens + b);
    m.sane = qs >= 0 && qe >= qs && (int64_t)qe <= p.num_q_tokens;
    const int qn = m.sane ? qe - qs : 0;
    m.ok = m.sane && m.L >= qn && (int64_t)m.L <= (int64_t)p.max_blocks * 16 && qn <= p.max_query_len &&
           m.L <= p.max_seq_len;
    m.qs = qs + first;
    m.qn = max(0, qn - first);
    if (m.ok || (tile + 1) >> p.tile_shift == b)  // (too many tokens: the last tile has the rest)
        m.qn = min(m.qn, p.tile_tokens);
    m.seen = m.L - qn + first;
    return m;
}

// A chunk of the dealt sequence: chunk lc of group (tile, kvh), tile-major.
template <int DH>
struct Chunk {
    int tile, kvh, lc, nch;
    int qs, qn, L, seen;
    const int32_t *row;  // the request's block table

    __device__ __forceinline__ void load(const Params &p)
    {
        const Meta m = meta_of(p, tile);
        qs = m.qs;
        qn = m.qn;
        L = m.L;
        seen = m.seen;
        nch = (L + chunk_keys(DH) - 1) / chunk_keys(DH);
        row = p.block_tables + (int64_t)(tile >> p.tile_shift) * p.max_blocks;
    }
    __device__ __forceinline__ void at(const Params &p, const int32_t *pre, int64_t x)
    {
        tile = owner_of(pre, p.num_tiles, (int)div_floor(x, p.hkv));
        load(p);
        const int r = (int)(x - (int64_t)p.hkv * pre[tile]);
        kvh = (int)((uint32_t)r / (uint32_t)nch);
        lc = r - kvh * nch;
    }
    // the first chunk of a CTA
    __device__ __forceinline__ void start(const Params &p, const int32_t *pre, int64_t x)
    {
        if (p.per_group == 0) {
            at(p, pre, x);
            return;
        }
        const uint32_t group = (uint32_t)x / (uint32_t)p.per_group;
        tile = (int)(group / (uint32_t)p.hkv);
        kvh = (int)(group - (uint32_t)tile * p.hkv);
        lc = (int)((uint32_t)x - group * p.per_group);
        load(p);
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
            ++tile;
        while (pre[tile + 1] == pre[tile]);
        load(p);
    }
    __device__ __forceinline__ bool has_page(int i) const { return (lc * chunk_pages(DH) + i) * 16 < L; }
    // block id of the chunk's page i (0 where there is none)
    __device__ __forceinline__ int id(int i) const { return has_page(i) ? __ldg(row + lc * chunk_pages(DH) + i) : 0; }
};

// A thread's share of a softmax state (of a chunk, a span or a group): NR
// query rows, for each of them NP pairs of neighbouring head-dim elements.
template <int NR, int NP>
struct State {
    float m[NR], l[NR];
    float2 o[NP][NR];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                o[i][r] = make_float2(0.f, 0.f);
        }
    }
    // This state, then x.  An empty state (m = -inf, l = 0, o = 0) changes
    // nothing: its factor is 0 and the other's exactly 1.
    __device__ __forceinline__ void fold(const State &x)
    {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float mn = fmaxf(m[r], x.m[r]), ref = mn == -INFINITY ? 0.f : mn;
            const float fa = ex2(m[r] - ref), fx = ex2(x.m[r] - ref);
            m[r] = mn;
            l[r] = __fmaf_rn(x.l[r], fx, l[r] * fa);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                o[i][r].x = __fmaf_rn(x.o[i][r].x, fx, o[i][r].x * fa);
                o[i][r].y = __fmaf_rn(x.o[i][r].y, fx, o[i][r].y * fa);
            }
        }
    }
};

template <int DH, int RN>
__global__ void __launch_bounds__(kAllThreads, ctas_per_sm(DH, RN)) quant_attn_kernel(const Params p)
{
    using Lay = Layout<DH, RN>;
    constexpr int NQ = Lay::NQ;
    constexpr int PPW = pages_per_warp(DH), kPages = chunk_pages(DH), kChunk = chunk_keys(DH);
    constexpr int NB = DH / 128;            // 128-element blocks of the head dim
    constexpr int NE = DH <= 256 ? 1 : 2;   // 32-element blocks of a warp
    constexpr bool HALVES = DH == 128;      // warps 4-7 take the other half of the pages
    constexpr int NR = RN / 4;  // rows of a thread's state
    constexpr int NP = HALVES ? 1 : 2 * NE;   // element pairs of a thread's state
    static_assert(NP * NR <= 32, "a bit each");
    constexpr int REC = quant_record_bytes(DH), CODES = quant_code_bytes(DH);
    constexpr bool kQRegs = NQ * DH <= 256;  // Q fragments in registers (else read from shared memory)
    constexpr int OT = 2 * NQ;              // accumulator tiles of a 32-element block
    using St = State<NR, NP>;
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ __align__(128) uint8_t smem[];
    uint2 *const s_q = reinterpret_cast<uint2 *>(smem + Lay::q);        // [NQ][DH/16][32]
    uint2 *const s_p = reinterpret_cast<uint2 *>(smem + Lay::p);            // [pages][NQ][32]
    uint2 *const s_spread = reinterpret_cast<uint2 *>(smem + Lay::spread);  // [pages][DH/16][4] x 4 tokens
    float *const s_half = reinterpret_cast<float *>(smem + Lay::half);
    float *const s_max = reinterpret_cast<float *>(smem + Lay::max);  // [rows][8 warps]
    float *const s_sum = reinterpret_cast<float *>(smem + Lay::sum);  // [rows][8 warps]
    float *const s_cq = reinterpret_cast<float *>(smem + Lay::cq);    // raw score -> log2 units
    int *const s_lim = reinterpret_cast<int *>(smem + Lay::lim);      // last key of a row
    int *const s_nan = reinterpret_cast<int *>(smem + Lay::nan);      // [chunk parity][DH/16] first NaN key of an element block
    volatile int *const s_bad = reinterpret_cast<int *>(smem + Lay::bad);  // [chunk parity] 1 + the last chunk with a bad block id
    volatile int *const s_flags = reinterpret_cast<int *>(smem + Lay::flags);  // [0] gave up [1] a copy for all to see
    int32_t *const s_pre = reinterpret_cast<int32_t *>(smem + Lay::pre);
    int32_t *const s_weight = s_pre + p.num_tiles + 1;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int G = p.group, hkv = p.hkv;
    enum { kFullK, kFullV, kEmptyK, kEmptyV };
    auto bar = [&](int i) { return smem_addr(smem + Lay::bars + 8 * i); };
    auto wait = [&](int i, int parity) { return wait_bar(bar(i), parity, s_flags, p.err, i, p.wait_ns); };

    // the work: chunks of the valid requests
    if (tid < 2 * (DH / 16))
        s_nan[tid] = 0x7fffffff;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i)
            mbar_init(bar(i), 1);
        s_flags[0] = p.wait_ns == 0;  // no time at all: given up from the start
        s_flags[1] = 0;
        s_bad[0] = s_bad[1] = 0;
        fence_barrier_init();
    }
    // rows of a tile with bad lengths, or in a call without room for its records
    auto nan_rows = [&](const Meta &m, bool over) {
        if (!m.sane || (m.ok && !over))
            return;
        const int64_t first = (int64_t)m.qs * p.hq, n = (int64_t)m.qn * p.hq;
        for (int64_t k = tid; k < n * DH; k += kAllThreads)
            p.out[first * DH + k] = __ushort_as_bfloat16(0x7FC0);
        if (p.lse)
            for (int64_t k = tid; k < n; k += kAllThreads)
                p.lse[first + k] = __int_as_float(0x7FC00000);
    };
    int64_t lo, hi;  // chunks of this CTA
    if (p.per_group) {
        // Few: a CTA for each that the bounds allow, found without the others
        // (4 requests 8.2 us, dealt out 8.8).
        Chunk<DH> c;
        c.start(p, s_pre, blockIdx.x);
        const Meta m = meta_of(p, c.tile);
        if (c.kvh == 0 && c.lc == 0) {
            if (!m.ok && tid == 0)
                record_error(p.err, kErrBadMetadata, c.tile >> p.tile_shift);
            nan_rows(m, false);
        }
        lo = blockIdx.x;
        hi = lo + (m.ok && m.qn > 0 && c.lc < c.nch);
        if (hi == lo)
            return;
        __syncthreads();  // the barriers are set up
    } else {
        // chunks of a KV head of each tile, and their weights: pages, and what a
        // chunk costs without any
        int2 total;  // (the host's limits keep the sums below 2^31)
        block_exclusive_sums2<kAllThreads>(
            p.num_tiles, s_pre, s_weight, reinterpret_cast<int2 *>(smem + Lay::sums), total,
            [&](int tile, int &chunks, int &weight) {
                const Meta m = meta_of(p, tile);
                if (!m.ok && blockIdx.x == 0)
                    record_error(p.err, kErrBadMetadata, tile >> p.tile_shift);
                if (m.ok && m.qn > 0) {
                    chunks = (m.L + kChunk - 1) / kChunk;
                    weight = (m.L + 15) / 16 + kChunkCost * chunks;
                }
            });
        bool over = false;
        if (p.max_pages != INT64_MAX) {
            // pages of the requests: of their first tiles
            long long pages = 0;
            for (int b = lane; b < p.num_tiles >> p.tile_shift; b += 32) {
                const int i = b << p.tile_shift;
                pages += s_weight[i + 1] - s_weight[i] - kChunkCost * (s_pre[i + 1] - s_pre[i]);
            }
#pragma unroll
            for (int w = 16; w; w >>= 1)
                pages += __shfl_xor_sync(0xffffffffu, pages, w);
            over = pages > p.max_pages;
            if (over && blockIdx.x == 0 && tid == 0)
                record_error(p.err, kErrBudget, pages);
        }
        for (int i = blockIdx.x; i < p.num_tiles; i += gridDim.x)
            if (s_pre[i + 1] == s_pre[i] || over)
                nan_rows(meta_of(p, i), over);
        if (blockIdx.x == 0)  // for the folding kernel
            for (int i = tid; i <= p.num_tiles; i += kAllThreads)
                p.offsets[i] = over ? 0 : s_pre[i];
        if (over)
            return;
        // The chunks in order, a group's one after another, are cut where their
        // weights add up to equal shares: a CTA takes those that start in its share
        // (one each when there are no more chunks than CTAs).
        const int64_t T = (int64_t)total.x * hkv, W = (int64_t)total.y * hkv;
        lo = blockIdx.x, hi = lo + 1;
        if (T > (int64_t)gridDim.x) {
            // lane 0 of each warp finds the start of this share, lane 1 of the next
            constexpr int kFull = kPages + kChunkCost;  // weight of a whole chunk
            const int64_t cta = (int64_t)blockIdx.x + (lane & 1);
            int64_t start = T;
            if (cta < gridDim.x) {
                const int64_t at = div_floor(cta * W + gridDim.x - 1, gridDim.x);
                const int i = owner_of(s_weight, p.num_tiles, (int)div_floor(at, hkv));
                const int n = s_pre[i + 1] - s_pre[i], w = s_weight[i + 1] - s_weight[i];
                const int64_t rem = at - (int64_t)hkv * s_weight[i];
                const int h = (int)div_floor(rem, w), lc = ((int)(rem - (int64_t)h * w) + kFull - 1) / kFull;
                start = (int64_t)hkv * s_pre[i] + (int64_t)h * n + min(lc, n);
            }
            lo = __shfl_sync(0xffffffffu, start, 0);
            hi = __shfl_sync(0xffffffffu, start, 1);
        }
        if (lo >= hi || lo >= T)
            return;

    }
    const int chunks = (int)(hi - lo);
    if (warp == kWarps) {
        // The copying warp: a lane per page, the K records of a chunk when the
        // one before is past its first product, the V records when it is past
        // its second; the block ids are loaded a chunk ahead.  (Copies issued
        // by the computing warps held them up: 600 clocks of every 256 keys as
        // bulk copies, 1700 of every 512 as 16-byte cp.async.)
        static_assert(kPages <= 32, "one lane per page");
        const uint64_t policy = l2_policy_evict_first();
        const uint32_t dst = smem_addr(smem) + lane * REC;
        Chunk<DH> c;
        c.start(p, s_pre, lo);
        int id = lane < kPages ? c.id(lane) : 0;
        bool ok = true;
        int landing[2] = {0, 0};  // chunks whose K, and V, were asked for
        for (int k = 0; k < chunks && ok; ++k) {
            const bool exists = lane < kPages && c.has_page(lane);
            const bool go = exists && id >= 0 && (int64_t)id < p.num_blocks;
            const int n = __popc(__ballot_sync(0xffffffffu, go));
            const uint64_t off = (uint64_t)(uint32_t)id * p.block_stride + (uint64_t)(uint32_t)c.kvh * p.head_stride;
            const int b = c.tile >> p.tile_shift;
            const bool any_bad = __any_sync(0xffffffffu, exists && !go);
            if (k + 1 < chunks) {
                c.next(p, s_pre);
                id = lane < kPages ? c.id(lane) : 0;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (k > 0 && ok)
                    ok = wait(v ? kEmptyV : kEmptyK, (k - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                if (lane == 0) {
                    if (v == 0 && any_bad) {
                        s_bad[k & 1] = k + 1;
                        record_error(p.err, kErrBadMetadata, b);
                    }
                    if (n)
                        mbar_arrive_expect_tx(bar(v ? kFullV : kFullK), n * REC);
                    else
                        mbar_arrive(bar(v ? kFullV : kFullK));
                }
                __syncwarp();
                if (go)
                    bulk_copy(dst + v * kPages * REC, (v ? p.v : p.k) + off, REC, bar(v ? kFullV : kFullK), policy);
                landing[v] = k + 1;
            }
        }
        // Shared memory is given up when the last warp ends, and the computing
        // warps do not wait for copies once one of them has given up: this warp
        // stays until the last copies of both kinds have landed (each was asked
        // for when the one before it had been consumed).
        wait_bar_drain(bar(kFullK), (landing[0] - 1) & 1);
        wait_bar_drain(bar(kFullV), (landing[1] - 1) & 1);
        // When the computing warps are done: if a wait ran out of time, the sums
        // of this CTA's records are NaN, which makes their rows NaN.  (Groups of
        // one chunk have none; those not begun stay unwritten.)
        named_sync(2, kAllThreads);
        if (!s_flags[0])
            return;
        if (lane == 0)
            record_error(p.err, kErrTimeout, ((long long)blockIdx.x << 8) | 0xFF);
        static_assert(RN <= 32, "a lane per row");
#pragma unroll 1
        for (int k = 0; k < chunks; ++k)
            if (lane < p.rows) {
                float *const rec = p.records + (lo + k) * (int64_t)part_record_floats(p.rows, DH) + lane;
                __stcg(rec, 0.f);
                __stcg(rec + p.rows, __int_as_float(0x7FC00000));
            }
        return;
    }
    auto sync = [&]() { named_sync(1, kThreads); };  // the computing warps

    // this thread's place in the second product: element pairs c0 = 16*wd + g
    // and c0 + 8 of each 32-element block
    const int wd = HALVES ? warp % 4 : warp;
    const int token0 = 4 * (g >> 1) + (g & 1);  // token of fragment row g; row g + 8 is token0 + 2
    // rows of a thread's scores (columns of S^T) and of its state
    auto score_row = [&](int n, int i) { return 8 * n + 2 * t + i; };
    auto state_row = [&](int r) { return 8 * (r / 2) + 2 * t + r % 2; };
    // state pair i: its index among the DH/2 pairs
    auto state_pair = [&](int i) { return HALVES ? 16 * wd + 8 * (warp / 4) + g : 16 * (NE * wd + i / 2) + 8 * (i % 2) + g; };

    Chunk<DH> c;
    c.start(p, s_pre, lo);
    const uint32_t rec_hdr = (uint32_t)part_header_floats(p.rows), rec_size = (uint32_t)part_record_floats(p.rows, DH);

    // ------------------------------------------------ one chunk's state --
    auto chunk_state = [&](auto masked_tag, int step, St &st) -> int {
        const int parity = step & 1;
        const uint8_t *const stage = smem;
        constexpr bool MASKED = decltype(masked_tag)::value;  // some row does not see some key of the chunk
        const int key0 = c.lc * kChunk;
        const int npages = MASKED ? min(kPages, (c.L - key0 + 15) / 16) : kPages;
        uint2 qf[kQRegs ? NQ * (DH / 16) : 1];
        if constexpr (kQRegs) {
#pragma unroll
            for (int i = 0; i < NQ * (DH / 16); ++i)
                qf[i] = s_q[i * 32 + lane];
        }
        wait(kFullK, parity);
        // two accumulators per tile, for the even and the odd steps: one
        // chain of dependent products is latency bound
        float s[PPW][NQ][4];
#pragma unroll
        for (int j = 0; j < PPW; ++j) {
            float acc[2][NQ][4];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[j][n][i] = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        acc[k][n][i] = 0.f;
                }
            const int page = PPW * warp + j;
            if (MASKED && page >= npages)
                continue;
            // S^T = K . Q^T: thread t takes elements 32t..32t+31 of each 128
            const uint8_t *kr = stage + page * REC + token0 * (DH / 2) + 16 * t;
            const uint8_t *ks = stage + page * REC + CODES + token0 * (DH / 16) + 2 * t;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 ka = *reinterpret_cast<const uint4 *>(kr + 64 * b);
                const uint4 kb = *reinterpret_cast<const uint4 *>(kr + DH + 64 * b);
                const uint32_t sa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(ks + 8 * b));
                const uint32_t sb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(ks + DH / 8 + 8 * b));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
                const uint32_t fa[2] = {__byte_perm(sa, 0u, 0x1010), __byte_perm(sa, 0u, 0x3232)};
                const uint32_t fb[2] = {__byte_perm(sb, 0u, 0x1010), __byte_perm(sb, 0u, 0x3232)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x[4], y[4];
                    e2m1x8_to_f16x2(wa[i], x);
                    e2m1x8_to_f16x2(wb[i], y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[k] = mul_f16x2(x[k], fa[i / 2]);
                        y[k] = mul_f16x2(y[k], fb[i / 2]);
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int step = n * (DH / 16) + 8 * b + 2 * i + k;
                            const uint2 q = kQRegs ? qf[kQRegs ? step : 0] : s_q[step * 32 + lane];
                            mma_f16(acc[k][n], x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1], q.x, q.y);
                        }
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[j][n][i] = acc[0][n][i] + acc[1][n][i];
            if (MASKED) {
                const int key = key0 + 16 * page + token0;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key + (i < 2 ? 0 : 2) > s_lim[score_row(n, i % 2)])
                            s[j][n][i] = -INFINITY;
            }
        }
        if (MASKED) {
            // pages that do not exist: no key
#pragma unroll
            for (int j = 0; j < PPW; ++j)
                if (PPW * warp + j >= npages)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[j][n][i] = -INFINITY;
        }
        // largest raw score of each row, over the warp's keys
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = fmaxf(s[0][n][i], s[0][n][2 + i]);
#pragma unroll
                for (int j = 1; j < PPW; ++j)
                    x = max3f(x, s[j][n][i], s[j][n][2 + i]);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1)
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
                if (g == 0)
                    s_max[score_row(n, i) * kWarps + warp] = x;
            }
        int gave_up = 0;  // of thread 0
        if (tid == 0)
            s_flags[1] = gave_up = s_flags[0];  // any thread may set [0] at any time
        sync();  // A: maxima written; K is consumed
        // read between A and B, so that every thread reads the same
        const int bad = s_flags[1] ? -1 : s_bad[parity] == step + 1;
        if (tid < DH / 16)
            s_nan[(parity ^ 1) * (DH / 16) + tid] = 0x7fffffff;  // for the next chunk
        // (after a wait that gave up the copies may not have landed: nothing may
        // be asked for in their place)
        if (tid == 0 && !gave_up)
            mbar_arrive(bar(kEmptyK));
        const bool have_v = wait(kFullV, parity);
#pragma unroll
        for (int j = 0; j < PPW; ++j) {
            const int page = PPW * warp + j;
            if (MASKED && page >= npages)
                break;
            // the page's V scales: lane = (element block lane/4 + 8b, tokens 4*(lane%4)..+3)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t w = reinterpret_cast<const uint32_t *>(stage + (kPages + page) * REC + CODES)[32 * b + lane];
                uint32_t s01 = e4m3x2_to_f16x2(w), s23 = e4m3x2_to_f16x2(w >> 16);
                if (MASKED) {
                    // tokens no row sees count as zero whatever their bytes; a
                    // NaN that only some rows see is given to those rows below
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + 16 * page + 4 * t + i;
                        const bool gone = key >= c.L, nan = ((w >> (8 * i)) & 0x7fu) == 0x7fu;
                        if (gone || (nan && key > c.seen)) {
                            (i < 2 ? s01 : s23) &= i % 2 ? 0x0000ffffu : 0xffff0000u;
                            if (!gone)
                                atomicMin(s_nan + parity * (DH / 16) + 8 * b + g, key);
                        }
                    }
                }
                s_spread[(page * (DH / 16) + 8 * b + g) * 4 + t] = make_uint2(s01, s23);
            }
        }
        float l[NQ][2], mrow[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float pr[PPW][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = score_row(n, i);
                const float4 u = *reinterpret_cast<const float4 *>(s_max + r * kWarps);
                const float4 v = *reinterpret_cast<const float4 *>(s_max + r * kWarps + 4);
                const float cq = s_cq[r];
                const float top = fmaxf(max3f(u.x, u.y, max3f(u.z, u.w, v.x)), max3f(v.y, v.z, v.w));
                mrow[n][i] = top * cq;
                // The maximum is taken off the raw score: p is then 2^kShift at
                // the largest key and never above.  (Off the score in log2
                // units, the two roundings of a product of 2^24 and more are
                // whole units, and p leaves f16's range.)
                const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int j = 0; j < PPW; ++j) {
                    pr[j][i] = ex2(__fmaf_rn(s[j][n][i] - ref, cq, kShift));  // 0 for keys left out
                    pr[j][2 + i] = ex2(__fmaf_rn(s[j][n][2 + i] - ref, cq, kShift));
                }
                l[n][i] = pr[0][i] + pr[0][2 + i];
#pragma unroll
                for (int j = 1; j < PPW; ++j)
                    l[n][i] += pr[j][i] + pr[j][2 + i];
            }
            // P^T fragments: after the transpose thread (g, t) holds column
            // g's keys in pairs, tokens 4t, 4t+1 (x) and 4t+2, 4t+3 (y)
#pragma unroll
            for (int j = 0; j < PPW; ++j) {
                const int page = PPW * warp + j;
                const uint32_t x = movmatrix(pack_f16x2(pr[j][0], pr[j][1])), y = movmatrix(pack_f16x2(pr[j][2], pr[j][3]));
                s_p[(page * NQ + n) * 32 + lane] = make_uint2(x, y);
            }
        }
        sync();  // B: P and scales written, V visible
        float o[NE][OT][4];
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int n = 0; n < OT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[e][n][i] = 0.f;
        const int first = HALVES ? warp / 4 * (kPages / 2) : 0;
        const int last = HALVES ? min(npages, first + kPages / 2) : npages;
        auto page_product = [&](int page) {
            const uint8_t *vr = stage + (kPages + page) * REC + (16 * NE * wd + g) * 16 + 4 * t;
            uint2 pf[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                pf[n] = s_p[(page * NQ + n) * 32 + lane];
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                // pairs c0 (element block 2*(NE*wd + e)) and c0 + 8 (the next block), tokens 4t..4t+3
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(vr + e * 256 + h * 128);
                    const uint2 f = s_spread[(page * (DH / 16) + 2 * (NE * wd + e) + h) * 4 + t];
                    uint32_t x[4];
                    e2m1x8_to_f16x2(w, x);  // token 4t + i: (even, odd) element
                    const uint32_t a0 = mul_f16x2(__byte_perm(x[0], x[1], 0x5410), f.x);  // even, tokens 4t, 4t+1
                    const uint32_t a1 = mul_f16x2(__byte_perm(x[0], x[1], 0x7632), f.x);  // odd
                    const uint32_t a2 = mul_f16x2(__byte_perm(x[2], x[3], 0x5410), f.y);  // even, tokens 4t+2, 4t+3
                    const uint32_t a3 = mul_f16x2(__byte_perm(x[2], x[3], 0x7632), f.y);
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        mma_f16(o[e][2 * n + h], a0, a1, a2, a3, pf[n].x, pf[n].y);
                }
            }
        };
        if constexpr (MASKED) {
#pragma unroll 1
            for (int page = first; page < last; ++page)
                page_product(page);
        } else {
#pragma unroll(NQ * NE == 1 ? 4 : 2)
            for (int i = 0; i < (HALVES ? kPages / 2 : kPages); ++i)
                page_product(first + i);
        }
        // accumulators by element pair: pr[i][k], i = 0 (c0) or 1 (c0 + 8) of
        // each 32-element block; k: N tile, parity, row
        constexpr int F = RN / 2;  // floats of a pair
        float pr[2 * NE][F];
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < F; ++k)
                    pr[2 * e + i][k] = o[e][2 * (k / 4) + i][k % 4];
        // row sums over the warp's keys
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1)
                    l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], w);
                if (g == 0)
                    s_sum[score_row(n, i) * kWarps + warp] = l[n][i];
            }
        if constexpr (HALVES) {
            // warps 0-3 keep the pairs c0, 4-7 the pairs c0 + 8; the others' go
            // through shared memory
            const int keep = warp / 4;
#pragma unroll
            for (int k = 0; k < F; ++k)
                s_half[k * kThreads + (tid ^ 128)] = keep ? pr[0][k] : pr[1][k];
        }
        // (before C: after it a new group's limits may be written)
        uint32_t nan_rows = 0;  // bit i * NR + r
        if constexpr (MASKED) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int k = s_nan[parity * (DH / 16) + state_pair(i) / 8];
                if (k != 0x7fffffff)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        nan_rows |= (uint32_t)(s_lim[state_row(r)] >= k) << (i * NR + r);
            }
        }
        sync();  // C: sums and halves written; V is consumed
        if (tid == 0 && have_v)
            mbar_arrive(bar(kEmptyV));
        if constexpr (HALVES) {
            const int keep = warp / 4;
#pragma unroll
            for (int k = 0; k < F; ++k) {
                const float own = keep ? pr[1][k] : pr[0][k], other = s_half[k * kThreads + tid];
                pr[0][k] = keep ? other + own : own + other;  // the first half of the pages first
            }
        }
        // the thread's state: rows' maxima and sums, pairs of elements
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            st.m[r] = mrow[r / 2][r % 2];
            const float *ss = s_sum + state_row(r) * kWarps;
            const float4 u = *reinterpret_cast<const float4 *>(ss), v = *reinterpret_cast<const float4 *>(ss + 4);
            st.l[r] = ((u.x + u.y) + (u.z + u.w)) + ((v.x + v.y) + (v.z + v.w));
#pragma unroll
            for (int i = 0; i < NP; ++i)
                st.o[i][r] = make_float2(pr[i][4 * (r / 2) + r % 2], pr[i][4 * (r / 2) + 2 + r % 2]);
        }
        if (MASKED && nan_rows) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (nan_rows >> (i * NR + r) & 1)
                        st.o[i][r] = make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
        }
        return bad;
    };

    // records: m, l and the element pairs of this thread's rows
    const int pair_zero = state_pair(0) == 0;  // this thread also speaks for the row's m and l
    auto write_record = [&](float *rec, const St &st, int rv) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = state_row(r);
            if (row >= rv)
                continue;
            if (pair_zero) {
                __stcg(rec + row, st.m[r]);
                __stcg(rec + p.rows + row, st.l[r]);
            }
#pragma unroll
            for (int i = 0; i < NP; ++i)
                __stcg(reinterpret_cast<float2 *>(rec + (rec_hdr + (uint32_t)(row * DH + 2 * state_pair(i)))), st.o[i][r]);
        }
    };
    auto output_pair = [&](int row, int pair, float2 o, float m, float l) {
        const int64_t at = (int64_t)(c.qs + row / G) * p.hq + c.kvh * G + row % G;
        const float f = __frcp_rn(l) * p.v_scale;
        reinterpret_cast<uint32_t *>(p.out + at * DH)[pair] = pack_bf16x2(o.x * f, o.y * f);
        if (pair == 0 && p.lse)
            p.lse[at] = lse_of(m, l * 0x1p-15f);
    };
    for (int step = 0; step < chunks; ++step) {
        const bool first_chunk = step == 0;
        if (!first_chunk)
            c.next(p, s_pre);
        if (first_chunk || c.lc == 0) {
            // a new group: its rows, scaled to [1, 2) by a power of two, in
            // fragment order (the previous group's readers are past a barrier)
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
                const int slot = 8 * k + warp, r = slot;
                const bool valid = r < c.qn * G;
                const int tok = valid ? r / G : 0;
                const uint2 *src = reinterpret_cast<const uint2 *>(p.q + (int64_t)(c.qs + tok) * p.q_tok_stride +
                                                                   (int64_t)(c.kvh * G + (valid ? r - tok * G : 0)) * DH);
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
                if (lane == 0) {
                    s_cq[slot] = fmaxf(1e-37f, fminf(p.score_scale * __int_as_float((127 + e) << 23), 3e38f));
                    s_lim[slot] = c.seen + (valid ? tok : c.qn - 1);
                }
            }
            sync();
        }
        St st;
        const bool masked = c.lc * kChunk + kChunk > c.seen + 1;
        const int bad = masked ? chunk_state(std::true_type{}, step, st) : chunk_state(std::false_type{}, step, st);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            if (bad != 0)
                st.l[r] = __int_as_float(0x7FC00000);
            if (st.l[r] != st.l[r] && st.m[r] == -INFINITY)
                st.m[r] = 0.f;  // a NaN state must not pass for an empty one
        }

        const int rv = c.qn * G;
        if (c.nch > 1) {
            write_record(p.records + (lo + step) * (int64_t)rec_size, st, rv);
        } else {
            // (any thread that gave up on this chunk did before its last barrier)
            const bool gone = s_flags[0];
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (state_row(r) < rv)
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        output_pair(state_row(r), state_pair(i), st.o[i][r], st.m[r],
                                    gone ? __int_as_float(0x7FC00000) : st.l[r]);
        }
        if (bad < 0)
            break;  // a wait ran out of time
    }
    bar_arrive(2, kAllThreads);
}

// Folds the chunk records of the groups with several chunks.  Bound by round
// trips to L2: a warp folds 128 * V elements of a row over a span, 16 / V
// records in flight; all parts, rows and spans (up to 16 warps to a CTA) side by
// side; then one warp folds the spans of a part.  V is 1 while an SM is there
// for every CTA, else the whole row (head dim 512, 4 requests 12.0 us against
// 14.0, but 64 of them 58.6 against 51.5).  131k
// keys on 8 KV heads: 32.2 us with spans of 32 chunks, 31.6 of 8, 30.1 of 16.
constexpr int kFoldThreads = 512;  // at most
// Up to this many tiles a CTA sums the chunks before its own while it waits for
// the attention kernel; above, it reads the sums that one has left (a round trip
// more, but 2048 tiles cost every CTA as many loads).
constexpr int kFoldSums = 256;

template <int DH, int V>  // V: float4 of a lane
__global__ void __launch_bounds__(kFoldThreads) quant_fold_kernel(const Params p, int SW)
{
    constexpr int PARTS = DH / (128 * V);
    __shared__ __align__(16) float s_state[kFoldThreads / 32][128 * V + 4];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int item = blockIdx.y * (blockDim.x / 32 / SW) + warp / SW, slot = warp % SW;
    const int row = item / PARTS, col = item % PARTS * 128 * V + 4 * lane;
    const int tile = blockIdx.x / p.hkv, kvh = blockIdx.x - tile * p.hkv;
    // The metadata's writers are done (the attention kernel waited for them
    // before it let this one start), so it is read while that one still runs.
    const Meta m = meta_of(p, tile);
    const int nch = m.ok && m.qn > 0 ? (m.L + chunk_keys(DH) - 1) / chunk_keys(DH) : 0;
    int c0 = 0;
    if (nch > 1 && p.per_group == 0 && p.num_tiles <= kFoldSums) {
        __shared__ int s_sum[kFoldThreads / 32];
        for (int i = threadIdx.x; i < tile; i += blockDim.x) {
            const Meta x = meta_of(p, i);
            c0 += x.ok && x.qn > 0 ? (x.L + chunk_keys(DH) - 1) / chunk_keys(DH) : 0;
        }
        c0 = __reduce_add_sync(0xffffffffu, c0);
        if (lane == 0)
            s_sum[warp] = c0;
        __syncthreads();
        c0 = 0;
        for (int w = 0; w < blockDim.x / 32; ++w)
            c0 += s_sum[w];
    }
    griddep_wait();
    griddep_launch_dependents();
    if (nch <= 1)  // none, or written already
        return;
    if (p.per_group == 0 && p.num_tiles > kFoldSums)
        c0 = __ldcg(p.offsets + tile);
    if (p.max_pages != INT64_MAX && __ldcg(p.offsets + p.num_tiles) == 0)
        return;  // no room for the records
    const bool live = row < m.qn * p.group;
    const uint32_t hdr = (uint32_t)part_header_floats(p.rows), size = (uint32_t)part_record_floats(p.rows, DH);
    const int64_t first_record =
        p.per_group ? (int64_t)blockIdx.x * p.per_group : (int64_t)p.hkv * c0 + (int64_t)kvh * nch;
    const float *rec = p.records + first_record * size + (live ? row : 0);
    const float *ro = rec - (live ? row : 0) + (hdr + (uint32_t)((live ? row : 0) * DH + col));
    State<1, 2 * V> acc;
    acc.clear();
    const int spans = (nch + kSpan - 1) / kSpan;
    for (int s0 = 0; s0 < spans; s0 += SW) {
        State<1, 2 * V> st;
        st.clear();
        const int first = (s0 + slot) * kSpan, n = live ? min(kSpan, nch - first) : 0;
        // lane k has record k's maximum and sum; the factors are known at once
        const int64_t span_at = (int64_t)first * size;
        float mk = -INFINITY, lk = 0.f;
        if (lane < n) {
            mk = __ldcg(rec + span_at + (int64_t)lane * size);
            lk = __ldcg(rec + span_at + (int64_t)lane * size + p.rows);
        }
        constexpr int U = 16 / V;  // records in flight
        float f = 0.f;
        for (int k0 = 0; k0 < n; k0 += U) {
            float4 x[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + u >= n)
                    break;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    x[u][i] = __ldcg(reinterpret_cast<const float4 *>(ro + span_at + (int64_t)(k0 + u) * size + 128 * i));
            }
            if (k0 == 0) {
                float m = mk;
#pragma unroll
                for (int w = 1; w < kSpan; w <<= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                m = __shfl_sync(0xffffffffu, m, 0);
                f = ex2(mk - (m == -INFINITY ? 0.f : m));  // 0 for an empty chunk
                float l = lk * f;
#pragma unroll
                for (int w = 1; w < kSpan; w <<= 1)
                    l += __shfl_xor_sync(0xffffffffu, l, w);
                st.m[0] = m;
                st.l[0] = __shfl_sync(0xffffffffu, l, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + u >= n)
                    break;
                const float fu = __shfl_sync(0xffffffffu, f, k0 + u);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float2 &a = st.o[2 * i][0], &b = st.o[2 * i + 1][0];
                    a = make_float2(__fmaf_rn(x[u][i].x, fu, a.x), __fmaf_rn(x[u][i].y, fu, a.y));
                    b = make_float2(__fmaf_rn(x[u][i].z, fu, b.x), __fmaf_rn(x[u][i].w, fu, b.y));
                }
            }
        }
        if (SW == 1) {
            acc.fold(st);
            continue;
        }
        // the spans of this pass, in order, by the part's first warp
#pragma unroll
        for (int i = 0; i < V; ++i)
            *reinterpret_cast<float4 *>(&s_state[warp][4 * lane + 128 * i]) =
                make_float4(st.o[2 * i][0].x, st.o[2 * i][0].y, st.o[2 * i + 1][0].x, st.o[2 * i + 1][0].y);
        if (lane == 0) {
            s_state[warp][128 * V] = st.m[0];
            s_state[warp][128 * V + 1] = st.l[0];
        }
        __syncthreads();
        if (slot == 0)
            for (int k = 0; k < SW && s0 + k < spans; ++k) {
                const float *t = s_state[warp + k];
                State<1, 2 * V> x;
                x.m[0] = t[128 * V];
                x.l[0] = t[128 * V + 1];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float4 v = *reinterpret_cast<const float4 *>(t + 4 * lane + 128 * i);
                    x.o[2 * i][0] = make_float2(v.x, v.y);
                    x.o[2 * i + 1][0] = make_float2(v.z, v.w);
                }
                acc.fold(x);
            }
        __syncthreads();
    }
    if (!live || slot != 0)
        return;
    const int64_t at = (int64_t)(m.qs + row / p.group) * p.hq + kvh * p.group + row % p.group;
    const float f = __frcp_rn(acc.l[0]) * p.v_scale;
#pragma unroll
    for (int i = 0; i < V; ++i)
        *reinterpret_cast<uint2 *>(p.out + at * DH + col + 128 * i) =
            make_uint2(pack_bf16x2(acc.o[2 * i][0].x * f, acc.o[2 * i][0].y * f),
                       pack_bf16x2(acc.o[2 * i + 1][0].x * f, acc.o[2 * i + 1][0].y * f));
    if (col == 0 && p.lse)
        p.lse[at] = lse_of(acc.m[0], acc.l[0] * 0x1p-15f);
}

template <int DH, int RN>
cudaError_t set_attributes()
{
    const int bytes = (int)Layout<DH, RN>::bytes(kQuantMaxTiles);
    return cudaFuncSetAttribute(quant_attn_kernel<DH, RN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bytes > kSmemAlone ? bytes : kSmemAlone);
}

static int rows_capacity(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32; }

// CTAs of the grid: one wave, fewer when there are fewer chunks.
static int64_t grid_of(int dh, int rn, int64_t max_chunks)
{
    const int64_t wave = (int64_t)kGridSms * ctas_per_sm(dh, rn);
    return max_chunks < 1 ? 1 : (max_chunks < wave ? max_chunks : wave);
}

static int64_t chunks_of(int dh, int32_t len) { return ((int64_t)len + chunk_keys(dh) - 1) / chunk_keys(dh); }
// log2 of the tiles that a request's share of the numbering has room for.
static int tile_shift_of(int tiles)
{
    int shift = 0;
    while (1 << shift < tiles)
        ++shift;
    return shift;
}

// Chunks of all groups at most, of tiles without tokens among them (a CTA for
// each chunk that the bounds allow numbers its records that way).
static int64_t max_chunks_of(int32_t num_seqs, int32_t tiles, int32_t hkv, int dh, int32_t max_seq_len,
                             int64_t max_pages)
{
    int64_t per_head = (int64_t)num_seqs * chunks_of(dh, max_seq_len);
    if (max_pages > 0 && max_pages / chunk_pages(dh) + num_seqs < per_head)
        per_head = max_pages / chunk_pages(dh) + num_seqs;  // whole ones, and one in part a request
    return (per_head << tile_shift_of(tiles)) * hkv;
}

template <int DH, int RN>
cudaError_t launch(const Params &p, cudaStream_t stream, int64_t grid)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kAllThreads);
    cfg.dynamicSmemBytes = Layout<DH, RN>::bytes(p.num_tiles);
    // no more CTAs than SMs: one to each (4 requests at head dim 256 10.6 us,
    // where some share an SM 12.1)
    if (grid <= kGridSms && cfg.dynamicSmemBytes < kSmemAlone)
        cfg.dynamicSmemBytes = kSmemAlone;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, quant_attn_kernel<DH, RN>, p);
    const int64_t chunks = chunks_of(DH, p.max_seq_len);
    if (e != cudaSuccess || chunks <= 1)
        return e;
    int sw = 1;  // spans of a part side by side
    while (sw < kFoldThreads / 32 && sw * kSpan < chunks)
        sw *= 2;
    const int most = kFoldThreads / 32 / sw, parts = p.rows * (DH / 128);
    const bool split = (int64_t)p.num_tiles * p.hkv * ((parts + most - 1) / most) <= kGridSms;
    const int items = split ? parts : p.rows, some = items < most ? items : most;
    cfg.gridDim = dim3((unsigned)(p.num_tiles * p.hkv), (unsigned)((items + some - 1) / some));
    cfg.blockDim = dim3(32 * sw * some);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, split ? quant_fold_kernel<DH, 1> : quant_fold_kernel<DH, DH / 128>, p, sw);
}

}  // namespace qa

// The tiles' offsets, then the records.
static size_t offset_bytes(int32_t num_tiles) { return (((size_t)num_tiles + 1) * 4 + 255) / 256 * 256; }

int quant_attn_tiles(int32_t num_seqs, int32_t num_kv_heads, int head_dim, int group, int32_t max_query_len,
                     int32_t max_seq_len)
{
    const int tokens = (head_dim == 512 ? 16 : 32) / group;
    if (tokens == 0)
        return 0;
    const int64_t tiles = max_query_len <= tokens ? 1 : ((int64_t)max_query_len + tokens - 1) / tokens;
    if (tiles > kQuantMaxTiles || ((int64_t)num_seqs << qa::tile_shift_of((int)tiles)) > kQuantMaxTiles)
        return 0;
    if (tiles > 2) {
        // Estimates in ns: a wave of chunks here, against a start and the keys
        // that one CTA of the BF16 attention takes one after another (with one
        // tile of 128 rows to an SM or less; where it has more, or splits the
        // keys, or the read-back is long, it takes longer).  Measured, direct
        // against read-back, 8 query and 2 KV heads unless said: 128 tokens of
        // 4096 keys 23 us to 59, 128 of 512 keys in 4 requests 13 to 66, 64 of
        // 1024 in 8 requests 25 to 26, 40 of 120 in 32 requests 28 to 18; 64 of
        // 1024 with 32 and 8 heads in 4 requests 45 to 27, of 4096 in one 36 to
        // 59; head dim 256, 157 of 4521 with 2 and 1 heads 23 to 81; head dim
        // 512, 27 of 4764 with 8 and 1 heads 31 to 139.
        const int64_t per_key = head_dim == 128 ? 12 : (head_dim == 256 ? 16 : 27);
        const int64_t wave = (int64_t)qa::kGridSms * qa::ctas_per_sm(head_dim, head_dim == 512 ? 16 : 32);
        const int64_t chunks = num_seqs * num_kv_heads * tiles * qa::chunks_of(head_dim, max_seq_len);
        if (9000 * ((chunks + wave - 1) / wave) > 12000 + per_key * max_seq_len)
            return 0;
    }
    return (int)tiles;
}

size_t quant_attn_bytes(int32_t num_seqs, int tiles, int32_t num_kv_heads, int32_t head_dim, int rows,
                        int32_t max_seq_len, int64_t max_pages)
{
    return offset_bytes(num_seqs << qa::tile_shift_of(tiles)) +
           (size_t)qa::max_chunks_of(num_seqs, tiles, num_kv_heads, head_dim, max_seq_len, max_pages) *
               (size_t)part_record_floats(rows, head_dim) * 4;
}

cudaError_t launch_quant_attention(const QuantAttnArgs &a, ErrState *err, cudaStream_t stream, char *info,
                                   size_t info_len)
{
    qa::Params p{};
    p.k = a.pool.k;
    p.v = a.pool.v;
    p.block_stride = (uint32_t)a.pool.block_stride;
    p.head_stride = (uint32_t)a.pool.head_stride;
    p.num_blocks = a.pool.num_blocks;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.q_tok_stride = a.q_tok_stride;
    p.num_q_tokens = a.num_q_tokens;
    p.block_tables = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.qsl = a.query_start_loc;
    p.max_blocks = a.max_blocks;
    p.hq = a.num_q_heads;
    p.hkv = a.pool.num_kv_heads;
    p.group = p.hq / p.hkv;
    p.max_query_len = a.max_query_len;
    p.max_seq_len = a.max_seq_len;
    const int tiles = quant_attn_tiles(a.num_seqs, p.hkv, a.pool.head_dim, p.group, a.max_query_len, a.max_seq_len);
    p.tile_shift = qa::tile_shift_of(tiles);
    p.tile_tokens = (a.max_query_len + tiles - 1) / tiles;
    p.num_tiles = a.num_seqs << p.tile_shift;
    p.rows = p.tile_tokens * p.group;
    p.score_scale = a.scale * 1.4426950408889634f * a.pool.k_scale;
    p.v_scale = a.pool.v_scale;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.err = err;
    p.wait_ns = fold_wait_limit_ns();
    p.max_pages = a.max_pages > 0 ? a.max_pages : INT64_MAX;
    const int64_t max_chunks =
        qa::max_chunks_of(a.num_seqs, tiles, p.hkv, a.pool.head_dim, p.max_seq_len, a.max_pages);
    const int rn = qa::rows_capacity(p.rows);
    int64_t grid = qa::grid_of(a.pool.head_dim, rn, max_chunks);
    const int64_t per_group = qa::chunks_of(a.pool.head_dim, p.max_seq_len);
    const bool limited = a.max_pages > 0 && a.max_pages < a.num_seqs * (((int64_t)p.max_seq_len + 15) / 16);
    if (!limited && per_group > 0 &&
        (int64_t)p.num_tiles * p.hkv * per_group <= (int64_t)qa::kGridSms * qa::ctas_per_sm(a.pool.head_dim, rn)) {
        p.per_group = (int32_t)per_group;
        grid = (int64_t)p.num_tiles * p.hkv * per_group;
        p.max_pages = INT64_MAX;
    }
    p.offsets = static_cast<int32_t *>(a.workspace);
    p.records = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + offset_bytes(p.num_tiles));
    cudaError_t e = cudaErrorNotSupported;
    auto go = [&](auto fn) { e = fn(p, stream, grid); };
    switch (a.pool.head_dim) {
    case 128:
        go(rn == 8    ? qa::launch<128, 8>
           : rn == 16 ? qa::launch<128, 16>
           : rn == 24 ? qa::launch<128, 24>
                      : qa::launch<128, 32>);
        break;
    case 256:
        go(rn == 8 ? qa::launch<256, 8> : rn == 16 ? qa::launch<256, 16> : rn == 24 ? qa::launch<256, 24> : qa::launch<256, 32>);
        break;
    case 512:
        go(rn == 8 ? qa::launch<512, 8> : qa::launch<512, 16>);
        break;
    }
    snprintf(info, info_len, "quant attention direct dh=%d tiles=%d rows=%d/%d grid=%lld chunks<=%lld", a.pool.head_dim,
             tiles, p.rows, rn, (long long)grid, (long long)max_chunks);
    return e;
}

cudaError_t init_quant_attention_attributes()
{
    cudaError_t e;
    if ((e = qa::set_attributes<128, 8>()) != cudaSuccess || (e = qa::set_attributes<128, 16>()) != cudaSuccess ||
        (e = qa::set_attributes<128, 32>()) != cudaSuccess || (e = qa::set_attributes<256, 8>()) != cudaSuccess ||
        (e = qa::set_attributes<256, 16>()) != cudaSuccess || (e = qa::set_attributes<256, 32>()) != cudaSuccess ||
        (e = qa::set_attributes<512, 8>()) != cudaSuccess || (e = qa::set_attributes<128, 24>()) != cudaSuccess ||
        (e = qa::set_attributes<256, 24>()) != cudaSuccess)
        return e;
    return qa::set_attributes<512, 16>();
}

}  // namespace pa

// pa_paged_attention_scored for many rows: prompts and chunks of them, on tcgen05.
//
// A group is one (request, KV head, NT tiles of 128 rows); row r of a group is
// query head r % G of query token r / G, so the heads that share a KV head share
// its tiles.  The items of a group are the tiles of 128 keys that some row sees;
// the items of all groups are dealt out as one wave of equal contiguous ranges, a
// CTA to an SM.  (A causal prompt's groups differ by a factor of its tiles:
// 4096 tokens of 8 and 2 heads are 128 groups of 1 to 32 items, 16.5 on
// average, and a group to a CTA would leave the time at the longest one's.)  A
// group that lies wholly in a range goes straight to the output; a part of one
// becomes a record (maximum, sum, unnormalised output), folded by a second kernel.
//
// Two score buffers in tensor memory keep the tensor pipe busy: with two row
// tiles (head dim 128) each has its own, and the softmax of one runs beside the
// products of the other; with one (head dims 256 and 512, or few rows) the key
// tiles take them in turn.  The order on the pipe is QK(0), QK(1), then PV(i),
// QK(i+2): probabilities overwrite their scores in tensor memory, and products
// issued by one thread run in order.
//   warp 0      copies units of 128 keys by 128 columns (32 KB, a TMA box for each
//               page and 64 columns) into a ring, in the order of their use
//   warp 1      issues the products (one thread)
//   warps 2, 3  Q of a group, once the products of the group before have read theirs:
//               TMA boxes where a row tile is whole tokens (G divides 128), else
//               row by row (63.4 us instead of 61.2 at the prompt below)
//   warps 4-7, 8-11   softmax of one score buffer each, a row to a thread, and
//               the output at a group's end
// Head dim 512: the output's halves are two groups, each with all of the scores
// (tensor memory holds 256 columns of output beside the scores): three halves of
// the products of a whole one instead of two, and no exchange.
//
// Measured: a prompt of 4096 tokens, 8 query and 2 KV heads of 128, capped: 62.5
// us, 0.55 PFLOP/s of the products that causality leaves (plain 56, with a window of
// 1024 40, with a bias 74, with both cap and bias 95; 80 with scores that are mostly
// above 3/8 of the cap, which then cost two exponentials and a reciprocal instead of
// one exponential: spread 4 under a cap of 30 instead of 50); at head dim 256 and 512
// (one KV head) 110 and 279; a prompt of 8192 tokens
// of five documents behind a prefix, 16 and 2 heads of 256, a bias by distance:
// 274 us, 0.55 PFLOP/s of those that the documents leave.  What bounds it is the
// chain of a step (scores, softmax, products), not the tensor pipe: a pair of
// 128-key tiles takes 4.9 k cycles at head dim 128, its products 2.1 k, a tile's
// softmax 2.0 to 2.4 k (of them 1.4 k issue slots where it is capped); at head dim
// 256 a tile takes 6.4 k, of which the issuing thread waits 2.3 k for K and V (128
// KB from L2, 6 TB/s over the GPU) and its products take 3.1 k.  Starting a CTA and
// its first scores take 15 k more, 12 percent of the prompt's time.  Slower when
// tried, against 61 us for the capped prompt then: two issuing threads (69 us),
// 16 softmax warps (74), tiles of 64 keys (79), probabilities in shared memory so
// that the next scores need not wait for the products (69: each product then
// reads both operands there, 950 cycles instead of 800).
#pragma once
#include "pa_scan.cuh"
#include "pa_scored.h"

namespace pa {

constexpr int kTileThreads = 384;
constexpr int kTileKeys = 128;
constexpr int kUnitBytes = kTileKeys * 256;  // 128 keys by 128 columns
// What a group costs beside its items, in items: it is dealt out with them, at
// the group's start.  (With two row tiles 1, 2, 3 and 4 took 61.4, 60.1, 62.3 and
// 64.7 us for the prompt above; with one 274.9, 281.3, 293.8 and 305.6 for the
// documents.)
template <int NT>
constexpr int kGroupSetup = NT == 2 ? 2 : 1;

// How a score becomes an exponent.
enum ScoreMode : int {
    kModePlain = 0,   // scaled
    kModeCapped = 1,  // capped, and the cap small enough to need no running maximum
    kModeAny = 2,     // with a bias, capped or not; the cap at most kCapNarrow
    kModeWide = 3,    // with or without a bias; the cap above that
};

template <int DH, int NT>
struct TileCfg {
    static constexpr int kSplit = DH == 512 ? 2 : 1;  // groups that share a row tile's columns
    static constexpr int kUnitsK = DH / 128, kUnitsV = DH / 128 / kSplit;
    static constexpr int kCols = DH / kSplit;         // output columns of a group
    static constexpr int kQBytes = NT * 128 * DH * 2;
    // The output passes through shared memory, 64 columns of a warp's rows at a
    // time (a row to a thread stores 16 bytes to 32 lines at once); at head dim
    // 512 there is no room for that.
    static constexpr int kOutBytes = DH == 512 ? 0 : 32 * 1024;
    static constexpr int kStages = (224 * 1024 - kQBytes - kOutBytes) / kUnitBytes;
    static constexpr int kOCol = 256;                 // tensor-memory column of the output
    static_assert(NT * kCols <= 256 && kStages >= 3, "tensor and shared memory");
};

struct TileWork {
    int4 *tails;       // [ctas] the group that goes on past a CTA's range and began in it:
                       // request, row tile, (KV head, part of the columns), CTAs that have a part; 0: none
    float *records;    // [2 * ctas] of record_floats
    int64_t record_floats;
    int32_t ctas, max_tiles;
    int32_t q_boxes;   // a tile's rows are whole tokens: Q by TMA boxes
};

// Floats of one row tile's record: m[128], l[128], then the output as [columns / 4][128 rows][4].
constexpr int64_t tile_record(int cols) { return 256 + (int64_t)cols * 128; }

constexpr int kTileSmall = 2048;  // barriers, flags, row exchange

template <int DH, int NT>
constexpr size_t tiles_smem()
{
    using C = TileCfg<DH, NT>;
    return 1024 + (size_t)C::kQBytes + (size_t)C::kStages * kUnitBytes + C::kOutBytes + kTileSmall;
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Row tiles of NT * 128 rows that a request's tokens form.
__device__ __forceinline__ int group_tiles(const ScoreParams &p, const ReqMeta &m, int rows)
{
    return m.ok ? (int)(((int64_t)m.qn * p.group + rows - 1) / rows) : 0;
}

// tile_view of rows [r0, r1) by a whole warp (without `gaps`: where the range has some,
// pages in them are copied if their ids are good, and hidden like any other key; with
// their pages left out the copying warp's longer loop took the prompts one percent).
__device__ __forceinline__ TileView warp_tile_view(const ScoreParams &p, int b, const ReqMeta &m, int r0, int r1)
{
    TileView v{0, 0, 0, false};
    if (r0 >= r1)
        return v;
    v.prefix = score_prefix(p, b, m.L);
    const int t0 = r0 / p.group, t1 = (r1 - 1) / p.group, base = m.L - m.qn;
    if (!p.first_keys) {
        v.lo = score_low(p, 0, base + t0);
        v.hi = base + t1 + 1;
        return v;
    }
    int lo = INT32_MAX, hi = 0;
    for (int t = t0 + (int)(threadIdx.x % 32); t <= t1; t += 32) {
        const int pos = base + t, l = score_low(p, (int64_t)m.qs + t, pos);
        if (l <= pos) {
            lo = min(lo, l);
            hi = pos + 1;
        }
    }
    v.lo = __reduce_min_sync(0xffffffffu, lo);
    v.hi = __reduce_max_sync(0xffffffffu, hi);
    return v;
}

// One group's part in a CTA's range, as every role walks through it.
struct TileGroup {
    int b, tile, hv;    // request, row tile, (KV head, part of the columns)
    int g0;             // first item
    int n, w;           // key tiles, items (kGroupSetup more, or none)
    ReqMeta m;
    TileView v;
    TileBlocks t;
};

// (x.m is request x.b's)
template <int DH, int NT>
__device__ __forceinline__ void load_group(const ScoreParams &p, TileGroup &x)
{
    constexpr int RT = NT * 128;
    const int rows = x.m.qn * p.group;
    x.v = warp_tile_view(p, x.b, x.m, min(x.tile * RT, rows), min(x.tile * RT + RT, rows));
    x.t = tile_blocks(x.v, kTileKeys);
    x.n = x.t.count;
    x.w = x.n ? x.n + kGroupSetup<NT> : 0;
}

// The next group with items (there is one: the range goes on).
template <int DH, int NT>
__device__ __forceinline__ void next_group(const ScoreParams &p, TileGroup &x, int heads)
{
    x.g0 += x.w;
    if (++x.hv < heads)
        return;
    x.hv = 0;
    do {
        ++x.tile;
        while (x.b < p.num_seqs && x.tile >= group_tiles(p, x.m, NT * 128)) {
            x.tile = 0;
            if (++x.b < p.num_seqs)
                x.m = score_meta(p, x.b);
        }
        if (x.b >= p.num_seqs)
            return;
        load_group<DH, NT>(p, x);
    } while (x.n == 0);
}

// Whether the page at k0 holds a key of the group's prefix or range.
__device__ __forceinline__ bool page_seen(const TileView &v, int k0)
{
    return k0 < v.prefix || (k0 < v.hi && k0 + 16 > v.lo);
}

__device__ __forceinline__ int tile_key(const TileBlocks &t, int i)
{
    return (i < t.np ? i : t.b0 + i - t.np) * kTileKeys;
}

// First V row of the tile at k0 that holds no token of the request (128: none
// that is loaded): rows past the length may hold anything.
__device__ __forceinline__ int stale_row(const TileGroup &x, int k0)
{
    const int page = x.m.L / 16 * 16;  // the request's partial page
    return x.m.L % 16 && page >= k0 && page < k0 + kTileKeys && page_seen(x.v, page) ? x.m.L - k0 : kTileKeys;
}

// f(values of 32 columns, chunk) for the four chunks of a score tile.  One copy
// of f: a CTA lives for some 15 tiles, so what the instruction cache has to fetch
// shows.  (With the next chunk's load in flight, in two copies of f: 65.6 and
// 342 us at the sizes above, against 63.4 and 302 before Q came by TMA.)
template <typename F>
__device__ __forceinline__ void for_chunks(uint32_t scol, F f)
{
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
        uint32_t a[32];
        tmem_ld32(scol + ch * 32, a);
        tmem_wait_ld();
        f(a, ch);
    }
}

// Bits below n.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// The rows of the groups that lie wholly in a CTA's range [lo, hi), which begins in
// row tile `tile` of request b (`first` items of one head before it), whose result is
// not finite though their sum is: computed again key by key, over exactly their own
// keys (one that only other rows of the tile see may have met a zero probability
// with an infinity or a NaN).  By all warps once the CTA's other work is done: a row
// takes 0.6 to 1 us for each key, and no wait of another warp may last so long. (One
// infinite value that all 4096 tokens of a prompt see makes its 60 us 110 ms.)
template <int DH, int NT>
__device__ __noinline__ void repair_groups(const ScoreParams &p, int b, int tile, int first, int lo, int hi)
{
    using C = TileCfg<DH, NT>;
    constexpr int RT = NT * 128;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, heads = p.hkv * C::kSplit;
    TileGroup x;
    x.b = b;
    x.tile = tile;
    x.m = score_meta(p, x.b);
    load_group<DH, NT>(p, x);
    x.hv = (lo - first * heads) / x.w;
    x.g0 = first * heads + x.hv * x.w;
    for (int item = lo; item < hi; item < hi ? next_group<DH, NT>(p, x, heads) : (void)0) {
        item = min(hi, x.g0 + x.w);
        if (x.g0 + kGroupSetup<NT> < lo || x.g0 + x.w > hi)
            continue;  // others have a part
        const int rows = min(RT, x.m.qn * p.group - x.tile * RT), part = x.hv % C::kSplit;
        for (int r = warp; r < rows; r += kTileThreads / 32) {
            const int row = x.tile * RT + r, tok = row / p.group, head = x.hv / C::kSplit * p.group + row - tok * p.group;
            const int64_t at = ((int64_t)x.m.qs + tok) * p.hq + head;
            const uint32_t *out = reinterpret_cast<const uint32_t *>(p.out + at * DH + part * C::kCols);
            bool odd = false;
            for (int k = lane; k < C::kCols / 2; k += 32) {
                const uint32_t v = __ldcg(out + k);
                odd |= (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
            }
            if (__any_sync(0xffffffffu, odd)) {
                const float lse = part == 0 && p.lse ? __ldcg(p.lse + at) : 0.f;
                scored_row<DH>(p, x.b, x.m, tok, head, part * C::kCols, C::kCols, lse != lse);
            }
        }
    }
}

template <int DH, int NT, int MODE>
__global__ void __launch_bounds__(kTileThreads, 1)
    scored_tiles_kernel(const __grid_constant__ ScoreParams p, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                        const TileWork w)
{
    using C = TileCfg<DH, NT>;
    constexpr int RT = NT * 128, NS = C::kStages, UK = C::kUnitsK, UV = C::kUnitsV;
    constexpr int COLS_W = NT == 2 ? 128 : C::kCols / 2;  // output columns that a softmax group reads
    constexpr uint32_t ID_QK = idesc_bf16_f32(128, kTileKeys, false), ID_PV = idesc_bf16_f32(128, 128, true);
    enum { B_FULL = 0, B_EMPTY = NS, B_S = 2 * NS, B_P = B_S + 2, B_M = B_P + 2, B_PV = B_M + 2, B_Q, B_QE, B_O, B_DONE, B_Z, NBARS = B_Z + NS };
    static_assert(NBARS * 8 <= 256, "barriers");
    static_assert(tiles_smem<DH, NT>() <= kMaxSmemPerBlock, "shared-memory layout");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *s_q = smem;                       // [NT][DH/64][128 rows][128 bytes]
    uint8_t *s_ring = s_q + C::kQBytes;        // [NS][2][128 keys][128 bytes]
    uint8_t *s_out = s_ring + NS * kUnitBytes; // [8 warps][32 rows][128 bytes]
    uint8_t *small = s_out + C::kOutBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(small);
    // [0] abort [1] tmem [2] odd rows [4..7) start [8..16) bad pages in a segment
    volatile int *s_flags = reinterpret_cast<volatile int *>(small + 256);
    float *s_m = reinterpret_cast<float *>(small + 512);                    // [128] the shared running maximum
    float *s_l = s_m + 128;                                                 // [2][128] the two halves' sums
    volatile int *abort_flag = s_flags;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    auto wait = [&](int i, uint32_t parity) { return wait_parked(bar(i), parity & 1u, abort_flag, p.err, i); };
    // (the warp that issues the products spins: it must not wake late)
    auto wait_spin = [&](int i, uint32_t parity) { return wait_bar(bar(i), parity & 1u, abort_flag, p.err, i); };
    if (tid == 0) {
        for (int i = 0; i < 2 * NS; ++i)
            mbar_init(bar(i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_M + i), 4);
        }
        mbar_init(bar(B_PV), 1);
        mbar_init(bar(B_Q), 2);
        mbar_init(bar(B_QE), 1);
        mbar_init(bar(B_O), 2);
        mbar_init(bar(B_DONE), 1);
        for (int i = 0; i < NS; ++i)
            mbar_init(bar(B_Z + i), 1);
        s_flags[0] = s_flags[2] = 0;
        fence_barrier_init();
    }
    griddep_wait();
    griddep_launch_dependents();

    // --------------------------------------- items before each row tile ----
    // (in the ring, which is not in use yet; the roles then walk on from the
    // range's first group by themselves)
    const int heads = p.hkv * C::kSplit, c = blockIdx.x;
    int32_t *s_first = reinterpret_cast<int32_t *>(s_ring);  // [num_seqs + 1] first row tile of a request
    int32_t *s_off = s_first + p.num_seqs + 1;               // [row tiles + 1] first item of a row tile (of one head)
    int *scratch = reinterpret_cast<int *>(small + 512);  // (all sums fit: at most INT32_MAX items)
    const int tiles = block_exclusive_sums<kTileThreads>(p.num_seqs, s_first, scratch, [&](int b) {
        const ReqMeta m = score_meta(p, b);
        if (!m.ok && c == 0)
            record_error(p.err, kErrBadMetadata, b);
        return group_tiles(p, m, RT);
    });
    // (the host's bound holds for requests that do not overlap; a query_start_loc
    // that decreases may give more: those rows are left out, its request is named)
    const int ntiles = min(tiles, w.max_tiles);
    const int per_head = block_exclusive_sums<kTileThreads>(ntiles, s_off, scratch, [&](int e) {
        const int b = owner_of(s_first, p.num_seqs, e), tile = e - s_first[b];
        const ReqMeta m = score_meta(p, b);
        const int rows = m.qn * p.group;
        const int n = tile_blocks(tile_view(p, b, m, min(tile * RT, rows), min(tile * RT + RT, rows)), kTileKeys).count;
        return n ? n + kGroupSetup<NT> : 0;
    });
    const int total = per_head * heads, ctas = min(w.ctas, total);
    // row tiles that see nothing
    for (int e = c; e < ntiles; e += w.ctas) {
        if (s_off[e + 1] > s_off[e])
            continue;
        const int b = owner_of(s_first, p.num_seqs, e), r0 = (e - s_first[b]) * RT;
        const ReqMeta m = score_meta(p, b);
        const int rows = min(RT, m.qn * p.group - r0);
        for (int i = tid; i < rows * p.hkv; i += kTileThreads) {
            const int row = r0 + i / p.hkv, tok = row / p.group;
            const int64_t at = ((int64_t)m.qs + tok) * p.hq + i % p.hkv * p.group + row - tok * p.group;
            for (int k = 0; k < DH / 8; ++k)
                reinterpret_cast<uint4 *>(p.out + at * DH)[k] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse)
                p.lse[at] = -INFINITY;
        }
    }
    for (int b = c; b < p.num_seqs; b += w.ctas) {
        const ReqMeta m = score_meta(p, b);
        if (!m.ok && m.sane) {
            const int64_t first = (int64_t)m.qs * p.hq, n = (int64_t)m.qn * p.hq;
            for (int64_t i = tid; i < n * DH; i += kTileThreads)
                p.out[first * DH + i] = __ushort_as_bfloat16(0x7FC0);
            if (p.lse)
                for (int64_t i = tid; i < n; i += kTileThreads)
                    p.lse[first + i] = __int_as_float(0x7FC00000);
        }
    }
    if (c >= ctas) {
        if (tid == 0)
            w.tails[c] = make_int4(0, 0, 0, 0);
        return;
    }
    const int lo = (int)range_lo(total, c, ctas), hi = (int)range_lo(total, c + 1, ctas);
    if (tid == 0) {
        const int e = owner_of(s_off, ntiles, lo / heads);
        const int b = owner_of(s_first, p.num_seqs, e);
        s_flags[4] = b;
        s_flags[5] = e - s_first[b];
        s_flags[6] = s_off[e];
    }
    if (tid == 64) {
        const int e = owner_of(s_off, ntiles, (hi - 1) / heads), b = owner_of(s_first, p.num_seqs, e);
        const int n = s_off[e + 1] - s_off[e], hv = (hi - 1 - s_off[e] * heads) / n;
        const int g0 = s_off[e] * heads + hv * n, keys = g0 + kGroupSetup<NT>;  // first item; first key tile
        w.tails[c] = make_int4(b, e - s_first[b], hv,
                               g0 + n > hi && keys >= lo && keys < hi ? range_owner(total, g0 + n - 1, ctas) - c + 1 : 0);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(const_cast<int *>(&s_flags[1])), 512);
        tmem_relinquish();
    }
    fence_proxy_async_smem();  // the sums have been read: copies may land on them
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)s_flags[1];
    TileGroup x;
    x.b = s_flags[4];
    x.tile = s_flags[5];
    x.m = score_meta(p, x.b);
    load_group<DH, NT>(p, x);
    {
        const int first = s_flags[6] * heads;
        x.hv = (lo - first) / x.w;
        x.g0 = first + x.hv * x.w;
    }
    // this CTA's key tiles [j0, j0 + n) of the group, and the items after them
    struct Part {
        int j0, n, next;
    };
    auto part_of = [&](int item) {
        Part s;
        s.next = min(hi, x.g0 + x.w);
        s.j0 = max(item - x.g0 - kGroupSetup<NT>, 0);
        s.n = max(s.next - x.g0 - kGroupSetup<NT>, 0) - s.j0;
        return s;
    };
    // position in the ring, within a segment of n tiles, of K or V of tile j
    auto pos_k = [&](int j) { return NT == 2 ? j * (UK + UV) : (j == 0 ? 0 : UK + (j - 1) * (UK + UV)); };
    auto pos_v = [&](int j, int n) {
        return NT == 2 ? j * (UK + UV) + UK : UK + j * (UK + UV) + (j + 1 < n ? UK : 0);
    };
    bool ok = true;
    uint32_t seg = 0;  // segments so far
    if (warp == 0) {
        // -------------------------------------------------------- producer --
        uint32_t pos = 0;  // units so far
        const int pg = lane % 8, cb = (lane / 8) % 2;
        auto ids_of = [&](int j) {
            const int k0 = tile_key(x.t, j) + pg * 16;
            return page_seen(x.v, k0) ? __ldg(p.block_tables + (int64_t)x.b * p.max_blocks + k0 / 16) : -1;
        };
        auto load = [&](const CUtensorMap *map, int units, int col0, int id) {
            for (int u = 0; ok && u < units; ++u, ++pos) {
                const int stage = pos % NS;
                if (pos >= NS)
                    ok = __all_sync(0xffffffffu, wait(B_EMPTY + stage, pos / NS - 1));
                if (!ok)
                    return;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(B_FULL + stage), kUnitBytes);
                __syncwarp();
                // (block -1 lies outside the pool: zeros, no bytes read)
                if (lane < 16)
                    tma_load_4d(smem_addr(s_ring + stage * kUnitBytes + cb * 16384 + pg * 2048), map, bar(B_FULL + stage),
                                col0 + u * 128 + cb * 64, x.hv / C::kSplit, 0, id);
            }
        };
        for (int item = lo; ok && item < hi; item < hi ? next_group<DH, NT>(p, x, heads) : (void)0) {
            const Part s = part_of(item);
            const int j0 = s.j0, n = s.n;
            item = s.next;
            if (n == 0)
                continue;
            const int v_col = x.hv % C::kSplit * C::kCols;
            // (Read when the segment's products are done.  The copies of a segment need
            // at least two stages, and the products of the next one wait for this one's
            // softmax, so the producer is less than eight segments ahead of a reader.)
            static_assert(NS <= 8, "flags of bad pages");
            if (lane == 0)
                s_flags[8 + seg % 8] = 0;
            auto check = [&](int raw, int j) {
                // (whether some row sees a key of the page is looked up at the segment's end)
                const bool bad = page_seen(x.v, tile_key(x.t, j) + pg * 16) && (raw < 0 || (int64_t)raw >= p.num_blocks);
                if (__any_sync(0xffffffffu, bad)) {
                    if (lane == 0)
                        s_flags[8 + seg % 8] = 1;
                    __syncwarp();
                }
                return bad ? -1 : raw;
            };
            int cur = check(ids_of(j0), j0), ahead = n > 1 ? ids_of(j0 + 1) : -1;
            load(&tm_k, UK, 0, cur);
            for (int j = 0; ok && j < n; ++j) {
                const int id = cur;
                if (j + 1 < n) {
                    cur = check(ahead, j0 + j + 1);
                    ahead = j + 2 < n ? ids_of(j0 + j + 2) : -1;
                }
                if (NT == 2)
                    load(&tm_v, UV, v_col, id);
                if (j + 1 < n)
                    load(&tm_k, UK, 0, cur);
                if (NT == 1)
                    load(&tm_v, UV, v_col, id);
            }
            ++seg;
            // V rows past the request's length (in its last tile) become zeros
            const int k_last = tile_key(x.t, j0 + n - 1), row0 = stale_row(x, k_last);
            if (ok && row0 < kTileKeys) {
                for (int u = 0; ok && u < UV; ++u) {
                    const uint32_t at = pos - UV + u;
                    ok = __all_sync(0xffffffffu, wait(B_FULL + at % NS, at / NS));
                    if (!ok)
                        break;
                    uint8_t *v = s_ring + at % NS * kUnitBytes;
                    for (int i = lane; i < (16 - x.m.L % 16) * 16; i += 32)
                        *reinterpret_cast<uint4 *>(v + (i % 16 / 8) * 16384 + (row0 + i / 16) * 128 + (i % 8) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(B_Z + at % NS));
                }
            }
        }
        // after a timeout: no copy may land in memory that the CTA has left
        if (!ok && lane == 0)
            for (uint32_t i = pos > NS ? pos - NS : 0; i < pos; ++i)
                wait_bar_drain(bar(B_FULL + i % NS), (i / NS) & 1u);
    } else if (warp == 1) {
        // -------------------------------------------------------- products --
        uint32_t base = 0;               // units before the segment
        uint32_t p_seen[2] = {0, 0};     // probabilities consumed of each buffer
        uint32_t zeroed = 0;             // a bit per stage: the phase of its B_Z
        for (int item = lo; ok && item < hi; item < hi ? next_group<DH, NT>(p, x, heads) : (void)0) {
            const Part s = part_of(item);
            const int j0 = s.j0, n = s.n, ni = n * NT;
            item = s.next;
            if (n == 0)
                continue;
            const bool zero = stale_row(x, tile_key(x.t, j0 + n - 1)) < kTileKeys;
            auto qk = [&](int i) {
                const int t = NT == 2 ? i % 2 : 0, j = i / NT;
                for (int u = 0; ok && u < UK; ++u) {
                    const uint32_t at = base + pos_k(j) + u, stage = at % NS;
                    ok = wait_spin(B_FULL + stage, at / NS);
                    if (!ok)
                        return;
                    const uint64_t qd = sdesc_sw128(smem_addr(s_q + t * 128 * DH * 2 + u * 32768), 16, 1024);
                    const uint64_t kd = sdesc_sw128(smem_addr(s_ring + stage * kUnitBytes), 16, 1024);
                    uint64_t a[8], b[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t step = (uint64_t)(((k / 4) * 16384 + (k % 4) * 32) >> 4);
                        a[k] = qd + step;
                        b[k] = kd + step;
                    }
                    tc_fence_after();
                    mma8_ss<1>(tmem + (uint32_t)(i % 2) * 128u, a, b, ID_QK, u > 0);
                    if (t == NT - 1)
                        mma_commit(bar(B_EMPTY + stage));
                }
                mma_commit(bar(B_S + i % 2));
                if (i == ni - 1)
                    mma_commit(bar(B_QE));  // Q may be replaced
            };
            auto pv = [&](int i) {
                const int t = NT == 2 ? i % 2 : 0, j = i / NT;
                ok = wait_spin(B_P + i % 2, p_seen[i % 2]);
                ++p_seen[i % 2];
                for (int u = 0; ok && u < UV; ++u) {
                    const uint32_t at = base + pos_v(j, n) + u, stage = at % NS;
                    ok = wait_spin(B_FULL + stage, at / NS);
                    if (ok && zero && j == n - 1 && t == 0) {
                        ok = wait_spin(B_Z + stage, zeroed >> stage);
                        zeroed ^= 1u << stage;
                    }
                    if (!ok)
                        return;
                    const uint64_t vd = sdesc_sw128(smem_addr(s_ring + stage * kUnitBytes), 16384, 1024);
                    uint32_t a[8];
                    uint64_t b[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        a[k] = tmem + (uint32_t)(i % 2) * 128u + (uint32_t)k * 8u;
                        b[k] = vd + (uint64_t)((k * 2048) >> 4);
                    }
                    tc_fence_after();
                    mma8_ts<1>(tmem + (uint32_t)(C::kOCol + (t + u) * 128), a, b, ID_PV, j > 0);
                    if (t == NT - 1)
                        mma_commit(bar(B_EMPTY + stage));
                }
                if (NT == 1 && MODE != kModeCapped)
                    mma_commit(bar(B_PV));
            };
            if (lane == 0) {
                ok = wait_spin(B_Q, seg);
                for (int i = 0; ok && i < min(2, ni); ++i)
                    qk(i);
                for (int i = 0; ok && i < ni; ++i) {
                    pv(i);
                    if (ok && i + 2 < ni)
                        qk(i + 2);
                }
                if (ok) {
                    mma_commit(bar(B_O));
                    mbar_arrive(bar(B_O));  // (and what this thread has seen of the producer's flags)
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            base += (uint32_t)n * (UK + UV);
            ++seg;
        }
        if (lane == 0) {
            mma_commit(bar(B_DONE));
            wait_bar_drain(bar(B_DONE), 0);
        }
        __syncwarp();
    } else if (warp < 4) {
        // -------------------------------------------------------------- Q --
        // A group's rows as soon as the products of the group before have read
        // theirs: a thread keeps its column, so that all copies are in flight.
        constexpr int CH = DH / 8, STEP = 64 / CH;  // 16-byte vectors of a row; rows apart
        uint32_t boxes = 0;  // segments that came by TMA
        const int qt = tid - 64, ch = qt % CH;
        const int step_tok = STEP / p.group, step_head = STEP - step_tok * p.group;
        for (int item = lo; ok && item < hi; item < hi ? next_group<DH, NT>(p, x, heads) : (void)0) {
            const Part s = part_of(item);
            item = s.next;
            if (s.n == 0)
                continue;
            if (seg > 0)
                ok = __all_sync(0xffffffffu, wait(B_QE, seg - 1));
            ++seg;
            if (!ok)
                break;
            const int kvh = x.hv / C::kSplit, rows = min(RT, x.m.qn * p.group - x.tile * RT);
            if (w.q_boxes) {
                // whole tokens to a row tile: a TMA box for each tile and 64 columns.
                // (Rows past the request's are other tokens', or zeros: their
                // results go nowhere.)
                if (lane == 0) {
                    if (warp == 2)
                        mbar_arrive_expect_tx(bar(B_Q), C::kQBytes);
                    else
                        mbar_arrive(bar(B_Q));
                }
                __syncwarp();
                if (warp == 2 && lane < NT * (DH / 64))
                    tma_load_3d(smem_addr(s_q) + lane * 16384, &tm_q, bar(B_Q), lane % (DH / 64) * 64, kvh * p.group,
                                x.m.qs + (x.tile * NT + lane / (DH / 64)) * (128 / p.group));
                boxes = seg;
                continue;
            }
            const int first = x.tile * RT + qt / CH;
            int tok = first / p.group, head = first - tok * p.group;
            const __nv_bfloat16 *src = p.q + (int64_t)x.m.qs * p.q_tok_stride + (int64_t)kvh * p.group * DH + ch * 8;
            const uint32_t dst = smem_addr(s_q) + (ch / 8) * 16384;
#pragma unroll 4
            for (int qr = qt / CH; qr < RT; qr += STEP) {
                const bool have = qr < rows;
                // (zeros for rows that are not there)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 dst + (qr / 128) * 128 * DH * 2 + (qr % 128) * 128 + (((ch % 8) ^ (qr & 7)) << 4)),
                             "l"(have ? src + tok * p.q_tok_stride + head * DH : p.q), "r"(have ? 16 : 0)
                             : "memory");
                tok += step_tok;
                head += step_head;
                if (head >= p.group) {
                    head -= p.group;
                    ++tok;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(B_Q));
        }
        if (!ok && boxes && lane == 0)
            wait_bar_drain(bar(B_Q), (boxes - 1) & 1u);
    } else {
        // --------------------------------------------------------- softmax --
        const int wg = (warp - 4) / 4, r = (warp % 4) * 32 + lane;
        const uint32_t lane_off = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t scol = tmem + lane_off + (uint32_t)wg * 128u;
        const uint32_t ocol = tmem + lane_off + C::kOCol + (NT == 2 ? (uint32_t)wg * 128u : 0u);
        uint32_t s_seen = 0, m_base[2] = {0, 0}, pv_base = 0;
        const float c1 = p.scale_log2, cap = p.cap_log2;
        const float y1 = c1 * (0.5f * kLn2);  // raw score to y: c1 = 2 scale log2 e / soft_cap
        const float limit = kTanhReach / y1;
        const uint64_t t0 = pack_f32x2(cap * kTanh0, cap * kTanh0);
        const uint64_t t1 = pack_f32x2(cap * kTanh1, cap * kTanh1);
        const uint64_t t2 = pack_f32x2(cap * kTanh2, cap * kTanh2);
        const uint64_t t3 = pack_f32x2(cap * kTanh3, cap * kTanh3);
        const uint64_t yy1 = pack_f32x2(y1, y1);
        for (int item = lo; item < hi; item < hi ? next_group<DH, NT>(p, x, heads) : (void)0) {
            const Part s = part_of(item);
            const int j0 = s.j0, n = s.n;
            item = s.next;
            if (n == 0)
                continue;
            const bool whole = n == x.n;
            const int kvh = x.hv / C::kSplit, part = x.hv % C::kSplit;
            const int rows = min(RT, x.m.qn * p.group - x.tile * RT);
            // what this thread's row sees
            const int gr = (NT == 2 ? wg * 128 : 0) + r, row = x.tile * RT + gr;
            const bool valid = gr < rows;
            const int tok = valid ? row / p.group : 0, head = kvh * p.group + (valid ? row - tok * p.group : 0);
            const int pos = x.m.L - x.m.qn + tok;
            const int prefix = valid ? x.v.prefix : 0;
            const int r_lo = valid ? score_low(p, (int64_t)x.m.qs + tok, pos) : 1;
            const int r_len = valid ? pos - r_lo + 1 : 0;
            const int near = valid ? score_nearest(r_lo, pos, prefix) : 0;
            const float slope = valid && p.slopes ? __ldg(p.slopes + head) : 0.f, slope2 = slope * kLog2e;
            const int lo_max = __reduce_max_sync(0xffffffffu, valid ? r_lo : 0);
            const int pos_min = __reduce_min_sync(0xffffffffu, valid ? pos : INT32_MAX);
            const int pre_min = __reduce_min_sync(0xffffffffu, valid ? prefix : INT32_MAX);
            float m = MODE == kModeCapped ? 0.f : -INFINITY, l = 0.f;
            for (int i = NT == 2 ? 0 : wg; i < n; i += NT == 2 ? 1 : 2) {
                const int k0 = tile_key(x.t, j0 + i);
                if (ok)
                    ok = wait(B_S + wg, s_seen);
                ok = __all_sync(0xffffffffu, ok);
                ++s_seen;
                tc_fence_after();
                // every row of the warp sees every key of the tile
                const bool past = k0 >= lo_max && k0 + kTileKeys - 1 <= pos_min;  // (and none lies after its position)
                const bool all = past || k0 + kTileKeys <= pre_min;
                const int rel_lo = r_lo - k0, rel_pre = prefix - k0;
                // bit k: column ch * 32 + k is seen
                auto seen = [&](int ch) {
                    const int a = rel_lo - ch * 32;
                    return (bits_below(a + r_len) & ~bits_below(a)) | bits_below(rel_pre - ch * 32);
                };
                uint64_t sum0 = 0, sum1 = 0;
                if (ok && MODE == kModeCapped) {
                    // no maximum: |z| <= cap, and 2^cap times any number of keys is far from overflow
                    for_chunks(scol, [&](uint32_t(&v)[32], int ch) {
                        // (chunks that are seen whole, or by no row, are common in a tile that is neither)
                        const uint32_t keep = all ? ~0u : seen(ch);
                        if (!all && !__any_sync(0xffffffffu, keep != 0u)) {
                            uint32_t o[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = 0u;
                            tmem_st16(scol + ch * 16, o);
                            return;
                        }
                        // (hidden scores take no part in the choice of a form either: what a row
                        // does not see changes no bit of its result)
                        const bool some = !all && __any_sync(0xffffffffu, ~keep != 0u);
                        auto hide = [&]() {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = keep & (1u << k) ? v[k] : 0u;
                        };
                        if (some)
                            hide();
                        float top = 0.f, top1 = 0.f;
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            top = max3f(top, fabsf(__uint_as_float(v[k])), fabsf(__uint_as_float(v[k + 1])));
                            top1 = max3f(top1, fabsf(__uint_as_float(v[k + 2])), fabsf(__uint_as_float(v[k + 3])));
                        }
                        // (a NaN passes the test unseen and stays one in both ways)
                        if (__all_sync(0xffffffffu, fmaxf(top, top1) <= limit || !valid)) {
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                const uint64_t y = mul_f32x2(pack_f32x2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), yy1);
                                const uint64_t u = mul_f32x2(y, y);
                                const uint64_t z = mul_f32x2(y, fma_f32x2(fma_f32x2(fma_f32x2(t3, u, t2), u, t1), u, t0));
                                float a, b;
                                unpack_f32x2(z, a, b);
                                v[k] = __float_as_uint(ex2(a));
                                v[k + 1] = __float_as_uint(ex2(b));
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint(ex2(capped(__uint_as_float(v[k]), c1, cap)));
                        }
                        if (some)
                            hide();
                        uint32_t o[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            sum0 = add_f32x2(sum0, pack_f32x2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                            sum1 = add_f32x2(sum1, pack_f32x2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])));
                            o[k / 2] = pack_bf16x2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                            o[k / 2 + 1] = pack_bf16x2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                        }
                        tmem_st16(scol + ch * 16, o);
                    });
                } else if (MODE != kModeCapped) {
                    // two passes over the scores in tensor memory: the maximum (and
                    // what the rules make of the scores, written back), the exponents
                    float mx = -INFINITY;
                    if (ok) {
                        float mx1 = -INFINITY;
                        const float b0 = -slope2 * (float)(pos - near - k0);
                        for_chunks(scol, [&](uint32_t(&v)[32], int ch) {
                            const uint32_t keep = all ? ~0u : seen(ch);
                            const bool some = all || __any_sync(0xffffffffu, keep != 0u);
                            if (MODE != kModePlain && some) {
                                if constexpr (MODE == kModeWide) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        v[k] = __float_as_uint(capped_wide(__uint_as_float(v[k]), c1, cap));
                                } else if (cap > 0.f) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        v[k] = __float_as_uint(capped(__uint_as_float(v[k]), c1, cap));
                                } else {
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        v[k] = __float_as_uint(__uint_as_float(v[k]) * c1);
                                }
                                if (past) {
                                    const float bc = __fmaf_rn(slope2, (float)(ch * 32), b0);
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        v[k] = __float_as_uint(__uint_as_float(v[k]) + __fmaf_rn(slope2, (float)k, bc));
                                } else {
                                    const int d = pos - k0 - ch * 32;
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        v[k] = __float_as_uint(
                                            __fmaf_rn(-slope2, (float)(abs(d - k) - near), __uint_as_float(v[k])));
                                }
                            }
                            if (!all && __any_sync(0xffffffffu, ~keep != 0u)) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    v[k] = keep & (1u << k) ? v[k] : 0xff800000u;
                            }
                            if (MODE != kModePlain || !all)
                                tmem_st32(scol + ch * 32, v);
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                mx = max3f(mx, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                                mx1 = max3f(mx1, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                            }
                        });
                        mx = fmaxf(mx, mx1);
                        if (MODE == kModePlain)
                            mx *= c1;
                    }
                    if (NT == 1 && i > 0) {
                        // the maximum after the tile before, which the other group holds
                        if (ok)
                            ok = wait(B_M + (wg ^ 1), m_base[wg ^ 1] + (uint32_t)(wg ? (i - 1) / 2 : i / 2 - 1));
                        ok = __all_sync(0xffffffffu, ok);
                        const float other = s_m[r];
                        if (other != m) {
                            l = l == 0.f ? 0.f : l * ex2(m - other);
                            m = other;
                        }
                    }
                    // the maximum moves when a tile's is more than 8 (2^8) above it
                    const bool move = mx > m + kTau || m == -INFINITY;
                    const float m_old = m;
                    if (move)
                        m = mx;
                    const float alpha = move && m_old != -INFINITY ? ex2(m_old - m) : 1.f;
                    if (NT == 1) {
                        s_m[r] = m;
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(B_M + wg));
                    }
                    l *= alpha;
                    if (__any_sync(0xffffffffu, alpha != 1.f) && i > 0 && ok) {
                        // (two row tiles: QK of this tile was issued behind PV of the one before)
                        if (NT == 1) {
                            ok = wait(B_PV, pv_base + (uint32_t)i - 1);
                            ok = __all_sync(0xffffffffu, ok);
                            tc_fence_after();
                        }
                        constexpr int OC = NT == 2 ? 128 : C::kCols;
                        if (ok)
#pragma unroll 1
                            for (int ch = 0; ch < OC; ch += 16) {
                                uint32_t o[16];
                                tmem_ld16(ocol + ch, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                                tmem_st16(ocol + ch, o);
                            }
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    const uint64_t nb = pack_f32x2(-base, -base);
                    const uint64_t cc = pack_f32x2(c1, c1);
                    tmem_wait_st();  // (what the first pass wrote back)
                    if (ok)
                        for_chunks(scol, [&](uint32_t(&v)[32], int ch) {
                            uint32_t o[16];
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                const uint64_t s = pack_f32x2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                                const uint64_t z = MODE == kModePlain ? fma_f32x2(s, cc, nb) : add_f32x2(s, nb);
                                float a, b;
                                unpack_f32x2(z, a, b);
                                a = ex2(a), b = ex2(b);
                                if (k % 4 == 0)
                                    sum0 = add_f32x2(sum0, pack_f32x2(a, b));
                                else
                                    sum1 = add_f32x2(sum1, pack_f32x2(a, b));
                                o[k / 2] = pack_bf16x2(a, b);
                            }
                            tmem_st16(scol + ch * 16, o);
                        });
                }
                {
                    float a, b, d, e;
                    unpack_f32x2(sum0, a, b);
                    unpack_f32x2(sum1, d, e);
                    l += (a + b) + (d + e);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(B_P + wg));
            }
            // ------------------------------------------------ the output --
            if (ok)
                ok = wait(B_O, seg);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (NT == 1) {
                // both groups' sums, relative to the maximum after the last tile
                if (MODE != kModeCapped) {
                    named_sync(1, 256);
                    const float m_end = s_m[r];
                    l = l == 0.f ? 0.f : l * ex2(m - m_end);
                    m = m_end;
                }
                s_l[wg * 128 + r] = l;
                named_sync(1, 256);
                l = s_l[r] + s_l[128 + r];
                // (a wait that ran out in the other group leaves the row without its tiles)
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            }
            // rows that see a key of a bad page (its keys and values came as zeros) are NaN;
            // a bad id whose keys no row sees does not matter
            if (ok && s_flags[8 + seg % 8]) {
                bool bad = false;
                for (int i = 0; valid && i < n * (kTileKeys / 16); ++i) {
                    const int page = tile_key(x.t, j0 + i / (kTileKeys / 16)) + i % (kTileKeys / 16) * 16;
                    if (page < prefix || (page <= pos && page + 16 > r_lo && r_len > 0)) {
                        const int id = __ldg(p.block_tables + (int64_t)x.b * p.max_blocks + page / 16);
                        bad |= id < 0 || (int64_t)id >= p.num_blocks;
                    }
                }
                if (bad) {
                    record_error(p.err, kErrBadMetadata, x.b);
                    l = __int_as_float(0x7FC00000);
                }
            }
            // (after a wait that ran out a part's sum is NaN, and so are whole rows)
            if (!ok)
                l = __int_as_float(0x7FC00000);
            const int col0 = NT == 2 ? 0 : wg * COLS_W;  // of the group's columns
            const float inv = l == 0.f ? 0.f : 1.f / l;
            bool odd = !ok;
            float *rec = w.records + (2 * (int64_t)c + (x.g0 + kGroupSetup<NT> < lo ? 0 : 1)) * w.record_floats +
                         (NT == 2 ? wg : 0) * tile_record(C::kCols);
            const int64_t at = ((int64_t)x.m.qs + tok) * p.hq + head;
            if (ok && !whole) {
#pragma unroll 1
                for (int ch = 0; ch < COLS_W; ch += 32) {
                    uint32_t o[32];
                    tmem_ld32(ocol + col0 + ch, o);
                    tmem_wait_ld();
                    float4 *dst = reinterpret_cast<float4 *>(rec + 256) + (int64_t)(col0 + ch) / 4 * 128 + r;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[k * 128] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                }
            } else if (ok) {
                uint8_t *stage = s_out + (warp - 4) * 4096;
                const int64_t dst_row = valid ? at : -1;
#pragma unroll 1
                for (int ch = 0; ch < COLS_W; ch += 32) {
                    uint32_t o[32];
                    tmem_ld32(ocol + col0 + ch, o);
                    tmem_wait_ld();
                    // (a sum, not a test for each: NaN and infinities stay in it)
                    float check = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float f = __uint_as_float(o[k]) * inv;
                        check = __fmaf_rn(f, 0.f, check);
                        o[k] = __float_as_uint(f);
                    }
                    odd |= check != 0.f && fabsf(l) < INFINITY;
                    __nv_bfloat16 *out = p.out + part * C::kCols + col0 + ch;
                    if (C::kOutBytes == 0) {
                        if (valid)
                            store_out32(out + at * DH, o);
                        continue;
                    }
                    // 32 columns into their half of the rows' 128 bytes
                    const int half = ch / 32 % 2;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + (((half * 4 + k) ^ (lane & 7)) << 4)) = make_uint4(
                            pack_bf16x2(__uint_as_float(o[8 * k]), __uint_as_float(o[8 * k + 1])),
                            pack_bf16x2(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3])),
                            pack_bf16x2(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5])),
                            pack_bf16x2(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7])));
                    if (half == 0)
                        continue;
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int sr = k * 4 + lane / 8, sc = lane % 8;
                        const int64_t to = __shfl_sync(0xffffffffu, dst_row, sr);
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + sr * 128 + ((sc ^ (sr & 7)) << 4));
                        if (to >= 0)
                            *reinterpret_cast<uint4 *>(out - 32 + to * DH + sc * 8) = v;
                    }
                    __syncwarp();
                }
            }
            if (!ok && whole && valid)
                for (int k = 0; k < COLS_W / 8; ++k)
                    reinterpret_cast<uint4 *>(p.out + at * DH + part * C::kCols + col0)[k] =
                        make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
            if (NT == 2 || wg == 0) {
                if (!whole) {
                    rec[r] = m;
                    rec[128 + r] = l;
                } else if (valid && part == 0 && p.lse) {
                    p.lse[at] = score_lse(m, l, slope * (float)near);
                }
            }
            if (whole && odd && valid)
                s_flags[2] = 1;
            m_base[0] += (uint32_t)(n + 1) / 2;
            m_base[1] += (uint32_t)n / 2;
            pv_base += (uint32_t)n;
            ++seg;
            tc_fence_before();
            if (NT == 1)
                named_sync(1, 256);  // the next group's products overwrite both groups' columns
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1)
        tmem_dealloc(tmem, 512);
    if (s_flags[2])
        repair_groups<DH, NT>(p, s_flags[4], s_flags[5], s_flags[6], lo, hi);
}

// Folds the records of the groups that several CTAs have a part of, each at the
// place of the CTA that it begins in: two threads per row, each with every second
// part, and 32 columns of the output a CTA.  (A few rows over many keys are a part to
// a CTA: one thread per row, part by part, took 27 of 42 us for 64 rows over 4096 keys.)
constexpr int kTileFoldThreads = 256;

template <int DH, int NT>
__global__ void __launch_bounds__(kTileFoldThreads) scored_tile_fold_kernel(const ScoreParams p, const TileWork w)
{
    using C = TileCfg<DH, NT>;
    griddep_wait();
    griddep_launch_dependents();
    constexpr int CB = C::kCols / 32;
    __shared__ float s_top[2][128], s_o[33][128];  // the second threads' sums and columns
    const int unit = blockIdx.x / CB, cb = blockIdx.x % CB, c0 = unit / NT, t = unit % NT;
    const int4 tail = w.tails[c0];
    const int b = tail.x, hv = tail.z, kvh = hv / C::kSplit, part = hv % C::kSplit, n = tail.w;
    if (n == 0)
        return;
    const ReqMeta m = score_meta(p, b);
    const int r = threadIdx.x % 128, half = threadIdx.x / 128, row = tail.y * (NT * 128) + t * 128 + r;
    const bool valid = row < m.qn * p.group;
    const int tok = valid ? row / p.group : 0, head = kvh * p.group + (valid ? row - tok * p.group : 0);
    auto record = [&](int c) {
        // (the group began in c0's range, and goes on in the others)
        return w.records + (2 * (int64_t)c + (c == c0 ? 1 : 0)) * w.record_floats + t * tile_record(C::kCols);
    };
    float top = -INFINITY;
#pragma unroll 8
    for (int i = half; i < n; i += 2)
        top = fmaxf(top, __ldcg(record(c0 + i) + r));
    s_top[half][r] = top;
    __syncthreads();
    top = fmaxf(top, s_top[half ^ 1][r]);
    float sum = 0.f, o[32];
#pragma unroll
    for (int k = 0; k < 32; ++k)
        o[k] = 0.f;
#pragma unroll 2
    for (int i = half; i < n; i += 2) {
        const float *rec = record(c0 + i);
        const float mi = __ldcg(rec + r), f = mi == top ? 1.f : ex2(mi - top);
        sum += __ldcg(rec + 128 + r) * f;
        const float4 *src = reinterpret_cast<const float4 *>(rec + 256) + (int64_t)cb * 8 * 128 + r;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 v = __ldcg(src + k * 128);
            o[4 * k] += v.x * f;
            o[4 * k + 1] += v.y * f;
            o[4 * k + 2] += v.z * f;
            o[4 * k + 3] += v.w * f;
        }
    }
    if (half) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
            s_o[k][r] = o[k];
        s_o[32][r] = sum;
    }
    __syncthreads();
    if (half)
        return;
#pragma unroll
    for (int k = 0; k < 32; ++k)
        o[k] += s_o[k][r];
    sum += s_o[32][r];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    bool odd = !(fabsf(sum) < INFINITY);
    uint32_t q[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const float f = o[k] * inv;
        odd |= !(fabsf(f) < INFINITY);
        q[k] = __float_as_uint(f);
    }
    const int64_t at = ((int64_t)m.qs + tok) * p.hq + head;
    if (valid) {
        store_out32(p.out + at * DH + part * C::kCols + cb * 32, q);
        if (p.lse && part == 0 && cb == 0) {
            const int pos = m.L - m.qn + tok;
            const int near = score_nearest(score_low(p, (int64_t)m.qs + tok, pos), pos, score_prefix(p, b, m.L));
            const float slope = p.slopes ? __ldg(p.slopes + head) : 0.f;
            p.lse[at] = score_lse(top, sum, slope * (float)near);
        }
    }
    __syncwarp();
    for (uint32_t todo = __ballot_sync(0xffffffffu, odd && valid); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1;
        scored_row<DH>(p, b, m, __shfl_sync(0xffffffffu, tok, from), __shfl_sync(0xffffffffu, head, from),
                       part * C::kCols + cb * 32, 32,
                       __shfl_sync(0xffffffffu, !(fabsf(sum) < INFINITY), from) && part == 0 && cb == 0);
    }
}

// --------------------------------------------------------------------- host --
template <int DH, int NT>
cudaError_t launch_tiles(const ScoreParams &p, const CUtensorMap (&tm)[3], const TileWork &w, int mode, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)w.ctas);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tiles_smem<DH, NT>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kern = mode == kModePlain    ? scored_tiles_kernel<DH, NT, kModePlain>
                : mode == kModeCapped ? scored_tiles_kernel<DH, NT, kModeCapped>
                : mode == kModeAny    ? scored_tiles_kernel<DH, NT, kModeAny>
                                      : scored_tiles_kernel<DH, NT, kModeWide>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, tm[0], tm[1], tm[2], w);
    if (e != cudaSuccess)
        return e;
    using C = TileCfg<DH, NT>;
    cfg.gridDim = dim3((unsigned)(w.ctas * NT * (C::kCols / 32)));
    cfg.blockDim = dim3(kTileFoldThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, scored_tile_fold_kernel<DH, NT>, p, w);
}

template <int DH, int NT>
cudaError_t tiles_attributes()
{
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(scored_tiles_kernel<DH, NT, kModePlain>, attr, (int)tiles_smem<DH, NT>());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(scored_tiles_kernel<DH, NT, kModeCapped>, attr, (int)tiles_smem<DH, NT>());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(scored_tiles_kernel<DH, NT, kModeAny>, attr, (int)tiles_smem<DH, NT>());
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(scored_tiles_kernel<DH, NT, kModeWide>, attr, (int)tiles_smem<DH, NT>());
    return e;
}

}  // namespace pa

// Between the parts of pa_paged_attention_scored: the choice of a kernel
// (pa_scored.cu), few rows (pa_scored_rows.cu), many rows (pa_scored_tiles*.cu).
#pragma once
#include "pa_score.cuh"

namespace pa {

constexpr int kScoredSms = 152;              // CTAs of a wave are counted by it, on the host alone

// Tensor maps of K and V: boxes of 64 columns by the 16 tokens of one page and head.
bool scored_pool_maps(const ScoreParams &p, int32_t head_dim, CUtensorMap (&tm)[2]);

// wait_bar for warps that wait beside warps at work: a try may sleep for up to a
// millisecond, and the abort flag and the clock are read between tries.
// (wait_bar's loop, which reads both at every try, was more than half of all
// instructions that scored_tiles_kernel issued.)
__device__ __forceinline__ bool wait_parked(uint32_t bar, uint32_t parity, volatile int *abort_flag, ErrState *err,
                                            int where)
{
    constexpr uint32_t kSleepNs = 1000000;
    uint64_t t0 = 0;
    for (;;) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(bar), "r"(parity), "r"(kSleepNs)
                     : "memory");
        if (done)
            return true;
        if (*abort_flag)
            return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0)
            t0 = now;
        if (now - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            record_error(err, kErrTimeout, ((long long)blockIdx.x << 8) | where);
            return false;
        }
    }
}

// Keys that a tile of rows sees: a prefix and one range.  Tokens that see something
// see their own position, so the range is a hull with keys that no row sees only
// where tokens that see nothing lie between tokens that do.
struct TileView {
    int prefix, lo, hi;  // [0, prefix) and [lo, hi); hi <= lo: no range
    bool gaps;           // some keys of the range may be hidden from every row
};

// rows [r0, r1) of a request (row = token * group + head)
__device__ __forceinline__ TileView tile_view(const ScoreParams &p, int b, const ReqMeta &m, int r0, int r1)
{
    TileView v{0, 0, 0, false};
    if (r0 >= r1)
        return v;
    v.prefix = score_prefix(p, b, m.L);
    const int t0 = r0 / p.group, t1 = (r1 - 1) / p.group;
    const int base = m.L - m.qn;
    int seeing = 0, from = 0;
    v.lo = INT32_MAX;
    v.hi = 0;
    if (!p.first_keys) {
        v.lo = score_low(p, 0, base + t0);  // later tokens' ranges start no earlier
        v.hi = base + t1 + 1;
    } else {
        for (int t = t0; t <= t1; ++t) {
            const int pos = base + t, lo = score_low(p, (int64_t)m.qs + t, pos);
            if (lo <= pos) {
                v.lo = min(v.lo, lo);
                v.hi = pos + 1;
                from = seeing++ ? from : pos;
            }
        }
        v.gaps = seeing < v.hi - from;
    }
    return v;
}

// Whether rows [r0, r1) of a request see a key of the page at k0 (v: their view).
__device__ __forceinline__ bool page_needed(const ScoreParams &p, const ReqMeta &m, const TileView &v, int r0, int r1,
                                            int k0)
{
    if (k0 < v.prefix)
        return true;
    if (k0 >= v.hi || k0 + 16 <= v.lo)
        return false;
    if (!v.gaps)
        return true;
    const int base = m.L - m.qn, t1 = (r1 - 1) / p.group;
    bool seen = false;
#pragma unroll 1
    for (int t = max(r0 / p.group, k0 - base); t <= t1 && !seen; ++t) {
        const int lo = score_low(p, (int64_t)m.qs + t, base + t);
        seen = lo <= base + t && lo < k0 + 16;
    }
    return seen;
}

// Blocks of `keys` keys that hold what a tile sees: the prefix's np first ones,
// then those from b0 on; `count` in all.
struct TileBlocks {
    int np, b0, count;
};

__device__ __forceinline__ TileBlocks tile_blocks(const TileView &v, int keys)
{
    TileBlocks t;
    t.np = (v.prefix + keys - 1) / keys;
    t.b0 = t.np;
    int n = 0;
    if (v.hi > v.lo) {
        t.b0 = max(v.lo / keys, t.np);
        n = max((v.hi + keys - 1) / keys - t.b0, 0);
    }
    t.count = t.np + n;
    return t;
}

// First item of CTA c's range: floor(total * c / ctas), in 32 bits (total is at
// most INT32_MAX, ctas a few hundred).
__device__ __forceinline__ int64_t range_lo(int64_t total, int c, int ctas)
{
    const uint32_t each = (uint32_t)total / (uint32_t)ctas, rest = (uint32_t)total - each * (uint32_t)ctas;
    return (int64_t)(each * (uint32_t)c + rest * (uint32_t)c / (uint32_t)ctas);
}

// The CTA whose range has an item (total >= ctas: every range has some).
__device__ __forceinline__ int range_owner(int64_t total, int64_t item, int ctas)
{
    int c = min((int)((float)item * (float)ctas / (float)total), ctas - 1);
    while (range_lo(total, c + 1, ctas) <= item)
        ++c;
    while (range_lo(total, c, ctas) > item)
        --c;
    return c;
}

bool scored_rows_fits(int32_t num_seqs, int32_t hkv, int32_t head_dim, int32_t max_seq_len);
size_t scored_rows_bytes(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len,
                         int32_t max_seq_len);
cudaError_t launch_scored_rows(const ScoreParams &p, int32_t head_dim, void *workspace, cudaStream_t stream, char *info,
                               size_t info_len);
cudaError_t init_scored_rows_attributes();

// Row tiles that the batch can form, and whether the kernels take that many
// (num_q_tokens < 0, for a workspace's size: left to the call itself).
constexpr int kScoredMaxEntriesHost = 24000;  // requests and row tiles that a CTA sums over
int64_t scored_tiles_bound(int32_t num_seqs, int group, int32_t head_dim, int32_t max_query_len, int64_t num_q_tokens);
bool scored_tiles_fits(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len,
                       int32_t max_seq_len, int64_t num_q_tokens);
size_t scored_tiles_bytes(int group, int32_t head_dim, int32_t max_query_len);
cudaError_t launch_scored_tiles(const ScoreParams &p, int32_t head_dim, void *workspace, cudaStream_t stream, char *info,
                                size_t info_len);
cudaError_t init_scored_tiles_attributes();

}  // namespace pa

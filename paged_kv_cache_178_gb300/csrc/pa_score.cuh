// What the kernels of pa_paged_attention_scored share: the call's parameters,
// which keys a row sees, its scores, and one row computed plainly.
#pragma once
#include <cuda_bf16.h>

#include "pa_attn_common.cuh"

namespace pa {

constexpr float kLog2e = 1.4426950408889634f;

struct ScoreParams {
    const __nv_bfloat16 *q;
    int64_t q_tok_stride;
    const __nv_bfloat16 *k, *v;
    int64_t num_blocks, block_stride, token_stride, head_stride;  // elements
    const int32_t *block_tables, *seq_lens, *qsl;
    const float *slopes;
    const int32_t *prefix_lens, *first_keys;
    __nv_bfloat16 *out;
    float *lse;
    ErrState *err;
    int64_t num_q_tokens;
    int32_t max_blocks, num_seqs, hq, hkv, group, max_query_len, max_seq_len;
    int32_t window;    // INT32_MAX: none
    float scale_log2;  // without a cap: scale * log2 e; with one: 2 * scale * log2 e / cap
    float cap_log2;    // cap * log2 e (0: no cap)
};

__device__ __forceinline__ ReqMeta score_meta(const ScoreParams &p, int b)
{
    ReqMeta m;
    const int qs = __ldg(p.qsl + b), qe = __ldg(p.qsl + b + 1), L = __ldg(p.seq_lens + b);
    m.qs = qs;
    m.qn = qe - qs;
    m.L = L;
    m.sane = qs >= 0 && qe >= qs && (int64_t)qe <= p.num_q_tokens;
    m.ok = m.sane && L >= m.qn && (int64_t)L <= (int64_t)p.max_blocks * 16 && m.qn <= p.max_query_len &&
           L <= p.max_seq_len;
    return m;
}

// Tokens of the prefix that request b's rows all see.
__device__ __forceinline__ int score_prefix(const ScoreParams &p, int b, int L)
{
    const int x = p.prefix_lens ? __ldg(p.prefix_lens + b) : 0;
    return x < 0 ? 0 : (x < L ? x : L);
}

// First key of the range that ends at position pos (pos + 1: the range is
// empty) for query token t (its index among all tokens).
__device__ __forceinline__ int score_low(const ScoreParams &p, int64_t t, int pos)
{
    const int first = p.first_keys ? __ldg(p.first_keys + t) : 0;
    int lo = first > 0 ? first : 0;
    if (pos - p.window >= lo)  // (no overflow: both are at least 0 ... INT32_MAX)
        lo = pos - p.window + 1;
    return lo <= pos ? lo : pos + 1;
}

// Distance from pos to the nearest key that a row sees.  Biases are taken
// relative to it: what is common to a row's keys would cost bits far away.
__device__ __forceinline__ int score_nearest(int lo, int pos, int prefix)
{
    return lo <= pos || prefix == 0 || pos < prefix ? 0 : pos - prefix + 1;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ln(l 2^m) - off, for a maximum m in log2 units and a sum l relative to it.  The
// power of two in l goes to m with the rounding of that sum kept, so that the
// error is the result's own half unit and what l brings (one logarithm of the
// whole sum was off by up to four units).
__device__ __forceinline__ float score_lse(float m, float l, float off)
{
    constexpr float kLn2Low = (float)(0.69314718055994530942 - (double)kLn2);
    if (l == 0.f)
        return -INFINITY;
    if (!(l < INFINITY))
        return l;
    int e = (__float_as_int(l) >> 23) - 127;
    float f = __int_as_float((__float_as_int(l) & 0x7fffff) | 0x3f800000);
    if (f > 1.41421356f) {
        f *= 0.5f;
        ++e;
    }
    const float x = (float)e, hi = m + x, y = hi - m, low = (m - (hi - y)) + (x - y);
    return __fmaf_rn(hi, kLn2, __fmaf_rn(hi, kLn2Low, __fmaf_rn(low, kLn2, logf(f)))) - off;
}

// tanh(y) / y as a polynomial in y^2 for |y| <= kTanhReach (least squares with
// weights moved to the largest errors: off by 5.8e-08 of itself at most).
// (For |y| <= 1/2 it is 2.3e-6 of itself, which lse showed, and another term took
// the prompts 4 percent of the time.)
constexpr float kTanhReach = 0.375f;
constexpr float kTanh0 = 0.9999999418615936f, kTanh1 = -0.33331991737634636f, kTanh2 = 0.13284822465485238f,
                kTanh3 = -0.04828743407056177f;

// cap * tanh(s / cap) in log2 units from the raw product q.k, as
// cap (1 - 2 / (1 + exp(2 s / cap))): exact limits at both ends, an absolute
// error of about 2^-22 cap.  exp takes differences of scores, so the absolute error
// is what counts, and it has to be small beside 1: for cap_log2 <= kCapNarrow.
constexpr float kCapNarrow = 80.f;
__device__ __forceinline__ float capped(float raw, float scale_log2, float cap_log2)
{
    const float e = ex2(raw * scale_log2);
    return __fmaf_rn(-2.f * cap_log2, rcp_approx(1.f + e), cap_log2);
}

// The same for any cap: where the score is small beside it the polynomial, whose
// error is a few roundings of the score itself.  (By the form above alone the
// largest cap, 2^20, cost single scores 0.1.)
__device__ __forceinline__ float capped_wide(float raw, float scale_log2, float cap_log2)
{
    const float y = raw * (scale_log2 * (0.5f * kLn2)), u = y * y;
    const float near = cap_log2 * (y * __fmaf_rn(__fmaf_rn(__fmaf_rn(kTanh3, u, kTanh2), u, kTanh1), u, kTanh0));
    return fabsf(y) <= kTanhReach ? near : capped(raw, scale_log2, cap_log2);
}

// One (token, head) row by one warp, key by key, over exactly the keys that it
// sees: what no row sees is not read, so nothing there (NaN, infinities, a
// page of another request) can matter.  Who finds its part of a row not finite
// has that part written, columns [c0, c0 + cols) (multiples of 32) and, with_lse,
// the row's lse: others may be storing theirs.
template <int DH>
__device__ __noinline__ void scored_row(const ScoreParams &p, int b, const ReqMeta &m, int i, int h, int c0, int cols,
                                        bool with_lse)
{
    constexpr int E = DH / 32;  // elements of a lane
    const int lane = threadIdx.x % 32, kvh = h / p.group;
    const int64_t t = (int64_t)m.qs + i;
    const int pos = m.L - m.qn + i, prefix = score_prefix(p, b, m.L), lo = score_low(p, t, pos);
    const int near = score_nearest(lo, pos, prefix);
    const float slope = p.slopes ? __ldg(p.slopes + h) : 0.f, slope2 = slope * kLog2e;
    const __nv_bfloat16 *qr = p.q + t * p.q_tok_stride + (int64_t)h * DH;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(qr[e * 32 + lane]);
        o[e] = 0.f;
    }
    // Sums of 2^-32 of the values: up to 2^31 of the largest stay below infinity, and
    // what that costs those below 2^-94 is less than 2^-116.  Every weight is
    // positive, also one below the smallest of 32 bits: an infinite value or a NaN
    // counts as it is.
    constexpr float kDown = 0x1p-32f, kUp = 0x1p32f;
    float mx = -INFINITY, l = 0.f;
    bool bad = false;
    const int32_t *bt = p.block_tables + (int64_t)b * p.max_blocks;
    // the prefix first, then what the range adds to it
    const int from[2] = {0, lo > prefix ? lo : prefix}, to[2] = {prefix, pos + 1};
    for (int part = 0; part < 2; ++part) {
        int id = -1;
        for (int j = from[part]; j < to[part]; ++j) {
            if (j == from[part] || j % 16 == 0)
                id = __ldg(bt + j / 16);
            if (id < 0 || (int64_t)id >= p.num_blocks) {
                bad = true;
                break;
            }
            const int64_t at = id * p.block_stride + (j % 16) * p.token_stride + kvh * p.head_stride;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                s = __fmaf_rn(q[e], __bfloat162float(p.k[at + e * 32 + lane]), s);
#pragma unroll
            for (int o2 = 16; o2 >= 1; o2 >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o2);
            float z = p.cap_log2 > kCapNarrow ? capped_wide(s, p.scale_log2, p.cap_log2)
                      : p.cap_log2 > 0.f      ? capped(s, p.scale_log2, p.cap_log2)
                                              : s * p.scale_log2;
            if (p.slopes)
                z -= slope2 * (float)((pos > j ? pos - j : j - pos) - near);
            const float m_new = fmaxf(mx, z);
            const float keep = mx == m_new ? 1.f : ex2(mx - m_new);
            const float w = z == -INFINITY ? 0.f : ex2(z - m_new);
            l = l * keep + w;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e * 32 >= c0 && e * 32 < c0 + cols) {
                    const float v = __bfloat162float(p.v[at + e * 32 + lane]);
                    o[e] = o[e] * (fabsf(o[e]) < INFINITY ? keep : 1.f) + (fabsf(v) < INFINITY ? w * (v * kDown) : v);
                }
            mx = m_new;
        }
    }
    const float inv = bad ? __int_as_float(0x7FC00000) : (l > 0.f || l != l ? 1.f / l : 0.f);
    __nv_bfloat16 *dst = p.out + (t * p.hq + h) * DH;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e * 32 >= c0 && e * 32 < c0 + cols)
            dst[e * 32 + lane] = __float2bfloat16_rn(o[e] * inv * kUp);
    if (lane == 0 && with_lse && p.lse)
        p.lse[t * p.hq + h] = bad ? __int_as_float(0x7FC00000)
                                  : score_lse(mx, l, slope * (float)near);
    if (bad && lane == 0)
        record_error(p.err, kErrBadMetadata, b);
}

}  // namespace pa

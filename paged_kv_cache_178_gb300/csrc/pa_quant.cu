// 4-bit cache: the slot-mapped write and the read-back of the pages that the
// block tables select.  Layout and conversions: pa_quant_common.cuh.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_attn_common.cuh"
#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_quant_common.cuh"
#include "pa_scan.cuh"

namespace pa {

constexpr int kQuantThreads = 256;
// CTAs per SM that write K, and as many V: one wave each.  16384 tokens of 8 KV
// heads and their read-back: 84.8 us at 4, 80.9 at 5, 82.5 at 8.
constexpr int kWriteCtas = 5;

// ---------------------------------------------------------------- write ----
// One thread per block of 16 elements: scale = e4m3(max / 6), codes =
// e2m1(x / scale).  The quotient is computed as x times a reciprocal r of the
// scale (good to 2^-22) plus one correction by its exact residual,
//   q0 = x*r,  q = q0 + (x - q0*scale)*r,
// which gives the exact value whenever x/scale is a tie of the code (x has
// 8 significant bits and the scale 4, so quotients that are not ties stay
// 2^-12 away from one, and a tie is representable).
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Quantised {
    uint32_t scale;    // e4m3 byte
    uint32_t code[2];  // 16 codes, element i in bits 4i
};

__device__ __forceinline__ Quantised quantise16(const uint4 &lo, const uint4 &hi, float tensor_scale,
                                                float inv_tensor_scale)
{
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    // largest magnitude as BF16 bits (an infinity or NaN is at least 0x7F80)
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    const uint32_t top = max(m & 0xffffu, m >> 16);
    Quantised o;
    if (top >= 0x7F80u) {
        o.scale = 0x7F;  // NaN: the whole block reads back as NaN
        o.code[0] = o.code[1] = 0u;
        return o;
    }
    const float amax = __uint_as_float(top << 16) * inv_tensor_scale;
    uint16_t sc;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sc) : "f"(0.f), "f"(amax * (1.f / 6.f)));
    o.scale = sc & 0xffu;
    if (o.scale == 0) {
        // codes of zero, the signs kept
        o.code[0] = o.code[1] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o.code[i / 4] |= (((w[i] >> 15) & 1u) << 3 | ((w[i] >> 31) & 1u) << 7) << (8 * (i % 4));
        return o;
    }
    const uint32_t sp = e4m3x2_to_f16x2(o.scale);
    const float s0 = __half2float(__ushort_as_half((unsigned short)(sp & 0xffffu)));
    // the tensor scale is a power of two: its products are exact
    const float s = s0 * tensor_scale, r = rcp_approx(s0) * inv_tensor_scale;
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        q[i] = __uint_as_float(i % 2 ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    if (o.scale == 0x7E) {
        // a saturated scale: values far above the largest code, up to
        // infinity after the product, would leave no finite residual
        const float cap = 65536.f * s;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            q[i] = fminf(fmaxf(q[i], -cap), cap);
    }
    // Everything with the sign turned, -q: a residual of zero is +0 for x of
    // either sign, its product with -r is then -0, which changes no summand,
    // the zeros of x = +0 and -0 included (with +r a -0 would be lost in the sum).
    const uint64_t nr = pack_f32x2(-r, -r), ss = pack_f32x2(s, s), nz = pack_f32x2(-0.f, -0.f);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const uint64_t x = pack_f32x2(q[i], q[i + 1]);
        const uint64_t n0 = fma_f32x2(x, nr, nz);  // -q0
        unpack_f32x2(fma_f32x2(fma_f32x2(n0, ss, x), nr, n0), q[i], q[i + 1]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(o.code[k])
            : "f"(q[8 * k]), "f"(q[8 * k + 1]), "f"(q[8 * k + 2]), "f"(q[8 * k + 3]), "f"(q[8 * k + 4]),
              "f"(q[8 * k + 5]), "f"(q[8 * k + 6]), "f"(q[8 * k + 7]));
        o.code[k] ^= 0x88888888u;  // the sign turned back
    }
    return o;
}

// K items run with the 16-element block fastest (a token's codes are
// contiguous), V items with the token fastest in groups of 16 (the codes of
// neighbouring tokens are): neighbouring lanes then store neighbouring bytes
// when the slots are consecutive, as in a prompt.  V lanes in fours whose slots
// are four aligned neighbours swap bytes, so that each stores four tokens of
// two element pairs as words, instead of one token of eight as bytes.  A thread
// loads its next item before it works on one.  The index arithmetic is 32 bits
// wide while the items allow; in 64 bits it took as long as the rest.
//
// 16384 tokens of 8 KV heads take 24 us at head dim 128, alone and with cold
// caches, where moving their 86 MB takes 13.  62% of the issue slots are taken
// (240 instructions per 16 elements of K or V) by 56% of the warps that an SM
// holds: neither alone bounds it, the instructions and what little is in flight
// (one item ahead) do together.
template <int DH, typename Index>
__global__ void __launch_bounds__(kQuantThreads) quant_write_kernel(
    const uint4 *__restrict__ key, int64_t key_stride, const uint4 *__restrict__ value, int64_t value_stride,
    int64_t num_tokens, QuantPool pool, const int64_t *__restrict__ slot_mapping, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int NB = DH / 16;  // blocks of a row
    const Index hk = (Index)pool.num_kv_heads;
    const int64_t num_slots = pool.num_blocks * 16;
    const Index groups = (Index)((num_tokens + 15) / 16);
    const Index per_kind = groups * 16 * hk * NB;  // whole groups of 16 tokens, so whole warps
    const bool is_v = blockIdx.y != 0;
    const float scale = is_v ? pool.v_scale : pool.k_scale, inv = 1.f / scale;
    const uint4 *const base = is_v ? value : key;
    const int64_t stride = is_v ? value_stride : key_stride;
    uint8_t *const out = is_v ? pool.v : pool.k;
    const uint32_t block_stride = (uint32_t)pool.block_stride, head_stride = (uint32_t)pool.head_stride;
    struct Item {
        uint4 a, b;
        int64_t slot;
        uint32_t h, blk;
    };
    auto fetch = [&](Index i, Item &x) {
        x.a = x.b = make_uint4(0u, 0u, 0u, 0u);
        x.slot = -1;
        x.h = x.blk = 0;
        if (i >= per_kind)
            return;
        Index t;
        if (is_v) {
            const Index y = i / (16 * NB);
            x.blk = (uint32_t)(i / 16 % NB);
            x.h = (uint32_t)(y % hk);
            t = y / hk * 16 + i % 16;
        } else {
            const Index y = i / NB;
            x.blk = (uint32_t)(i % NB);
            x.h = (uint32_t)(y % hk);
            t = y / hk;
        }
        if ((int64_t)t >= num_tokens)
            return;
        const uint4 *src = base + (int64_t)t * stride + (x.h * (DH / 8) + 2 * x.blk);
        x.a = __ldg(src);
        x.b = __ldg(src + 1);
        x.slot = __ldg(slot_mapping + t);
        if (x.slot >= num_slots) {
            if (!is_v && x.blk == 0 && x.h == 0)
                record_error(err, kErrBadMetadata, (long long)t);
            x.slot = -1;
        }
    };
    const Index step = (Index)gridDim.x * kQuantThreads;
    Index i = (Index)blockIdx.x * kQuantThreads + threadIdx.x;
    Item next;
    fetch(i, next);
    for (; i < per_kind; i += step) {
        const Item x = next;
        fetch(i + step, next);
        const Quantised q = quantise16(x.a, x.b, scale, inv);
        const int tok = (int)(x.slot & 15);
        uint8_t *rec = out + (x.slot >> 4) * block_stride + (uint64_t)x.h * head_stride;
        if (is_v) {
            const int me = threadIdx.x & 3;
            const uint32_t first = __shfl_sync(0xffffffffu, (uint32_t)x.slot, threadIdx.x & 28);
            const uint32_t first_hi = __shfl_sync(0xffffffffu, (uint32_t)(x.slot >> 32), threadIdx.x & 28);
            const bool four = x.slot >= 0 && (int64_t)((uint64_t)first_hi << 32 | first) == x.slot - me && (first & 3) == 0;
            uint8_t *p = rec + x.blk * 128 + tok;
            if (__all_sync(0xffffffffu, four)) {
                // byte j of lane k -> byte k of lane j, for both words
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t w = q.code[k];
                    uint32_t y = __shfl_xor_sync(0xffffffffu, w, 1);
                    w = __byte_perm(w, y, me & 1 ? 0x3715 : 0x6240);
                    y = __shfl_xor_sync(0xffffffffu, w, 2);
                    w = __byte_perm(w, y, me & 2 ? 0x3276 : 0x5410);
                    *reinterpret_cast<uint32_t *>(p - me + (4 * k + me) * 16) = w;
                }
            } else if (x.slot >= 0) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    p[c * 16] = (uint8_t)(q.code[c / 4] >> (8 * (c % 4)));
            }
            if (x.slot >= 0)
                rec[quant_code_bytes(DH) + x.blk * 16 + tok] = (uint8_t)q.scale;
        } else if (x.slot >= 0) {
            *reinterpret_cast<uint2 *>(rec + tok * (DH / 2) + x.blk * 8) = make_uint2(q.code[0], q.code[1]);
            rec[quant_code_bytes(DH) + tok * NB + x.blk] = (uint8_t)q.scale;
        }
    }
}

template <typename Index>
static auto quant_write_of(int head_dim)
{
    return head_dim == 128 ? quant_write_kernel<128, Index>
                           : (head_dim == 256 ? quant_write_kernel<256, Index> : quant_write_kernel<512, Index>);
}

cudaError_t launch_quant_write(const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                               int64_t num_tokens, const QuantPool &pool, const int64_t *slot_mapping, ErrState *err,
                               cudaStream_t stream, int num_sms, int64_t *grid)
{
    const int64_t items = (num_tokens + 15) / 16 * 16 * pool.num_kv_heads * (pool.head_dim / 16);
    int64_t blocks = (items + kQuantThreads - 1) / kQuantThreads;
    if (blocks > (int64_t)num_sms * kWriteCtas)
        blocks = (int64_t)num_sms * kWriteCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 2);
    cfg.blockDim = dim3(kQuantThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *grid = 2 * blocks;
    // the loop's last step and its fetch may pass the items by two grids
    const bool narrow = items + 2 * blocks * kQuantThreads <= (int64_t)UINT32_MAX;
    auto kern = narrow ? quant_write_of<uint32_t>(pool.head_dim) : quant_write_of<uint64_t>(pool.head_dim);
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const uint4 *>(key), key_stride / 8,
                              static_cast<const uint4 *>(value), value_stride / 8, num_tokens, pool, slot_mapping,
                              err);
}

// ------------------------------------------------------------- read-back ----
// Bound by the BF16 bytes it writes (16 of every 20.5 bytes moved).  Eight
// codes (one 32-bit word) become one 16-byte store.  A warp takes a run of
// units of 4096 elements of K and of V (two records at head dim 128, one at
// 256, half of one at 512).  K: neighbouring lanes take neighbouring words of
// a token.  V: a lane takes eight head-dim elements of all 16 tokens (four
// 16-byte loads, the bytes regrouped by token with permutes), neighbouring
// lanes neighbouring elements; every store instruction then covers whole rows.
// 66 thousand tokens of 8 KV heads at head dim 128 (76 MB read, 268 written)
// take 57 us alone, 6.0 TB/s, with three CTAs per SM.  (Marked as streaming,
// loads and stores took 67 us instead of 71 in a row of launches, but write and
// read-back of 19 thousand tokens of 2 KV heads 11.0 instead of 9.9: what is
// read back is read again soon.)
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t scale_pair, float tensor_scale)
{
    uint32_t p[4];
    e2m1x8_to_f16x2(codes, p);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = mul_f16x2(p[i], scale_pair);  // exact
        const __half2 hv = *reinterpret_cast<const __half2 *>(&v);
        const float2 f = __half22float2(hv);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * tensor_scale, f.y * tensor_scale);  // exact
        o[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int DH>
__global__ void __launch_bounds__(kQuantThreads) dequantize_kv_kernel(
    QuantPool pool, const int32_t *__restrict__ block_tables, int32_t max_blocks,
    const int32_t *__restrict__ seq_lens, int32_t num_seqs, uint4 *__restrict__ k_out, uint4 *__restrict__ v_out,
    int64_t capacity_pages, int32_t *__restrict__ compact_tables, int32_t out_cols,
    int32_t *__restrict__ compact_offsets, bool poison_tables, uint4 *__restrict__ zero, int64_t zero16, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int32_t s_off[];  // [num_seqs + 1]
    __shared__ long long s_sums[kQuantThreads / 32];
    const int tid = threadIdx.x;
    const int64_t gtid = (int64_t)blockIdx.x * kQuantThreads + tid, gsize = (int64_t)gridDim.x * kQuantThreads;
    for (int64_t i = gtid; i < zero16; i += gsize)
        zero[i] = make_uint4(0u, 0u, 0u, 0u);
    const long long total = block_exclusive_sums<kQuantThreads>(num_seqs, s_off, s_sums, [&](int b) {
        const int L = __ldg(seq_lens + b);
        if (L < 0 || (int64_t)L > (int64_t)out_cols * 16) {
            if (blockIdx.x == 0)
                record_error(err, kErrBadMetadata, b);
            return 0;
        }
        return (L + 15) / 16;
    });
    if (compact_offsets && blockIdx.x == 0)
        for (int b = tid; b <= num_seqs; b += kQuantThreads)
            compact_offsets[b] = s_off[b];
    const bool over = total > capacity_pages;
    if (over && gtid == 0)
        record_error(err, kErrBudget, total);
    if (over && !poison_tables)
        return;
    const int64_t n_tab = (int64_t)num_seqs * out_cols;
    for (int64_t e = gtid; e < n_tab; e += gsize) {
        const int b = (int)div_floor(e, out_cols), p = (int)(e - (int64_t)b * out_cols);
        if (!poison_tables || over || p > 0)
            compact_tables[e] = !over && p < s_off[b + 1] - s_off[b] ? s_off[b] + p : -1;
    }
    if (over)
        return;
    if (poison_tables)
        // The first entry of each request: -1 if any of its block ids is bad.
        // Every row sees that page, so all of the request's rows become NaN,
        // whether they see the bad one or not.
        for (int b = blockIdx.x; b < num_seqs; b += gridDim.x) {
            const int n = s_off[b + 1] - s_off[b];
            bool bad = n == 0;
            for (int p = tid; p < n; p += kQuantThreads) {
                const int id = __ldg(block_tables + (int64_t)b * max_blocks + p);
                bad |= id < 0 || (int64_t)id >= pool.num_blocks;
            }
            bad = __syncthreads_or(bad);
            if (tid == 0)
                compact_tables[(int64_t)b * out_cols] = bad ? -1 : s_off[b];
        }
    constexpr int VEC = DH / 8;  // 16-byte vectors of an output row
    const int hk = pool.num_kv_heads;
    const uint4 qnan = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    // this warp's units, one after another: consecutive records, so the
    // request and the block id follow with the page (dealt in turn to the
    // warps of a CTA instead, so that they write next to one another, no faster)
    const int lane = tid & 31;
    const int64_t records = (int64_t)total * hk, units = (records * DH + 255) / 256;
    const int64_t warps = gsize / 32, w = gtid / 32;
    const int64_t u_lo = div_floor(w * units, warps), u_hi = div_floor((w + 1) * units, warps);
    // per lane: the page a record index stands in, followed as it grows
    struct Where {
        int64_t rec;  // record index (page * heads + head)
        int c, h, b, id;
    };
    auto seek = [&](Where &x, int64_t rec) {
        x.rec = rec;
        if (rec >= records)
            return;
        x.c = (int)div_floor(rec, hk);
        x.h = (int)(rec - (int64_t)x.c * hk);
        x.b = owner_of(s_off, num_seqs, x.c);
        x.id = __ldg(block_tables + (int64_t)x.b * max_blocks + (x.c - s_off[x.b]));
    };
    auto advance = [&](Where &x, int by) {
        x.rec += by;
        if (x.rec >= records)
            return;
        x.h += by;
        bool moved = false;
        while (x.h >= hk) {
            x.h -= hk;
            ++x.c;
            moved = true;
        }
        if (moved) {
            while (x.c >= s_off[x.b + 1])
                ++x.b;
            x.id = __ldg(block_tables + (int64_t)x.b * max_blocks + (x.c - s_off[x.b]));
        }
    };
    auto good = [&](const Where &x) { return x.id >= 0 && (int64_t)x.id < pool.num_blocks; };
    constexpr int RPU = DH == 128 ? 2 : 1;    // records of a unit
    constexpr int HPR = DH == 512 ? 2 : 1;    // units of a record
    Where kx[RPU], vx;
#pragma unroll
    for (int j = 0; j < RPU; ++j)
        seek(kx[j], u_lo / HPR * RPU + j);
    seek(vx, u_lo / HPR * RPU + (RPU == 2 ? lane / 16 : 0));
    for (int64_t u = u_lo; u < u_hi; ++u) {
        // --- K: 512 words, sixteen a lane
        const int part = HPR == 2 ? (int)(u & 1) : 0;  // tokens 8*part.. of the record
#pragma unroll
        for (int j = 0; j < RPU; ++j) {
            constexpr int STEPS = 16 / RPU;
            if (kx[j].rec < records) {
                const bool ok = good(kx[j]);
                const uint8_t *rec = pool.k + (int64_t)(ok ? kx[j].id : 0) * pool.block_stride + kx[j].h * pool.head_stride;
                uint32_t word[STEPS];
                uint8_t sb[STEPS];
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int x = 512 * part + 32 * i + lane;
                    word[i] = __ldg(reinterpret_cast<const uint32_t *>(rec) + x);
                    sb[i] = __ldg(rec + quant_code_bytes(DH) + x / 2);
                }
                uint4 *dst = k_out + ((int64_t)kx[j].c * 16 * hk + kx[j].h) * VEC;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int x = 512 * part + 32 * i + lane;
                    const uint32_t s = e4m3x2_to_f16x2(sb[i]);
                    dst[(int64_t)(x / VEC) * hk * VEC + x % VEC] =
                        ok ? values8(word[i], __byte_perm(s, 0u, 0x1010), pool.k_scale) : qnan;
                }
            }
        }
        // --- V: eight elements of all tokens a lane
        if (vx.rec < records) {
            const int i = (RPU == 2 ? lane % 16 : lane) + 32 * part;
            const bool ok = good(vx);
            if (!ok && i == 0 && vx.h == 0)
                record_error(err, kErrBadMetadata, vx.b);
            const uint8_t *rec = pool.v + (int64_t)(ok ? vx.id : 0) * pool.block_stride + vx.h * pool.head_stride;
            uint4 *dst = v_out + ((int64_t)vx.c * 16 * hk + vx.h) * VEC + i;
            uint4 col[4];  // element pairs 4i .. 4i+3, sixteen tokens each
#pragma unroll
            for (int j = 0; j < 4; ++j)
                col[j] = __ldg(reinterpret_cast<const uint4 *>(rec) + 4 * i + j);
            const uint4 sc = __ldg(reinterpret_cast<const uint4 *>(rec + quant_code_bytes(DH)) + i / 2);
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4) {
                auto part4 = [&](const uint4 &v) { return t4 == 0 ? v.x : t4 == 1 ? v.y : t4 == 2 ? v.z : v.w; };
                const uint32_t w0 = part4(col[0]), w1 = part4(col[1]), w2 = part4(col[2]), w3 = part4(col[3]);
                // 4x4 byte transpose: tokens 4*t4 .. +3
                const uint32_t a = __byte_perm(w0, w1, 0x5140), bb = __byte_perm(w0, w1, 0x7362);
                const uint32_t e = __byte_perm(w2, w3, 0x5140), f = __byte_perm(w2, w3, 0x7362);
                const uint32_t tw[4] = {__byte_perm(a, e, 0x5410), __byte_perm(a, e, 0x7632),
                                        __byte_perm(bb, f, 0x5410), __byte_perm(bb, f, 0x7632)};
                const uint32_t s4 = part4(sc);
                const uint32_t s01 = e4m3x2_to_f16x2(s4), s23 = e4m3x2_to_f16x2(s4 >> 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t sp = __byte_perm(k < 2 ? s01 : s23, 0u, k % 2 ? 0x3232 : 0x1010);
                    dst[(int64_t)(4 * t4 + k) * hk * VEC] = ok ? values8(tw[k], sp, pool.v_scale) : qnan;
                }
            }
        }
        if (HPR == 1 || (u & 1)) {
#pragma unroll
            for (int j = 0; j < RPU; ++j)
                advance(kx[j], RPU);
            advance(vx, RPU);
        }
    }
}

cudaError_t launch_dequantize_kv(const QuantPool &pool, const int32_t *block_tables, int32_t max_blocks,
                                 const int32_t *seq_lens, int32_t num_seqs, void *k_out, void *v_out,
                                 int64_t capacity_pages, int32_t *compact_tables, int32_t out_cols,
                                 int32_t *compact_offsets, bool poison_tables, void *zero, size_t zero_bytes,
                                 ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid)
{
    int64_t pages = (int64_t)num_seqs * out_cols;
    if (pages > capacity_pages)
        pages = capacity_pages;
    // one unit a warp, at most one wave
    constexpr int kWarpsPerCta = kQuantThreads / 32;
    int64_t blocks = (pages * pool.num_kv_heads * pool.head_dim / 256 + kWarpsPerCta - 1) / kWarpsPerCta;
    const int64_t tab = ((int64_t)num_seqs * out_cols + kQuantThreads - 1) / kQuantThreads;
    if (blocks < tab)
        blocks = tab;
    if (blocks > (int64_t)num_sms * 3)
        blocks = (int64_t)num_sms * 3;
    if (blocks < 1)
        blocks = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kQuantThreads);
    cfg.dynamicSmemBytes = (size_t)(num_seqs + 1) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *grid = blocks;
    void (*kern)(QuantPool, const int32_t *, int32_t, const int32_t *, int32_t, uint4 *, uint4 *, int64_t, int32_t *,
                 int32_t, int32_t *, bool, uint4 *, int64_t, ErrState *) =
        pool.head_dim == 128 ? dequantize_kv_kernel<128>
                             : (pool.head_dim == 256 ? dequantize_kv_kernel<256> : dequantize_kv_kernel<512>);
    return cudaLaunchKernelEx(&cfg, kern, pool, block_tables, max_blocks, seq_lens, num_seqs,
                              static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out), capacity_pages, compact_tables,
                              out_cols, compact_offsets, poison_tables, static_cast<uint4 *>(zero),
                              (int64_t)(zero_bytes / 16), err);
}

cudaError_t init_quant_attributes()
{
    const int bytes = (kScanMaxSeqs + 1) * 4;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(dequantize_kv_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(dequantize_kv_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) !=
            cudaSuccess)
        return e;
    return cudaFuncSetAttribute(dequantize_kv_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace pa

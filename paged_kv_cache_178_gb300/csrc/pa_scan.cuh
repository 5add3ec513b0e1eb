// Block-wide exclusive sums over the requests of a batch, shared by the
// kernels that turn per-request lengths into offsets.
#pragma once
#include <cstdint>

namespace pa {

// floor(a / b), 0 <= a, 0 < b: one 32-bit division when both fit
__device__ __forceinline__ int64_t div_floor(int64_t a, int64_t b)
{
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0)
        return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Largest batch those kernels take: their offsets sit in shared memory.
constexpr int kScanMaxSeqs = 8192;

// Adds up what the warps of a CTA left in warp_sums: `before` gets the sums of
// the warps before this one, `all` those of all NTH / 32.  (In 32 bits a lane
// reads one and the warp reduces: with 32 warps that read all 32, the reads took a
// thousand cycles.)
template <int NTH, typename Sum>
__device__ __forceinline__ void add_warp_sums(const Sum *warp_sums, int stride, Sum &before, Sum &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (sizeof(Sum) == 4) {
        const Sum s = lane < NTH / 32 ? warp_sums[lane * stride] : 0;
        before += __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
        all += __reduce_add_sync(0xffffffffu, s);
    } else {
#pragma unroll
        for (int w = 0; w < NTH / 32; ++w) {
            const Sum s = warp_sums[w * stride];
            before += w < warp ? s : 0;
            all += s;
        }
    }
}

// Exclusive prefix sums of count(b), b in [0, n), into off[0..n] (off[n] =
// the total) by all NTH threads of the CTA.  The returned total is exact in
// 64 bits; off[] holds the low 32 bits, so callers check the total against
// their own (32-bit) limit before they use it.  `warp_sums` is scratch for
// NTH/32 values; of type int where the sums are known to fit.  Ends with a CTA
// barrier.
template <int NTH, typename Sum, typename Count>
__device__ __forceinline__ Sum block_exclusive_sums(int n, int32_t *off, Sum *warp_sums, Count count)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Sum base = 0;
    for (int b0 = 0; b0 < n; b0 += NTH) {
        const int b = b0 + tid;
        const Sum c = b < n ? (Sum)count(b) : 0;
        Sum incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sum x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += x;
        }
        if (lane == 31)
            warp_sums[warp] = incl;
        __syncthreads();
        Sum before = base, total = base;
        add_warp_sums<NTH>(warp_sums, 1, before, total);
        if (b < n)
            off[b] = (int32_t)(before + incl - c);
        base = total;
        __syncthreads();  // warp_sums is reused by the next pass
    }
    if (tid == 0)
        off[n] = (int32_t)base;
    __syncthreads();
    return base;
}

// The same for two counts at once: count(b, first, second).  Pair is longlong2,
// or int2 where the sums are known to fit.
template <int NTH, typename Pair, typename Count>
__device__ __forceinline__ void block_exclusive_sums2(int n, int32_t *off0, int32_t *off1, Pair *warp_sums, Pair &total,
                                                      Count count)
{
    using Sum = decltype(Pair::x);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Pair base{0, 0};
    for (int b0 = 0; b0 < n; b0 += NTH) {
        const int b = b0 + tid;
        int c0 = 0, c1 = 0;
        if (b < n)
            count(b, c0, c1);
        Sum i0 = c0, i1 = c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sum x0 = __shfl_up_sync(0xffffffffu, i0, o), x1 = __shfl_up_sync(0xffffffffu, i1, o);
            if (lane >= o) {
                i0 += x0;
                i1 += x1;
            }
        }
        if (lane == 31)
            warp_sums[warp] = Pair{i0, i1};
        __syncthreads();
        Pair before = base;
        add_warp_sums<NTH>(&warp_sums->x, 2, before.x, base.x);
        add_warp_sums<NTH>(&warp_sums->y, 2, before.y, base.y);
        if (b < n) {
            off0[b] = (int32_t)(before.x + i0 - c0);
            off1[b] = (int32_t)(before.y + i1 - c1);
        }
        if (b0 + NTH < n)
            __syncthreads();  // warp_sums is reused by the next pass
    }
    if (tid == 0) {
        off0[n] = (int32_t)base.x;
        off1[n] = (int32_t)base.y;
    }
    total = base;
    __syncthreads();
}

// The last b in [0, n) with off[b] <= x: the request that owns item x (off[]
// as above, x below the total; requests without items are passed over).
__device__ __forceinline__ int owner_of(const int32_t *off, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

}  // namespace pa

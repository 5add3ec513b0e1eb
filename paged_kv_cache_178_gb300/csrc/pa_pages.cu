// Pages of a cache between its requests: copies of pages (pa_copy_pages,
// pa_copy_pages_quant), forks that share whole pages (pa_fork_requests), the
// release of pages (pa_release_pages) and the compaction of a pool
// (pa_compact_pages).
//
// shares[p] counts the owners of page p beyond its first, so a free page and a
// page of one request both hold 0 and pa_build_step_metadata needs to know
// nothing of it.
#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_scan.cuh"

namespace pa {

// ------------------------------------------------------------ page copies --
// Bytes in, bytes out: bound by the memory (2000 pages of 8 heads of 128 in two
// layers: 78.9 us, 6.65 TB/s; 16 pages in four layers: 2.8 us; in 4 bits 2000 pages
// of 8 heads in two layers 24.0 us, 6.1 TB/s, 8000 of one head in four 28.7: a
// view's page is then 72 vectors, of which a warp could take 256).  A warp takes 4 KB of one view
// (K or V) of one page at a time, eight 16-byte vectors a lane, all loaded
// before the first is stored.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyUnit = 32 * kCopyUnroll;  // vectors

// FLAT: a view's page is one run of bytes; otherwise it is c0 x c1 runs of
// run_vecs vectors.
template <bool FLAT>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32;
    const uint32_t upp = (uint32_t)(a.page_vecs + kCopyUnit - 1) / kCopyUnit;  // units of a page
    const int64_t per_view = (int64_t)a.num_pairs * upp, units = per_view * a.num_caches * 2;
    const int64_t step = (int64_t)gridDim.x * (kCopyThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32; u < units; u += step) {
        const int64_t view = div_floor(u, per_view), w = u - view * per_view, pair = div_floor(w, upp);
        const int part = (int)(w - pair * upp);
        const int src = __ldg(a.src + pair), dst = __ldg(a.dst + pair);
        if (src < 0 || src == dst)
            continue;
        if (src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
            if (view == 0 && part == 0 && lane == 0)
                record_error(err, kErrBadMetadata, pair);
            continue;
        }
        uint4 *base = (view & 1 ? a.v : a.k)[view >> 1];
        const uint4 *from = base + src * a.block_stride;
        uint4 *to = base + dst * a.block_stride;
        uint4 x[kCopyUnroll];
        auto at = [&](int i) {
            const uint32_t v = (uint32_t)part * kCopyUnit + i * 32 + lane;
            if (FLAT)
                return (int64_t)v;
            const uint32_t run = v / (uint32_t)a.run_vecs, r0 = run / (uint32_t)a.c1;
            return (int64_t)r0 * a.s0 + (int64_t)(run - r0 * a.c1) * a.s1 + (v - run * a.run_vecs);
        };
#pragma unroll
        for (int i = 0; i < kCopyUnroll; ++i)
            if (part * kCopyUnit + i * 32 + lane < a.page_vecs)
                x[i] = from[at(i)];
#pragma unroll
        for (int i = 0; i < kCopyUnroll; ++i)
            if (part * kCopyUnit + i * 32 + lane < a.page_vecs)
                to[at(i)] = x[i];
    }
}

cudaError_t launch_copy_pages(const CopyArgs &a, ErrState *err, cudaStream_t stream, int num_sms, int64_t *grid)
{
    const int64_t units = (int64_t)a.num_caches * 2 * a.num_pairs * ((a.page_vecs + kCopyUnit - 1) / kCopyUnit);
    int64_t blocks = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    if (blocks > (int64_t)num_sms * 16)
        blocks = (int64_t)num_sms * 16;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *grid = blocks;
    const bool flat = a.run_vecs == a.page_vecs;
    return cudaLaunchKernelEx(&cfg, flat ? copy_pages_kernel<true> : copy_pages_kernel<false>, a, err);
}

// ------------------------------------------------- fork, release, compact --
// A few KB to a few MB of 32-bit numbers, in phases that depend on one another:
// launch and latency bound.  Each is one kernel of one cluster with a cluster
// barrier between its phases, so that lengths, cursor, counts and tables may
// advance in place.  The sums over the requests are repeated by every CTA.
// A CTA to 1024 pages or so, up to 16: the large calls are bound by what an SM
// does with scattered words (an atomic takes it 3 cycles, a load 1.5).  16
// instead of 8 took 192 forks of 36 k pages from 14.4 to 11.0 us, a release of 35
// k references from 27.4 to 21.6 and a pool of 300000 pages from 34.0 to 24.3.
// Measured: those calls 9.2, 18.8 and 19.5 us; 4 forks of a prompt 4.3 us, the
// drafts of 64 requests 9.4, a pool of 2048 pages 7.5: chains of loads, sums and
// barriers, of some 2 us for a launch.
constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kPageClusterMax = 16;

static cudaError_t launch_cluster(void (*kern)(const PageArgs, ErrState *), const PageArgs &a, ErrState *err,
                                  cudaStream_t stream, int64_t items, size_t smem, int *grid)
{
    int ctas = 1;
    while (ctas < kPageClusterMax && (int64_t)ctas * kPageThreads < items)
        ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPageThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *grid = ctas;
    return cudaLaunchKernelEx(&cfg, kern, a, err);
}

__device__ __forceinline__ int pages_of(int tokens) { return tokens / 16 + (tokens % 16 != 0); }

// Loads that a thread keeps in flight where the next step waits for them.
constexpr int kPageBatch = 8;

// shares_out = shares_in, by all threads of the cluster
__device__ __forceinline__ void copy_shares(const PageArgs &a)
{
    if (a.shares_out == a.shares_in)
        return;
    const int64_t gsize = (int64_t)gridDim.x * kPageThreads, blocks = a.num_blocks;
    for (int64_t p0 = (int64_t)blockIdx.x * kPageThreads + threadIdx.x; p0 < blocks; p0 += gsize * kPageBatch) {
        int32_t v[kPageBatch];
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k)
            v[k] = p0 + k * gsize < blocks ? a.shares_in[p0 + k * gsize] : 0;
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k)
            if (p0 + k * gsize < blocks)
                a.shares_out[p0 + k * gsize] = v[k];
    }
}

__global__ void __launch_bounds__(kPageThreads, 1) fork_requests_kernel(const PageArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int32_t s_fork[];
    __shared__ int2 s_sums[kPageWarps];
    const int n = a.num_forks, tid = threadIdx.x;
    int32_t *s_page = s_fork;         // [n + 1] first page of a fork's child among all
    int32_t *s_tail = s_page + n + 1; // [n + 1] forks before it with a partial page
    int32_t *s_len = s_tail + n + 1;  // [n] tokens (-1: refused)
    int32_t *s_owner = s_len + n;     // [num_seqs] the first fork to a child
    const int64_t limit = (int64_t)a.max_blocks * 16;
    const int cursor = *a.cursor_in;
    for (int b = tid; b < a.num_seqs; b += kPageThreads)
        s_owner[b] = INT32_MAX;
    __syncthreads();
    for (int i = tid; i < n; i += kPageThreads) {
        const int c = a.children[i];
        if (c >= 0 && c < a.num_seqs)
            atomicMin(s_owner + c, i);
    }
    copy_shares(a);
    __syncthreads();
    int2 total;  // (num_seqs * max_blocks is below 2^31)
    block_exclusive_sums2<kPageThreads>(n, s_page, s_tail, s_sums, total, [&](int i, int &pages, int &tails) {
        const int p = a.parents[i], c = a.children[i];
        int len = -1;
        if (p >= 0 && p < a.num_seqs && c >= 0 && c < a.num_seqs && s_owner[c] == i && a.context_lens[c] == 0) {
            const int ctx = a.context_lens[p], l = a.fork_lens ? a.fork_lens[i] : ctx;
            if (ctx >= 0 && (int64_t)ctx <= limit && l >= 0 && l <= ctx)
                len = l;
        }
        s_len[i] = len;
        if (len >= 0) {
            pages = pages_of(len);
            tails = len % 16 != 0;
        } else if (blockIdx.x == 0) {
            record_error(err, kErrBadMetadata, i);
        }
    });
    const int pages = total.x, tails = total.y;
    const bool bad_cursor = cursor < 0 || cursor > a.num_free;
    const bool short_pages = !bad_cursor && tails > a.num_free - cursor;
    const bool empty = bad_cursor || short_pages;
    cluster_sync_all();  // every CTA has read what advances in place; shares_out is complete
    const int gtid = blockIdx.x * kPageThreads + tid, gsize = gridDim.x * kPageThreads;
    if (gtid == 0) {
        if (short_pages)
            record_error(err, kErrBudget, tails);
        else if (empty)
            record_error(err, kErrBadMetadata, n);
        *a.cursor_out = empty ? cursor : cursor + tails;
    }
    for (int b = gtid; b < a.num_seqs; b += gsize) {
        const int i = s_owner[b], len = !empty && i != INT32_MAX ? s_len[i] : -1;
        a.seq_lens[b] = len >= 0 ? len : a.context_lens[b];
    }
    for (int i = gtid; i < n; i += gsize)
        if (empty || s_len[i] < 0 || s_len[i] % 16 == 0)
            a.copy_src[i] = a.copy_dst[i] = -1;
    if (empty)
        return;
    for (int64_t x0 = gtid; x0 < pages; x0 += gsize) {
        const int x = (int)x0, i = owner_of(s_page, n, x), j = x - s_page[i];
        const int id = a.block_tables[(int64_t)a.parents[i] * a.max_blocks + j];
        const bool known = id >= 0 && (int64_t)id < a.num_blocks;
        int entry = id;
        if (j < s_len[i] / 16) {
            if (known)
                atomicAdd(a.shares_out + id, 1);
            else
                record_error(err, kErrBadMetadata, i);
        } else {
            entry = a.free_pages[cursor + s_tail[i]];
            const bool both = known && entry >= 0 && (int64_t)entry < a.num_blocks;
            a.copy_src[i] = both ? id : -1;
            a.copy_dst[i] = both ? entry : -1;
            if (!both)
                record_error(err, kErrBadMetadata, i);
        }
        a.block_tables[(int64_t)a.children[i] * a.max_blocks + j] = entry;
    }
}

static size_t fork_smem(int num_forks, int num_seqs) { return ((size_t)3 * num_forks + 2 + num_seqs) * 4; }

cudaError_t launch_fork_requests(const PageArgs &a, ErrState *err, cudaStream_t stream, int *grid)
{
    const int64_t items = (int64_t)a.num_forks * (a.max_blocks < 512 ? a.max_blocks : 512);
    return launch_cluster(fork_requests_kernel, a, err, stream, items, fork_smem(a.num_forks, a.num_seqs), grid);
}

// The reference that takes a page's last owner is the one that frees it.  In
// order: every dropped reference takes one off its page's count, and those that
// find it 0 are counted: as many pages are freed, and where the stack has no room
// for them the references give back what they took (before anything else has
// become of the counts, so they end as they began); then the
// references of pages whose count went below 0 meet in an atomic minimum of
// -(2^30 + index), which the last of them wins; the winners' order among all
// dropped references gives each page its place on the free stack.  So the
// result is the one of a loop over requests and columns, without one.  A lane
// takes kPageBatch references through each phase at a time (their atomics return
// values: 30.1 -> 21.6 us for 35 k references; a warp to sum one CTA's counts, 18.8).
constexpr int kReleaseMark = 1 << 30;

__global__ void __launch_bounds__(kPageThreads, 1) release_pages_kernel(const PageArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int32_t s_rel[];
    __shared__ int s_sums[kPageWarps];
    __shared__ int32_t s_freed[kPageWarps];  // pages that a warp frees
    __shared__ int32_t s_ctas[kPageClusterMax];
    const int n = a.num_seqs, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int32_t *s_off = s_rel;          // [n + 1] first dropped page of a request among all
    int32_t *s_keep = s_off + n + 1; // [n] tokens that stay
    const int64_t limit = (int64_t)a.max_blocks * 16;
    const int cursor = *a.cursor_in;
    const int total = block_exclusive_sums<kPageThreads>(n, s_off, s_sums, [&](int b) {
        const int c = a.context_lens[b], k = a.keep_lens[b];
        int keep = c;
        bool ok = c >= 0 && (int64_t)c <= limit && k <= c;
        if (ok && k >= 0 && k < c) {
            if (k % 16 != 0) {
                // the page that the kept tokens end in will be written again
                const int id = a.block_tables[(int64_t)b * a.max_blocks + k / 16];
                ok = id >= 0 && (int64_t)id < a.num_blocks && a.shares_in[id] == 0;
            }
            if (ok)
                keep = k;
        }
        if (!ok && blockIdx.x == 0)
            record_error(err, kErrBadMetadata, b);
        s_keep[b] = keep;
        return keep < c ? pages_of(c) - pages_of(keep) : 0;
    });
    copy_shares(a);
    const bool empty = cursor < 0 || cursor > a.num_free || total > kReleaseMark;
    cluster_sync_all();
    const int gtid = blockIdx.x * kPageThreads + tid, gsize = gridDim.x * kPageThreads;
    // a warp takes 32 neighbouring references at a time of a range of its own
    const int items = empty ? 0 : total;
    const int warps = gridDim.x * kPageWarps, per = ((items + warps - 1) / warps + 31) / 32 * 32;
    const int64_t lo = (int64_t)(blockIdx.x * kPageWarps + warp) * per;
    const int64_t hi = lo + per < items ? lo + per : items;
    auto page = [&](int64_t x) {
        const int b = owner_of(s_off, n, (int)x);
        const int id = a.block_tables[(int64_t)b * a.max_blocks + pages_of(s_keep[b]) + (int)x - s_off[b]];
        return id >= 0 && (int64_t)id < a.num_blocks ? id : -1;
    };
    // the pages of a lane's first kPageBatch references stay in registers
    int kept[kPageBatch];
#pragma unroll
    for (int k = 0; k < kPageBatch; ++k)
        kept[k] = lo + lane + 32 * k < hi ? page(lo + lane + 32 * k) : -1;
    // batch by batch: f(first reference of the lane, its pages)
    auto for_batches = [&](auto f) {
        f(lo + lane, kept);
        for (int64_t x0 = lo + lane + 32 * kPageBatch; x0 - lane < hi; x0 += 32 * kPageBatch) {
            int ids[kPageBatch];
#pragma unroll
            for (int k = 0; k < kPageBatch; ++k)
                ids[k] = x0 + 32 * k < hi ? page(x0 + 32 * k) : -1;
            f(x0, ids);
        }
    };
    auto counts_of = [&](const int(&ids)[kPageBatch], int(&v)[kPageBatch]) {
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k)
            v[k] = ids[k] >= 0 ? __ldcg(a.shares_out + ids[k]) : 0;
    };
    // the pages freed by all (s_freed of every warp), and before this warp's: a warp
    // adds up one CTA's counts
    auto sum_freed = [&](int &before) {
        if (warp < (int)gridDim.x) {
            int x;
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(x)
                         : "r"(mapa_shared(smem_addr(s_freed + lane), (uint32_t)warp))
                         : "memory");
            x = __reduce_add_sync(0xffffffffu, x);
            if (lane == 0)
                s_ctas[warp] = x;
        }
        __syncthreads();
        const int x = lane < (int)gridDim.x ? s_ctas[lane] : 0;
        before = __reduce_add_sync(0xffffffffu, (lane < (int)blockIdx.x ? x : 0) + (lane < warp ? s_freed[lane] : 0));
        return __reduce_add_sync(0xffffffffu, x);
    };
    int last = 0, before;
    for_batches([&](int64_t x0, const int(&ids)[kPageBatch]) {
        int v[kPageBatch];
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k)
            v[k] = ids[k] >= 0 ? atomicSub(a.shares_out + ids[k], 1) : -1;
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k) {
            last += v[k] == 0;
            if (v[k] < 0 && x0 + 32 * k < hi)
                record_error(err, kErrBadMetadata, owner_of(s_off, n, (int)(x0 + 32 * k)));
        }
    });
    last = __reduce_add_sync(0xffffffffu, last);
    if (lane == 0)
        s_freed[warp] = last;
    cluster_sync_all();
    const int wanted = sum_freed(before);
    if (!empty && wanted > cursor) {
        // nothing is released: give every reference back
        for_batches([&](int64_t, const int(&ids)[kPageBatch]) {
            for (int k = 0; k < kPageBatch; ++k)
                if (ids[k] >= 0)
                    atomicAdd(a.shares_out + ids[k], 1);
        });
        for (int b = gtid; b < n; b += gsize)
            a.seq_lens[b] = a.context_lens[b];
        if (gtid == 0) {
            record_error(err, kErrBudget, wanted);
            *a.cursor_out = cursor;
        }
        cluster_sync_all();  // (the sums in shared memory have been read too)
        return;
    }
    for_batches([&](int64_t x0, const int(&ids)[kPageBatch]) {
        int v[kPageBatch];
        counts_of(ids, v);
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k)
            if (v[k] < 0)
                atomicMin(a.shares_out + ids[k], -kReleaseMark - (int)(x0 + 32 * k));
    });
    cluster_sync_all();
    int freed = 0;
    for_batches([&](int64_t x0, const int(&ids)[kPageBatch]) {
        int v[kPageBatch];
        counts_of(ids, v);
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k)
            freed += __popc(__ballot_sync(0xffffffffu, v[k] == -kReleaseMark - (int)(x0 + 32 * k)));
    });
    if (lane == 0)
        s_freed[warp] = freed;
    cluster_sync_all();
    // (as many as were counted, but for counts below 0 at the call's start: a page
    // of such a count that does not fit is not kept)
    const int all = sum_freed(before);
    for_batches([&](int64_t x0, const int(&ids)[kPageBatch]) {
        int v[kPageBatch];
        counts_of(ids, v);
#pragma unroll
        for (int k = 0; k < kPageBatch; ++k) {
            // (a page's other references read its mark or 0: neither is theirs)
            const bool mine = v[k] == -kReleaseMark - (int)(x0 + 32 * k);
            const uint32_t who = __ballot_sync(0xffffffffu, mine);
            if (mine) {
                const int at = cursor - all + before + __popc(who & ((1u << lane) - 1u));
                if (at >= 0)
                    a.free_pages[at] = ids[k];
                a.shares_out[ids[k]] = 0;
            }
            before += __popc(who);
        }
    });
    for (int b = gtid; b < n; b += gsize)
        a.seq_lens[b] = empty ? a.context_lens[b] : s_keep[b];
    if (gtid == 0) {
        if (empty)
            record_error(err, kErrBadMetadata, n);
        *a.cursor_out = empty ? cursor : max(cursor - all, 0);
    }
    cluster_sync_all();  // (the counts in shared memory have been read too)
}

static size_t release_smem(int num_seqs) { return ((size_t)2 * num_seqs + 1) * 4; }

cudaError_t launch_release_pages(const PageArgs &a, ErrState *err, cudaStream_t stream, int *grid)
{
    const int64_t items = (int64_t)a.num_seqs * (a.max_blocks < 64 ? a.max_blocks : 64);
    return launch_cluster(release_pages_kernel, a, err, stream, items, release_smem(a.num_seqs), grid);
}

// With n pages in use, the k-th page in use from n on moves to the k-th unused
// page below n: the fewest moves, and sources and destinations never meet, so
// the copies need no order.  A bitmap of the pages in use is gathered in global
// memory; every CTA then takes all of it into shared memory, with a running
// count of bits, so that the rank of a page is two loads and two popcounts.
// (At most 2^20 pages: 128 KB of bitmap and 64 KB of counts.)
__global__ void __launch_bounds__(kPageThreads, 1) compact_pages_kernel(const PageArgs a, ErrState *err)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int32_t s_comp[];
    __shared__ int s_sums[kPageWarps];
    const int n = a.num_seqs, tid = threadIdx.x, blocks = (int)a.num_blocks;
    const int words = (blocks + 31) / 32, pairs = (words + 1) / 2;
    uint32_t *s_bits = reinterpret_cast<uint32_t *>(s_comp);             // [2 * pairs]
    int32_t *s_count = s_comp + 2 * pairs;                               // [pairs + 1] bits before two words
    int32_t *s_off = s_count + pairs + 1;                                // [n + 1] first page of a request
    const int gtid = blockIdx.x * kPageThreads + tid, gsize = gridDim.x * kPageThreads;
    const int64_t limit = (int64_t)a.max_blocks * 16;
    const int cursor = *a.cursor_in;
    for (int w = gtid; w < words; w += gsize)
        a.bitmap[w] = 0;
    const int total = block_exclusive_sums<kPageThreads>(n, s_off, s_sums, [&](int b) {
        const int c = a.context_lens[b];
        if (c >= 0 && (int64_t)c <= limit)
            return pages_of(c);
        if (blockIdx.x == 0)
            record_error(err, kErrBadMetadata, b);
        return 0;
    });
    cluster_sync_all();
    // (num_seqs * max_blocks is below 2^31)
    auto entry = [&](int x) {
        const int b = owner_of(s_off, n, x);
        return (int64_t)b * a.max_blocks + x - s_off[b];
    };
    for (int64_t x = gtid; x < total; x += gsize) {
        const int id = a.block_tables[entry((int)x)];
        if (id >= 0 && id < blocks)
            atomicOr(a.bitmap + (id >> 5), 1u << (id & 31));
        else
            record_error(err, kErrBadMetadata, owner_of(s_off, n, (int)x));
    }
    cluster_sync_all();
    for (int w = tid; w < 2 * pairs; w += kPageThreads)
        s_bits[w] = w < words ? __ldcg(a.bitmap + w) : 0u;
    __syncthreads();
    const int live = block_exclusive_sums<kPageThreads>(
        pairs, s_count, s_sums, [&](int i) { return __popc(s_bits[2 * i]) + __popc(s_bits[2 * i + 1]); });
    auto is_live = [&](int id) { return (s_bits[id >> 5] >> (id & 31)) & 1u; };
    // pages in use below id
    auto rank = [&](int id) {
        if (id >= blocks)
            return live;
        const int w = id >> 5;
        return s_count[w >> 1] + (w & 1 ? __popc(s_bits[w - 1]) : 0) + __popc(s_bits[w] & ((1u << (id & 31)) - 1u));
    };
    const int below = rank(live), moves = live - below;
    const bool empty = moves > a.max_moves;
    for (int64_t k = gtid; k < a.max_moves; k += gsize)
        if (empty || k >= moves)
            a.copy_src[k] = a.copy_dst[k] = -1;
    if (!empty)
        for (int id = gtid; id < blocks; id += gsize) {
            const bool used = is_live(id);
            if (id < live && !used)
                a.copy_dst[id - rank(id)] = id;
            else if (id >= live && used)
                a.copy_src[rank(id) - below] = id;
        }
    cluster_sync_all();
    for (int64_t x = gtid; x < total; x += gsize) {
        const int64_t e = entry((int)x);
        const int id = a.block_tables[e];
        const bool moved = !empty && id >= live && id < blocks;
        a.tables_out[e] = moved ? __ldcg(a.copy_dst + rank(id) - below) : id;
    }
    if (empty) {
        copy_shares(a);
    } else {
        for (int id = gtid; id < live; id += gsize) {
            const bool used = is_live(id);
            const int from = used ? id : __ldcg(a.copy_src + id - rank(id));
            if (from != id || a.shares_out != a.shares_in)
                a.shares_out[id] = a.shares_in[from];
        }
        const int64_t shift = (int64_t)a.num_free - blocks;  // >= 0
        for (int id = live + gtid; id < blocks; id += gsize)
            a.free_pages[shift + id] = id;
        cluster_sync_all();  // in place: the sources' counts have been read
        for (int id = live + gtid; id < blocks; id += gsize)
            a.shares_out[id] = 0;
    }
    if (gtid == 0) {
        a.counts[0] = live;
        a.counts[1] = moves;
        *a.cursor_out = empty ? cursor : (int)((int64_t)a.num_free - blocks) + live;
        if (empty)
            record_error(err, kErrBudget, moves);
    }
}

static size_t compact_smem(int64_t num_blocks, int num_seqs)
{
    const size_t pairs = ((size_t)num_blocks + 63) / 64;
    return (3 * pairs + 1 + num_seqs + 1) * 4;
}

cudaError_t launch_compact_pages(const PageArgs &a, ErrState *err, cudaStream_t stream, int *grid)
{
    const int64_t items = a.num_blocks + (int64_t)a.num_seqs * 64;
    return launch_cluster(compact_pages_kernel, a, err, stream, items, compact_smem(a.num_blocks, a.num_seqs), grid);
}

static_assert(kPageMaxBlocksHost / 64 * 3 * 4 + (kPageMaxSeqsHost + 2) * 4 <= 227 * 1024 - 1024, "shared memory of the compaction");
static_assert((4 * kPageMaxSeqsHost + 2) * 4 <= 227 * 1024 - 1024, "shared memory of the fork");

static cudaError_t page_attributes(void (*kern)(const PageArgs, ErrState *), size_t smem)
{
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t init_page_attributes()
{
    cudaError_t e = page_attributes(fork_requests_kernel, fork_smem(kPageMaxSeqsHost, kPageMaxSeqsHost));
    if (e == cudaSuccess)
        e = page_attributes(release_pages_kernel, release_smem(kPageMaxSeqsHost));
    if (e == cudaSuccess)
        e = page_attributes(compact_pages_kernel, compact_smem(kPageMaxBlocksHost, kPageMaxSeqsHost));
    return e;
}

}  // namespace pa

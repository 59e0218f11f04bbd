// kv_tables.cu -- block tables, slot maps and positions of one step from the
// requests' lengths.
//
// Two exclusive prefix sums over the requests (new tokens, new pages), then
// one independent entry per new page and per token.  Every CTA sums all
// requests itself -- 8 bytes a request out of L2, cheaper than a second launch
// or a grid-wide wait -- keeps the sums in shared memory and takes its share
// of the pages and tokens, finding a token's request by bisection.  Only
// entries of pages that are new are written and only older ones are read, so
// no order between CTAs is needed.  Lengths may be anything: sums stop at 2^32 - 1
// instead of wrapping (64-bit sums: 3.25 us instead of 3.1 for 8 requests).  Bound by
// latency, not by its few bytes: 8 requests of a token 3.1 us, 1000 requests with
// 261000 tokens (3.1 MB written) 7.1 us, the launch included.
#include "../../include/nvfp4_kv.h"
#include "kv.cuh"
#include "launch_cache.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 512;

// Requests before which `x` lies: the largest r in [0, n) with pre[r] <= x.
template <typename T>
__device__ __forceinline__ int bisect(const T* pre, int n, T x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The page list index of the first page a request of these lengths takes, its
// end, and its clipped length.
struct Lens {
    int32_t past, now, held, fresh;
    bool bad;
};

__device__ __forceinline__ Lens lens_of(const KvTablesArgs& a, int r)
{
    Lens l;
    const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
    const int64_t past = max(a.kv_len[r], 0), sum = past + max(a.q_len[r], 0);
    const int32_t round = (1 << a.page_shift) - 1;
    l.past = (int32_t)min(past, cap);
    l.now = (int32_t)min(sum, cap);
    l.held = (l.past + round) >> a.page_shift;
    l.fresh = ((l.now + round) >> a.page_shift) - l.held;
    l.bad = sum > cap;
    return l;
}

// Sums of tokens and of pages that stop at 2^32 - 1.
struct Sums {
    uint32_t tok, page;
};

__device__ __forceinline__ uint32_t add_to_most(uint32_t a, uint32_t b)
{
    return a + b < a ? UINT32_MAX : a + b;
}

__device__ __forceinline__ Sums operator+(Sums a, Sums b)
{
    return {add_to_most(a.tok, b.tok), add_to_most(a.page, b.page)};
}

__device__ __forceinline__ int32_t as_int32(uint32_t x)
{
    return (int32_t)min(x, (uint32_t)INT32_MAX);
}

__global__ void __launch_bounds__(kThreads) kv_tables_kernel(const KvTablesArgs a)
{
    extern __shared__ uint32_t sums[];
    uint32_t* tok0 = sums;                // [reqs + 1] first token of a request
    uint32_t* page0 = sums + a.reqs + 1;  // [reqs + 1] its first new page
    __shared__ Sums warp_sum[kThreads / 32];
    kv_pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = false;

    // a run of requests a thread
    const int per = (a.reqs + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, a.reqs), r1 = min(r0 + per, a.reqs);
    Sums inc = {0u, 0u};
    for (int r = r0; r < r1; ++r) {
        const Lens l = lens_of(a, r);
        inc = inc + Sums{(uint32_t)max(a.q_len[r], 0), (uint32_t)l.fresh};
        bad |= l.bad;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = {__shfl_up_sync(0xFFFFFFFFu, inc.tok, d), __shfl_up_sync(0xFFFFFFFFu, inc.page, d)};
        if (lane >= d)
            inc = inc + o;
    }
    if (lane == 31)
        warp_sum[warp] = inc;
    // what lies before the thread's run
    Sums at = {__shfl_up_sync(0xFFFFFFFFu, inc.tok, 1), __shfl_up_sync(0xFFFFFFFFu, inc.page, 1)};
    if (lane == 0)
        at = {0u, 0u};
    __syncthreads();
    Sums all = {0u, 0u};
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp)
            at = at + all;
        all = all + warp_sum[w];
    }
    for (int r = r0; r < r1; ++r) {
        const Lens l = lens_of(a, r);
        tok0[r] = at.tok;
        page0[r] = at.page;
        if (blockIdx.x == 0) {
            a.seq_len[r] = l.now;
            a.q_start[r] = as_int32(at.tok);
        }
        at = at + Sums{(uint32_t)max(a.q_len[r], 0), (uint32_t)l.fresh};
    }
    const int32_t head = a.free_head[0];
    if (tid == 0) {
        tok0[a.reqs] = all.tok;
        page0[a.reqs] = all.page;
        if (blockIdx.x == 0) {
            a.q_start[a.reqs] = as_int32(all.tok);
            a.free_next[0] = (int32_t)min((int64_t)head + all.page, (int64_t)INT32_MAX);
            bad |= all.tok > (uint32_t)a.tokens;
        }
    }
    __syncthreads();

    const int64_t gid = (int64_t)blockIdx.x * kThreads + tid, step = (int64_t)gridDim.x * kThreads;
    for (int64_t f = gid; f < all.page; f += step) {
        const int r = bisect(page0, a.reqs, (uint32_t)f);
        const Lens l = lens_of(a, r);
        const int64_t at_free = head + f;
        const bool got = at_free >= 0 && at_free < a.num_free;
        bad |= !got;
        a.table[r * a.table_stride + l.held + ((uint32_t)f - page0[r])] =
            got ? a.free_pages[at_free] : -1;
    }
    // pages that are not counted any more lie past every free list (num_free < 2^31)
    if (all.page == UINT32_MAX)
        for (int64_t r = gid; r < a.reqs; r += step) {
            const Lens l = lens_of(a, (int)r);
            for (int32_t j = l.fresh - 1; j >= 0 && add_to_most(page0[r], j) == UINT32_MAX; --j)
                a.table[r * a.table_stride + l.held + j] = -1;
        }
    const uint32_t rows = min(all.tok, (uint32_t)a.tokens);
    for (int32_t t = (int32_t)gid; t < a.tokens; t += (int32_t)step) {
        int64_t slot = -1;
        uint32_t pos = 0;
        if ((uint32_t)t < rows) {
            const int r = bisect(tok0, a.reqs, (uint32_t)t);
            const Lens l = lens_of(a, r);
            const int32_t i = (int32_t)(t - tok0[r]);
            pos = (uint32_t)max(a.kv_len[r], 0) + (uint32_t)i;
            if (i < l.now - l.past) {  // else past the table's end (and pos past int32, perhaps)
                const int32_t b = (int32_t)pos >> a.page_shift;
                int32_t page = -1;
                if (b < l.held) {
                    page = a.table[r * a.table_stride + b];
                } else {
                    const int64_t at_free = (int64_t)head + page0[r] + (b - l.held);
                    if (at_free >= 0 && at_free < a.num_free)
                        page = a.free_pages[at_free];
                }
                if (page >= 0)
                    slot = ((int64_t)page << a.page_shift) | (pos & ((1 << a.page_shift) - 1));
                else
                    bad = true;
            }
        }
        a.slots[t] = slot;
        a.positions[t] = as_int32(pos);
    }
    if (bad)
        atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesArgs& a, cudaStream_t stream, bool pdl)
{
    const int dev = current_device();
    const size_t smem = (size_t)(a.reqs + 1) * 2 * sizeof(uint32_t);
    const cudaError_t e = ensure_smem_limit(kv_tables_kernel, smem, dev);
    if (e != cudaSuccess)
        return e;
    // one token or request a thread, at most one CTA an SM (each sums all requests)
    int64_t grid = ((int64_t)a.tokens + a.reqs + kThreads - 1) / kThreads;
    const int64_t sms = device_sm_count(dev);
    grid = grid < 1 ? 1 : grid > sms ? sms : grid;
    return kv_launch(kv_tables_kernel, (unsigned)grid, kThreads, smem, stream, pdl, a);
}

}  // namespace nvfp4

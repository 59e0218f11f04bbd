// kv_tables.cu -- block tables, slot maps and positions of one step from the
// requests' lengths.
//
// Two exclusive prefix sums over the requests (new tokens, new pages), then
// one independent entry per new page and per token.  Every CTA sums all
// requests itself -- 8 bytes a request out of L2, cheaper than a second launch
// or a grid-wide wait -- keeps the sums in shared memory and takes its share
// of the pages and tokens, finding a token's request by bisection.  Only
// entries of pages that are new are written and only older ones are read, so
// no order between CTAs is needed.  Bound by latency, not by its few bytes: 8
// requests of a token 3.0 us, 1000 requests with 261000 tokens (3.1 MB written)
// 6.9 us, the launch included.
#include "../../include/nvfp4_kv.h"
#include "kv.cuh"
#include "launch_cache.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 512;

// Requests before which `x` lies: the largest r in [0, n) with pre[r] <= x.
__device__ __forceinline__ int bisect(const int32_t* pre, int n, int32_t x)
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

__global__ void __launch_bounds__(kThreads) kv_tables_kernel(const KvTablesArgs a)
{
    extern __shared__ int32_t sums[];
    int32_t* tok0 = sums;               // [reqs + 1] first token of a request
    int32_t* page0 = sums + a.reqs + 1;  // [reqs + 1] its first new page
    __shared__ unsigned long long warp_sum[kThreads / 32];
    kv_pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = false;

    // a run of requests a thread; both sums in one word (each below 2^31)
    const int per = (a.reqs + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, a.reqs), r1 = min(r0 + per, a.reqs);
    unsigned long long mine = 0;
    for (int r = r0; r < r1; ++r) {
        const Lens l = lens_of(a, r);
        mine += ((unsigned long long)(uint32_t)max(a.q_len[r], 0) << 32) | (uint32_t)l.fresh;
        bad |= l.bad;
    }
    unsigned long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d)
            inc += o;
    }
    if (lane == 31)
        warp_sum[warp] = inc;
    __syncthreads();
    unsigned long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp)
            before += warp_sum[w];
        all += warp_sum[w];
    }
    unsigned long long at = before + inc - mine;
    for (int r = r0; r < r1; ++r) {
        const Lens l = lens_of(a, r);
        tok0[r] = (int32_t)(at >> 32);
        page0[r] = (int32_t)(uint32_t)at;
        if (blockIdx.x == 0) {
            a.seq_len[r] = l.now;
            a.q_start[r] = (int32_t)(at >> 32);
        }
        at += ((unsigned long long)(uint32_t)max(a.q_len[r], 0) << 32) | (uint32_t)l.fresh;
    }
    const int32_t total = (int32_t)(all >> 32), pages = (int32_t)(uint32_t)all;
    const int32_t head = a.free_head[0];
    if (tid == 0) {
        tok0[a.reqs] = total;
        page0[a.reqs] = pages;
        if (blockIdx.x == 0) {
            a.q_start[a.reqs] = total;
            a.free_next[0] = head + pages;
            bad |= total > a.tokens;
        }
    }
    __syncthreads();

    const int64_t gid = (int64_t)blockIdx.x * kThreads + tid, step = (int64_t)gridDim.x * kThreads;
    for (int64_t f = gid; f < pages; f += step) {
        const int r = bisect(page0, a.reqs, (int32_t)f);
        const Lens l = lens_of(a, r);
        const int64_t at_free = (int64_t)head + f;
        const bool got = at_free >= 0 && at_free < a.num_free;
        bad |= !got;
        a.table[r * a.table_stride + l.held + ((int32_t)f - page0[r])] =
            got ? a.free_pages[at_free] : -1;
    }
    for (int64_t t = gid; t < a.tokens; t += step) {
        int64_t slot = -1;
        int32_t pos = 0;
        if (t < total) {
            const int r = bisect(tok0, a.reqs, (int32_t)t);
            const Lens l = lens_of(a, r);
            pos = max(a.kv_len[r], 0) + ((int32_t)t - tok0[r]);
            if (pos < l.now) {
                const int32_t b = pos >> a.page_shift;
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
        a.positions[t] = pos;
    }
    if (bad)
        atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesArgs& a, cudaStream_t stream, bool pdl)
{
    const int dev = current_device();
    const size_t smem = (size_t)(a.reqs + 1) * 2 * sizeof(int32_t);
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

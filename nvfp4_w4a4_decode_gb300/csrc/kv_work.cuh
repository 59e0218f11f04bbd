// kv_work.cuh -- what the attention kernels over the paged cache share: bounded
// mbarrier waits, and the list of work that is cut into equal shares on the
// device (lengths are device data, and a captured graph replays with others).
#pragma once

#include "../../include/nvfp4_kv.h"
#include "kv.cuh"

namespace nvfp4 {

constexpr long long kKvWaitBudget = 2000000000LL;  // clock cycles a wait may take

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
// Wait for phase `parity`; false when the budget (or another wait's) ran out.
// Clock and flag are looked at once in kKvPolls tests only: at every test they
// took a quarter of the issue slots of a kernel whose warps wait in turn.
constexpr int kKvPolls = 64;
static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity,
                                                   volatile int* abort_flag, unsigned* status)
{
    const long long t0 = clock64();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < kKvPolls; ++i)
            if (mbar_test(bar, parity))
                return true;
        if (*abort_flag)
            return false;
        if (clock64() - t0 > kKvWaitBudget) {
            *abort_flag = 1;
            atomicOr(status, (unsigned)NVFP4_DEVICE_WAIT_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned* status)
{
    return mbar_test(bar, parity) || mbar_wait_slow(bar, parity, abort_flag, status);
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// ---- the work list ---------------------------------------------------------------
// An item is (request, kv head, tile of R query rows), rows being token * group
// + head of the group.  Its units are the blocks of UT tokens that any of its
// rows sees (one when it sees none, so that its rows are written).  Items are
// ordered request, head, tile; each takes COST places, which stand for its
// start and its join, and one a unit.  The list is cut into equal shares, one a
// CTA; an item whose units lie in several shares is cut between them.

struct KvReq {
    int32_t seq;   // tokens in the cache
    int32_t base;  // first query row
    int32_t nq;    // query rows (tokens)
};

__device__ __forceinline__ KvReq kv_req(const KvAttnArgs& a, int r)
{
    KvReq q;
    int32_t b, e;
    if (a.q_start) {
        b = a.q_start[r];
        e = a.q_start[r + 1];
    } else {
        b = r * a.q_per_req;
        e = b + a.q_per_req;
    }
    b = min(max(b, 0), a.tokens);
    e = min(max(e, b), a.tokens);
    q.base = b;
    q.nq = e - b;
    const int64_t cap = (int64_t)a.max_blocks << a.c.page_shift;
    q.seq = (int32_t)min((int64_t)max(a.seq_len[r], 0), cap);
    return q;
}

// Zeros (and lse = -inf) for the call's rows [0, begin) and [end, tokens), by `threads`
// threads of every CTA.  A function of its own, its arguments by value: the common call
// has no such rows, and in line it cost the tcgen05 kernel 2 % of a chunk.
static __device__ __noinline__ void kv_fill_rows(const KvAttnArgs a, int32_t begin, int32_t end,
                                                 int thread, int threads)
{
    const int64_t rows = begin + a.tokens - end;
    const int heads = a.c.heads * a.group;
    const int64_t at = (int64_t)blockIdx.x * threads + thread, step = (int64_t)gridDim.x * threads;
    // four elements at a time (rows are aligned to that)
    const int parts = heads * a.c.dim / 4, part = a.out_bf16 ? 8 : 16;
    for (int64_t i = at; i < rows * parts; i += step) {
        const int64_t j = i / parts, t = j < begin ? j : j - begin + end;
        uint8_t* p = static_cast<uint8_t*>(a.out) + t * a.out_stride * (part / 4) + (i - j * parts) * part;
        if (a.out_bf16)
            *reinterpret_cast<uint2*>(p) = make_uint2(0u, 0u);
        else
            *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (a.lse)
        for (int64_t i = at; i < rows * heads; i += step) {
            const int64_t j = i / heads, t = j < begin ? j : j - begin + end;
            a.lse[t * heads + (i - j * heads)] = -INFINITY;
        }
}

// The rows that lie before the first or behind the last request.
__device__ __forceinline__ void kv_write_other_rows(const KvAttnArgs& a, int thread, int threads)
{
    int32_t begin = 0, end = a.reqs ? a.tokens : 0;
    if (a.q_start) {
        begin = min(max(a.q_start[0], 0), a.tokens);
        end = min(max(a.q_start[a.reqs], begin), a.tokens);
    }
    if (begin > 0 || end < a.tokens)
        kv_fill_rows(a, begin, end, thread, threads);
}

// Whether a request is longer than its table (its end is then cut off).
__device__ __forceinline__ bool kv_too_long(const KvAttnArgs& a, int r)
{
    return (int64_t)a.seq_len[r] > (int64_t)a.max_blocks << a.c.page_shift;
}

// The token of a query row: row / group, by a multiplication (the group is a
// launch's constant; a division took a tenth of an item's start).
__device__ __forceinline__ int kv_token(const KvAttnArgs& a, int row)
{
    if (a.group == 1)
        return row;
    const uint32_t q = __umulhi((uint32_t)row, a.group_magic);  // one too large at most
    return (int)(q - (q * (uint32_t)a.group > (uint32_t)row ? 1u : 0u));
}

// a / b of places; 32 bits where they do (a 64-bit division takes half as long as
// a token's request takes to load).
__device__ __forceinline__ int64_t kv_divide(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return (uint32_t)a / (uint32_t)b;
    return a / b;
}

struct KvItem {
    int r, h, tile;
    KvReq q;
    int rows;       // query rows of the request (tokens * group)
    int row0, row1;
    int64_t begin;  // its place in the list: COST, then its units
    int32_t first, n;
    int32_t u0, u1;  // the units of this CTA's share
};

// A CTA's share of the list.  Items of up to `least` units are not cut between
// shares: joining their parts would take longer than the units do.
struct KvShare {
    int64_t lo, hi, size;
    int32_t least;
    bool cut;  // longer items may be
};

// Items of up to WHOLE units, or an eighth of a share, stay whole.
template <int R, int UT, int COST, int WHOLE>
struct KvWork {
    // Units [first, first + n) of the rows [row0, row1) of a request.
    static __device__ __forceinline__ void tile_units(const KvAttnArgs& a, const KvReq& q, int row0,
                                                      int row1, int32_t& first, int32_t& n)
    {
        const int32_t i0 = kv_token(a, row0), i1 = kv_token(a, row1 - 1);
        const int32_t p0 = q.seq - q.nq;
        const int32_t hi = p0 + i1 + 1;  // keys [lo, hi)
        const int32_t lo = a.window > 0 ? max(0, p0 + i0 - a.window + 1) : 0;
        if (hi <= lo) {
            first = 0;
            n = 1;
            return;
        }
        first = lo / UT;
        n = (hi + UT - 1) / UT - first;
    }

    // The first key that any row of an item sees.  What lies before it in the item's
    // first unit is not looked at: its page may serve another request by now.
    static __device__ __forceinline__ int32_t first_key(const KvAttnArgs& a, const KvItem& it)
    {
        return a.window > 0 ? max(0, it.q.seq - it.q.nq + kv_token(a, it.row0) - a.window + 1) : 0;
    }

    static __device__ __forceinline__ void units(const KvAttnArgs& a, KvItem& it)
    {
        it.row0 = it.tile * R;
        it.row1 = min(it.row0 + R, it.rows);
        tile_units(a, it.q, it.row0, it.row1, it.first, it.n);
    }

    // The first item of the first request at or after r that has rows.
    static __device__ __forceinline__ bool request(const KvAttnArgs& a, KvItem& it, int r)
    {
        for (; r < a.reqs; ++r) {
            it.q = kv_req(a, r);
            if (it.q.nq > 0)
                break;
        }
        it.r = r;
        it.h = it.tile = 0;
        if (r >= a.reqs)
            return false;
        it.rows = it.q.nq * a.group;
        units(a, it);
        return true;
    }

    static __device__ __forceinline__ bool after(const KvAttnArgs& a, KvItem& it)
    {
        it.begin += COST + it.n;
        if ((it.tile + 1) * R < it.rows) {
            ++it.tile;
            units(a, it);
            return true;
        }
        it.tile = 0;
        if (++it.h < a.c.heads) {
            units(a, it);
            return true;
        }
        return request(a, it, it.r + 1);
    }

    // Steps on, from an item that may have no unit in the share, to one that has.
    static __device__ __forceinline__ bool settle(const KvAttnArgs& a, const KvShare& s, KvItem& it,
                                                  bool more)
    {
        for (; more; more = after(a, it)) {
            const int64_t at = it.begin + COST;  // place of unit 0
            if (at >= s.hi)
                return false;
            if (s.cut && it.n > s.least) {
                it.u0 = (int32_t)max((int64_t)0, s.lo - at);
                it.u1 = (int32_t)min((int64_t)it.n, s.hi - at);
                if (it.u0 < it.u1)
                    return true;
            } else {  // a whole item belongs to the share that holds its unit 0
                it.u0 = 0;
                it.u1 = it.n;
                if (at >= s.lo)
                    return true;
            }
        }
        return false;
    }

    static __device__ __forceinline__ bool next(const KvAttnArgs& a, const KvShare& s, KvItem& it)
    {
        return settle(a, s, it, after(a, it));
    }

    // The CTAs that hold the first and the last unit of an item.
    static __device__ __forceinline__ int first_cta(const KvShare& s, const KvItem& it)
    {
        return (int)kv_divide(it.begin + COST, s.size);
    }
    static __device__ __forceinline__ int last_cta(const KvShare& s, const KvItem& it)
    {
        return (int)kv_divide(it.begin + COST + it.n - 1, s.size);
    }

    // Places of one kv head of a request, summed by one thread or by a warp.
    static __device__ __forceinline__ int64_t head_places(const KvAttnArgs& a, const KvReq& q,
                                                          int start, int step)
    {
        int64_t s = 0;
        const int rows = q.nq * a.group;
        for (int64_t row0 = (int64_t)start * R; row0 < rows; row0 += (int64_t)step * R) {
            int32_t first, n;
            tile_units(a, q, (int)row0, (int)min(row0 + R, (int64_t)rows), first, n);
            s += COST + n;
        }
        return s;
    }
    static __device__ __forceinline__ int64_t head_places_warp(const KvAttnArgs& a, const KvReq& q)
    {
        int64_t s = head_places(a, q, threadIdx.x & 31, 32);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        return s;
    }

    struct Smem {
        int64_t warp_sum[32];
        int64_t req_sum[256];
        int64_t rem;
        int r;
    };

    // The share of this CTA, of a list of `total` places; false when it is empty.
    static __device__ __forceinline__ bool cut_share(const KvAttnArgs& a, int64_t total, int64_t least,
                                                     KvShare& sh)
    {
        sh.size = max(kv_divide(total + gridDim.x - 1, gridDim.x), least);
        sh.lo = sh.size * blockIdx.x;
        sh.hi = min(sh.lo + sh.size, total);
        sh.cut = a.part != nullptr;
        sh.least = (int32_t)min(max((int64_t)WHOLE, sh.size >> 3), (int64_t)INT32_MAX);
        return sh.lo < total;
    }

    // The item at place sh.lo, `rem` places into request `it.r` (it.q, it.rows and
    // the request's places of a head are known); then the first with a unit.
    static __device__ __forceinline__ bool locate(const KvAttnArgs& a, const KvShare& sh, KvItem& it,
                                                  int64_t rem, int64_t head)
    {
        it.begin = sh.lo - rem;
        it.h = (int)kv_divide(rem, head);
        it.begin += it.h * head;
        it.tile = 0;
        const int tiles = (it.rows + R - 1) / R, lane = threadIdx.x & 31;
        for (int t0 = 0; tiles > 1 && t0 < tiles; t0 += 32) {  // 32 tiles at a time
            int32_t first, n = 0;
            const int t = t0 + lane;
            if (t < tiles) {
                tile_units(a, it.q, t * R, min(t * R + R, it.rows), first, n);
                n += COST;
            }
            int32_t sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d)
                    sum += o;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, it.begin + sum <= sh.lo);
            const int skip = __popc(past);  // whole tiles before sh.lo
            if (skip < 32) {
                it.tile = t0 + skip;
                it.begin += skip ? __shfl_sync(0xFFFFFFFFu, sum, skip - 1) : 0;
                break;
            }
            it.begin += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        units(a, it);
        return settle(a, sh, it, true);
    }

    // Up to 32 requests of few tiles: every warp finds the share by itself, a lane a
    // request, without a barrier (the CTA-wide form took 3 of a single request's 12 us).
    static __device__ __forceinline__ bool start_warp(const KvAttnArgs& a, int64_t least, KvShare& sh,
                                                      KvItem& it)
    {
        const int lane = threadIdx.x & 31;
        KvReq q = {0, 0, 0};
        int64_t head = 0;
        if (lane < a.reqs) {
            q = kv_req(a, lane);
            head = head_places(a, q, 0, 1);
            if (blockIdx.x == 0 && kv_too_long(a, lane))
                atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
        }
        const int64_t mine = a.c.heads * head;
        int64_t inc = mine;
        for (int d = 1; d < a.reqs; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d)
                inc += o;
        }
        if (!cut_share(a, __shfl_sync(0xFFFFFFFFu, inc, a.reqs - 1), least, sh))
            return false;
        // the first request that ends behind sh.lo
        const uint32_t behind = __ballot_sync(0xFFFFFFFFu, lane < a.reqs && inc > sh.lo);
        it.r = __ffs(behind) - 1;
        const int64_t rem = sh.lo - __shfl_sync(0xFFFFFFFFu, inc - mine, it.r);
        head = __shfl_sync(0xFFFFFFFFu, head, it.r);
        it.q.seq = __shfl_sync(0xFFFFFFFFu, q.seq, it.r);
        it.q.base = __shfl_sync(0xFFFFFFFFu, q.base, it.r);
        it.q.nq = __shfl_sync(0xFFFFFFFFu, q.nq, it.r);
        it.rows = it.q.nq * a.group;
        return locate(a, sh, it, rem, head);
    }

    // The whole CTA (THREADS threads) computes its share of the list and the
    // first item with a unit in it; false when there is none.
    template <int THREADS>
    static __device__ bool start(const KvAttnArgs& a, Smem& sm, int64_t least, KvShare& sh,
                                 KvItem& it)
    {
        if (a.reqs <= 32 && (int64_t)a.tokens * a.group <= 4 * R * (int64_t)a.reqs) {
            const bool more = start_warp(a, least, sh, it);
            __syncthreads();  // what the caller initialised
            return more;
        }
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        // few requests of many tiles: a warp sums a request; else a thread a run of them
        const bool by_warp = a.reqs <= 256 && (int64_t)a.tokens * a.group > 2 * (int64_t)R * a.reqs;
        int per = (a.reqs + THREADS - 1) / THREADS;
        if (by_warp) {
            for (int r = warp; r < a.reqs; r += THREADS / 32) {
                const int64_t s = head_places_warp(a, kv_req(a, r));
                if (lane == 0)
                    sm.req_sum[r] = a.c.heads * s;
            }
            per = (a.reqs + THREADS - 1) / THREADS;
            __syncthreads();
        }
        auto places = [&](int r) {
            return by_warp ? sm.req_sum[r] : a.c.heads * head_places(a, kv_req(a, r), 0, 1);
        };
        const int ra = min(tid * per, a.reqs), rb = min(ra + per, a.reqs);
        int64_t mine = 0;
        for (int r = ra; r < rb; ++r) {
            mine += places(r);
            if (blockIdx.x == 0 && kv_too_long(a, r))
                atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
        }
        int64_t inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d)
                inc += o;
        }
        if (lane == 31)
            sm.warp_sum[warp] = inc;
        __syncthreads();
        int64_t before = inc - mine, total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp)
                before += sm.warp_sum[w];
            total += sm.warp_sum[w];
        }
        if (!cut_share(a, total, least, sh))
            return false;
        if (sh.lo >= before && sh.lo < before + mine) {
            int64_t at = before;
            for (int r = ra; r < rb; ++r) {
                const int64_t n = places(r);
                if (sh.lo < at + n) {
                    sm.r = r;
                    sm.rem = sh.lo - at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        if (!request(a, it, sm.r))
            return false;
        return locate(a, sh, it, sm.rem, places_of_head(a, it.q));
    }

private:
    static __device__ __forceinline__ int64_t places_of_head(const KvAttnArgs& a, const KvReq& q)
    {
        return (int64_t)q.nq * a.group <= 4 * R ? head_places(a, q, 0, 1) : head_places_warp(a, q);
    }
};

}  // namespace nvfp4

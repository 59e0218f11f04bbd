// kv_attention_rows.cuh -- attention over the paged NVFP4 cache with few query
// rows a request: single tokens, drafted tokens, short prompts.  Which keys a row sees is a
// template's matter (KvSees): causal attention, all keys (cross attention; a prefix that a group of
// requests shares, whose rows are then one request's), the keys behind such a prefix.
//
// Mathematics.  With K = k_g sK cK (codes cK, block scales sK), a score is
// scale k_g sum_d q_d (sK cK)_d.  sK cK has at most 6 significant bits and
// magnitudes 2^-10 .. 2688, so it is an f16 value exactly; a BF16 query row
// multiplied by a power of two that brings its largest element to [2^14, 2^15)
// is exact in f16 but for elements 2^30 times smaller, an FP32 one is the sum
// of two f16 (22 bits).  So f16 MMAs with FP32 accumulation give FP32 scores.
// The softmax runs online: p = 2^(s - m + 7) with a per-row reference m that
// is raised only when a score passes it by more than 2^8 (any reference gives
// the same quotient; p stays below 2^15 and f16 resolves 2^-31 of the largest),
// row sums in FP32 from the unrounded p.  p goes into the second MMA as one
// f16 (outputs in BF16) or two (FP32), against exact values.  The tensor cores'
// own accumulation truncates, which a chain of thousands of tokens would carry
// into the sixth digit: with FP32 terms 16 tokens' products are summed alone and
// added in FP32, and the queries' second terms have an accumulator of their own
// (largest error of 24 requests of 1..6000 tokens: 4e-7 of the largest output,
// from 0.8..2.1e-6, in the same time).
//
// Layout.  The query rows (token, head of the group) are the narrow side of
// m16n8k16 tiles, 8 NT of them: S^T = K Q^T and O^T = V^T P^T, so a single
// token of a group of 4 to 8 heads fills the tile and the 4-bit cache is
// decoded once for all of them.  A warp takes 16 tokens a tile, two tiles at a time: lane
// (g, t) = (lane / 4, lane % 4) reads K of token rows g, g + 8 -- its quarter
// of the head dim, one vector -- and V of four tokens -- its eighth -- so that
// every load is one contiguous vector and a lane meets one or two block scales
// a token.  V's codes of two tokens are interleaved as nibbles before they are
// converted, which gives the f16 pairs along the tokens that the MMA wants.
//
// Work.  One list of 64-token groups for all requests (kv_work.cuh), equal shares a
// CTA; the 32-token units of an item's groups are dealt to the CTA's seven
// compute warps (three behind a prefix) in turn.  One more warp runs ahead through the list, across
// items: it looks up the pages and fills a ring of groups with bulk copies --
// a page of up to 64 tokens holds all four pieces of a kv head in one run of
// bytes, so a group is one to four copies.  Compute warps join through shared
// memory at an item's end; items cut between CTAs are joined by the last of
// them to arrive, in CTA order, or where two passes share a row's keys are left to
// kv_join.cu as they are.  Each item counts kItemCost groups more than it
// has: its start and join cost about that, so that shares of many short
// requests take equal time.  Every wait has a clock budget: one that runs out
// sets NVFP4_DEVICE_WAIT_TIMEOUT and all waits after it are passed over.
//
// What bounds it: for many tokens the latency of its chains, with four warps a scheduler.
// 16 tokens of a kv head of 128 take about 310 warp instructions, most of them conversions
// of codes and scales at half rate, each waiting for the last; issue is active 49 % of
// the time, ALU 44 %, DRAM 56 %, and the registers allow no more warps (64 requests of
// 6000..8191 tokens, 8 kv heads, a token each: 110 us, 4.6 TB/s of codes and scales; two of
// 100000..131071: 59.5 us, 4.3 TB/s).  For few tokens the chain list - queries - units -
// join, about 9.5 us (one request of 1000); a launch's fixed parts measured in cycles: list 2300, queries
// 1700, first units 2800, warps' join 1400, part and counter 2000, CTAs' join 5000.  Where every SM has one or
// two short items each of these runs once, and a third to a half of a warp's time goes into fetching its
// instructions (20 requests of 300..1500 states, 16 heads of 64: 15.0 us, no instruction 4.4 of 9.7 stalls
// an issue; 16 tokens at a time instead of two times 16, half the code, gained nothing).
#pragma once

#include "formats.cuh"
#include "kv_work.cuh"
#include "launch_cache.cuh"
#include "mma_frag.cuh"

namespace nvfp4 {

namespace {

constexpr int kUnit = 32;       // tokens a unit
constexpr int kGroup = 64;      // tokens a group
constexpr int kSub = kGroup / kUnit;
constexpr int kBatch = 3;       // groups the copying warp brings at a time
constexpr int kMaxCtas = 512;   // workspace extent
constexpr int kMaxRows = 32;
constexpr float kRaise = 8.0f;  // log2 a score may pass the reference by
constexpr float kLift = 7.0f;   // p = 2^(s - m + kLift)

// Barrier of the compute warps.
template <int THREADS>
__device__ __forceinline__ void compute_barrier()
{
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

__device__ __forceinline__ uint32_t movm_trans(uint32_t v)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// What an f16 pair leaves of the two floats it came from, as another pair.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_f16(lo - f.x, hi - f.y);
}

// MMA row k of 16 tokens holds this token: rows 2j are tokens 0..3, rows 2j + 1
// tokens 4..7 (paired j with j ^ 1), and the same eight further on; so the
// four lanes of a V load and the two rows of a K load phase fall on different
// banks as far as 64-byte rows allow.
__device__ __forceinline__ int token_of_row(int k)
{
    const int j = (k & 7) >> 1;
    return (k & 8) | ((k & 1) ? 4 + (j ^ 1) : j);
}

// W compute warps a CTA.  Seven: with the copying warp eight, two for each of the SM's four
// register files.  Three, with four CTAs an SM, for the few keys that requests mostly have behind a
// shared prefix: an item's start and end, which wait for memory and for instructions, overlap
// those of three other CTAs (seven / three warps, us: four requests of 300 tokens behind 2000 19.7 / 15.9, 64
// of 30..900 41.0 / 38.3, but 64 of 3000 83.8 / 87.3, eight of 20000 66.8 / 72.6).  All keys are left to seven,
// as their number is not known on the host (64 of 100 12.0 / 8.8, but 20 of 300..1500 15.0 / 16.0, eight of
// 1500 12.1 / 13.4, 64 of 6000..8191 108.5 / 124.3).
template <int D, int NT, bool SPLIT, int W>
struct Cfg {
    static constexpr int kCompute = 32 * W;
    static constexpr int kThreads = kCompute + 32;
    static constexpr int R = 8 * NT;             // query rows a tile
    static constexpr int KS = D / 16;            // k16 steps of Q K, m16 tiles of V
    static constexpr int kStageBytes = kGroup * D * 9 / 8;
    // two CTAs an SM where the registers allow it: the joins and starts of one
    // overlap the other's stream (with FP32 terms that takes the queries out of
    // registers and one half at a time: 24 ragged requests 25.9 -> 20.9 us)
    static constexpr int kCtas = W == 3 ? 4 : NT == 1 ? 2 : 1;
    static constexpr int kStages = W == 3 ? (D == 128 ? 3 : 6) : 7;
    static constexpr int kQTerms = SPLIT ? 2 : 1;
    static constexpr int kQBytes = kQTerms * NT * KS * 32 * 8;
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kRedBytes = W * KS * 32 * 16;
    static constexpr int kSmem = kRingBytes + kRedBytes + kQBytes;
    // queries held in registers while the accumulators leave room (32 rows, or FP32
    // terms, read them from shared memory at each use)
    static constexpr bool kQRegs = NT <= 2 && !SPLIT;
    // A parity tells a phase from its neighbours only: a warp must see every
    // phase of the slots it reads.  Units are dealt by their number in the CTA's
    // whole sequence, so a unit's place in the ring always has the same warp.
    static_assert(kStages * kSub % W == 0, "a ring holds whole rounds of the warps");
};

// How the list is cut.  Groups that an item's start and join cost: seven warps, us for 24 requests
// of 1..6000 tokens, FP32 queries / three FP32 prompts: 1 25 / 72, 2 21 / 59, 5 20 / 45, 8 18.8 / 42,
// 12 20 / 44; three warps, whose parts are left to kv_join.cu, 64 requests of 30..900 tokens behind a
// prefix: 2 43.8, 4 41.4, 6 43.9.  Items of up to kWhole groups, or of two shares and up to kWholeMax,
// stay whole (the same requests: 2 41.2, 8 41.4, 16 45.1).
template <int W>
struct Cut {
    static constexpr int kItemCost = W == 3 ? 4 : 8;
    static constexpr int kWhole = W == 3 ? 2 : 4;
    static constexpr int kWholeMax = W == 3 ? 8 : 4;
};

template <KvSees S, int D, int NT, bool SPLIT, int W>
__global__ void __launch_bounds__(Cfg<D, NT, SPLIT, W>::kThreads, Cfg<D, NT, SPLIT, W>::kCtas)
    kv_rows_kernel(const KvAttnArgs a)
{
    using C = Cfg<D, NT, SPLIT, W>;
    constexpr int kWarps = W, kCompute = C::kCompute, kThreads = C::kThreads;
    auto compute_sync = []() { compute_barrier<C::kCompute>(); };
    constexpr int R = C::R, KS = C::KS, ST = C::kStages;
    using Work = KvWork<R, kGroup, Cut<W>::kItemCost, Cut<W>::kWhole, Cut<W>::kWholeMax, S>;
    using Item = KvItem;
    using Share = KvShare;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[ST], empty_bar[ST];
    __shared__ typename Work::Smem work_sm;
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R], sm_f[R], sm_sum[R];
    __shared__ int32_t sm_pos[R];
    __shared__ int last_s, abort_s;
    float4* red = reinterpret_cast<float4*>(smem + C::kRingBytes);
    uint2* sq = reinterpret_cast<uint2*>(smem + C::kRingBytes + C::kRedBytes);
    volatile int* abort_flag = &abort_s;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&full_bar[i]), 1);
            mbar_init(smem_u32(&empty_bar[i]), kSub);
        }
        abort_s = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    kv_pdl_begin<S>(a.keep);

    // at least as many groups as the warps take in one round
    Share sh;
    Item it;
    bool more = Work::template start<kThreads>(a, work_sm, (kWarps + (W == 3)) / kSub, sh, it);
    if (sh.lo >= sh.hi) {
        if (a.all_rows && warp == kWarps)
            kv_write_other_rows(a, lane, 32);
        kv_pdl_end<S>();
        return;
    }

    const int64_t head_bytes = kv_head_bytes(a.c.page_shift, D);
    const uint32_t ring = smem_u32(smem);

    if (warp == kWarps) {
        // ---- the copying warp: kBatch groups at a time, four lanes a group ----------------
        // pages of up to 64 tokens: a piece is a page; longer ones: K codes, V
        // codes, K scales, V scales of the group's part of the page.  (One group
        // at a time took this warp about 800 cycles each, the SM's whole time
        // for two groups.)
        const int P = a.c.page_shift, sub = lane >> 2, piece = lane & 3;
        const bool by_page = P <= 6;
        const int pieces = by_page ? kGroup >> P : 4;
        const bool mine_to_copy = sub < kBatch && piece < pieces;
        const int row_bytes = by_page ? D * 9 / 8 : piece < 2 ? D / 2 : D / 16;
        const uint32_t bytes = by_page ? (uint32_t)row_bytes << P : (uint32_t)row_bytes * kGroup;
        const int before_me = piece < 2 ? piece * (D / 2) : D + (piece - 2) * (D / 16);
        const uint32_t in_slot = by_page ? piece * bytes : before_me * kGroup;
        const uint8_t* src0 = a.c.pool + (by_page ? 0 : (int64_t)before_me << P);
        bool bad = false;
        uint32_t sent = 0;  // groups so far
        // the page of this lane's piece of groups u .. of an item (any below 0: none in the
        // pool; kNothing, which no entry becomes: nothing of the request there)
        constexpr int32_t kNothing = -2;
        auto page_of = [&](const Item& x, int32_t u) {
            const int32_t tok = (x.first + u + sub) * kGroup + (by_page ? piece << P : 0);
            const int32_t b = tok >> P;
            return mine_to_copy && u + sub < x.u1 && tok < x.q.seq && b < a.max_blocks &&
                           ((b + 1) << P) > Work::first_key(a, x)
                       ? max(a.table[x.r * a.table_stride + b], -1)
                       : kNothing;
        };
        int32_t u = more ? it.u0 : 0;
        int32_t page = more ? page_of(it, u) : kNothing;
        while (more) {
            Item nx = it;
            int32_t nu = u + kBatch;
            bool nmore = true;
            if (nu >= it.u1) {
                nmore = Work::next(a, sh, nx);
                nu = nx.u0;
            }
            const int32_t npage = nmore ? page_of(nx, nu) : kNothing;
            const int n = min(kBatch, it.u1 - u);
            const uint32_t k = sent + sub, slot = k % ST;
            const uint32_t fb = smem_u32(&full_bar[slot]);
            const bool free_slot =
                sub >= n || k < ST ||
                mbar_wait(smem_u32(&empty_bar[slot]), (k / ST - 1) & 1, abort_flag, a.status);
            if (!__all_sync(0xFFFFFFFFu, free_slot))
                break;
            const bool ok = page >= 0 && page < a.c.num_pages;
            // a page outside the pool counts as zeros (no bytes of other pages stay in its place)
            if (!ok && page != kNothing) {
                bad = true;
                uint8_t* place = smem + slot * C::kStageBytes + in_slot;
                for (uint32_t i = 0; i < bytes; i += 16)
                    *reinterpret_cast<uint4*>(place + i) = make_uint4(0u, 0u, 0u, 0u);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            // a piece past the request's end or before its window is left out: its place
            // holds old bytes, which count for nothing
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, ok) >> (4 * sub) & 0xFu;
            if (piece == 0 && sub < n) {
                const uint32_t all = by_page ? __popc(there) * bytes : there ? C::kStageBytes : 0;
                if (all)
                    mbar_expect_tx(fb, all);
                else
                    mbar_arrive(fb);
            }
            __syncwarp();
            if (ok) {
                const int32_t off =
                    by_page ? 0 : ((it.first + u + sub) * kGroup) & ((1 << P) - 1);
                bulk_copy(ring + slot * C::kStageBytes + in_slot,
                          src0 + page * a.c.page_stride + it.h * head_bytes + off * row_bytes,
                          bytes, fb);
            }
            sent += n;
            it = nx;
            u = nu;
            page = npage;
            more = nmore;
        }
        // copies still in flight must land before the CTA ends, also where a wait of another
        // warp runs out after this one is through
        for (uint32_t k = sent > ST ? sent - ST : 0; k < sent; ++k) {
            const long long t0 = clock64();
            while (!mbar_test(smem_u32(&full_bar[k % ST]), (k / ST) & 1) &&
                   clock64() - t0 < kKvWaitBudget) {
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
            atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
        if (a.all_rows)
            kv_write_other_rows(a, lane, 32);
        kv_pdl_end<S>();
        return;
    }

    const int g = lane >> 2, t = lane & 3;
    const float vg = a.c.v_g[0], qk = a.scale_log2 * a.c.k_g[0];
    const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar);
    uint32_t taken = 0;  // groups of the items before
    // a group is blocks of 2^bs tokens: K codes, V codes, K scales, V scales each
    const int bs = min(a.c.page_shift, 6);
    const int v_part = (D / 2) << bs, s_part = (D / 16) << bs, whole_block = (D * 9 / 8) << bs;
    // from 16 tokens to the next 16, and from unit to unit, of codes and of scales
    const int code_half = bs == 4 ? whole_block : 16 * (D / 2);
    const int scale_half = bs == 4 ? whole_block : 16 * (D / 16);
    const int code_step = bs == 4 ? 2 * whole_block : bs == 5 ? whole_block : kUnit * (D / 2);
    const int scale_step = bs == 4 ? 2 * whole_block : bs == 5 ? whole_block : kUnit * (D / 16);
    const int ka = token_of_row(g), v_tok = token_of_row(2 * t), v_odd = token_of_row(2 * t + 1) - v_tok;
    constexpr int HB = NT == 1 && !SPLIT ? kUnit / 16 : 1;  // 16-token halves in flight at once

    // four consecutive elements of row c of an item's query tile
    auto query = [&](const Item& x, int c) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const int row = x.row0 + c;
        if (c < R && row < x.row1 && 4 * lane < D) {
            const int tok = kv_token(a, row);
            const int64_t at = (x.q.base + tok) * a.q_stride +
                               (int64_t)(x.h * a.group + row - tok * a.group) * D + 4 * lane;
            if (a.q_bf16) {
                const uint2 w =
                    *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at);
                v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
            } else {
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
            }
        }
        return v;
    };
    constexpr int QR = (R + kWarps - 1) / kWarps;
    float4 qv[QR];  // the next item's rows warp, warp + kWarps ..
    if (more) {
#pragma unroll
        for (int j = 0; j < QR; ++j)
            qv[j] = query(it, warp + j * kWarps);
    }

    while (more) {
        const int32_t u0 = it.u0, u1 = it.u1;
        const int units = (u1 - u0) * kSub;
        const int32_t first_tok = (it.first + u0) * kGroup;

        // queries of this item as B fragments, in f16 terms, rows scaled by powers of two
#pragma unroll
        for (int j = 0; j < QR; ++j) {
            const int c = warp + j * kWarps;
            if (c >= R)
                break;
            float4 v = qv[j];
            const float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
            const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));
            // 2^(14 - exponent of the largest), kept a normal number
            const int e = min(max(14 - ((int)(bits >> 23) - 127), -100), 100);
            const float up = bits ? __uint_as_float((uint32_t)(e + 127) << 23) : 1.0f;
            const float down = bits ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f;
            if (4 * lane < D) {
                v.x *= up, v.y *= up, v.z *= up, v.w *= up;
                const int at = ((c >> 3) * KS + lane % KS) * 32 + (c & 7) * 4 + lane / KS;
                const uint2 h = make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
                sq[at] = h;
                if constexpr (SPLIT)
                    sq[NT * KS * 32 + at] =
                        make_uint2(pack_rest(v.x, v.y, h.x), pack_rest(v.z, v.w, h.y));
            }
            if (lane == 0) {
                const int row = it.row0 + c;
                sm_f[c] = qk * down;
                sm_pos[c] = row < it.row1 ? kv_position<S>(it.q, kv_token(a, row)) : -1;
            }
        }
        compute_sync();

        uint2 qf[C::kQRegs ? C::kQTerms * NT * KS : 1];
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int j = 0; j < C::kQTerms * NT * KS; ++j)
                qf[j] = sq[j * 32 + lane];
        }
        float f[NT][2], m[NT][2], l[NT][2], acc[NT][KS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[nt][e] = sm_f[nt * 8 + 2 * t + e];
                m[nt][e] = -INFINITY;  // reference minus kLift
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[nt][i][e] = 0.f;
        }
        // positions every row of the tile sees: keys in [all_lo, all_hi]
        const int32_t all_hi = kv_position<S>(it.q, kv_token(a, it.row0));
        const int32_t all_lo = Work::first_key(a, it.q, kv_token(a, it.row1 - 1));

        for (int i = (warp + kWarps - taken * kSub % kWarps) % kWarps; i < units; i += kWarps) {
            const uint32_t group = taken + i / kSub, slot = group % ST;
            const int32_t unit0 = first_tok + i * kUnit;
            mbar_wait(full0 + 8 * slot, (group / ST) & 1, abort_flag, a.status);
            // Lanes poll each for itself.  One that is still at it when another frees the slot
            // could find the phase after next and wait for good; and the MMAs want a whole warp.
            __syncwarp();
            if (unit0 < it.q.seq) {  // else past the end: nothing to do in this unit
                const uint8_t* st = smem + slot * C::kStageBytes + (i % kSub) * code_step;
                const uint8_t* sk = smem + slot * C::kStageBytes + 2 * v_part + (i % kSub) * scale_step;
#pragma unroll HB
                for (int h0 = 0; h0 < kUnit / 16; h0 += HB) {
                    const int32_t tok0 = unit0 + 16 * h0;

                    // ---- S^T = K Q^T: HB times 16 tokens x 8 NT rows ---------------------------
                    float s[HB][NT][4];
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        const uint8_t* kc = st + (h0 + h) * code_half;
                        const uint8_t* ks = sk + (h0 + h) * scale_half;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                s[h][nt][e] = 0.f;
                        float rest[SPLIT ? NT : 1][4] = {};
                        uint32_t wa[D / 32], wb[D / 32];
                        uint32_t sa[D / 64], sb[D / 64];  // block scales of the two rows, doubled
                        if constexpr (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(kc + ka * 64 + 16 * t);
                            const uint4 y =
                                *reinterpret_cast<const uint4*>(kc + (ka + 8) * 64 + 16 * t);
                            wa[0] = x.x, wa[1] = x.y, wa[2] = x.z, wa[3] = x.w;
                            wb[0] = y.x, wb[1] = y.y, wb[2] = y.z, wb[3] = y.w;
                            const uint32_t u = e4m3x2_to_f16x2_bits(
                                *reinterpret_cast<const uint16_t*>(ks + ka * 8 + 2 * t));
                            const uint32_t v = e4m3x2_to_f16x2_bits(
                                *reinterpret_cast<const uint16_t*>(ks + (ka + 8) * 8 + 2 * t));
                            sa[0] = f16x2_dup_lo(u), sa[1] = f16x2_dup_hi(u);
                            sb[0] = f16x2_dup_lo(v), sb[1] = f16x2_dup_hi(v);
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(kc + ka * 32 + 8 * t);
                            const uint2 y =
                                *reinterpret_cast<const uint2*>(kc + (ka + 8) * 32 + 8 * t);
                            wa[0] = x.x, wa[1] = x.y;
                            wb[0] = y.x, wb[1] = y.y;
                            const uint32_t two = e4m3x2_to_f16x2_bits(
                                ks[ka * 4 + t] | (ks[(ka + 8) * 4 + t] << 8));
                            sa[0] = f16x2_dup_lo(two);
                            sb[0] = f16x2_dup_hi(two);
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            uint32_t ha[4], hb[4];
                            e2m1x8_to_f16(wa[w], ha);
                            e2m1x8_to_f16(wb[w], hb);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                ha[e] = f16x2_mul(ha[e], sa[w / 2]);
                                hb[e] = f16x2_mul(hb[e], sb[w / 2]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int x = 0; x < C::kQTerms; ++x)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int j = (x * NT + nt) * KS + 2 * w + e;
                                        const uint2 b =
                                            C::kQRegs ? qf[C::kQRegs ? j : 0] : sq[j * 32 + lane];
                                        // small terms (the queries' second) on their own
                                        mma_m16n8k16(x ? rest[nt] : s[h][nt], ha[2 * e], hb[2 * e],
                                                     ha[2 * e + 1], hb[2 * e + 1], b.x, b.y);
                                    }
                        }
                        if constexpr (SPLIT) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    s[h][nt][e] += rest[nt][e];
                        }
                    }

                    // ---- softmax: rows of S^T are tokens ka, ka + 8; columns 2t, 2t + 1 ----------
                    float x[HB][NT][4];
                    float top = 0.f;
#pragma unroll
                    for (int h = 0; h < HB; ++h)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[h][nt][e] = fmaf(s[h][nt][e], f[nt][e & 1], -m[nt][e & 1]);
                    const bool edge = tok0 < all_lo || tok0 + 16 * HB - 1 > all_hi;
                    if (edge) {
#pragma unroll
                        for (int h = 0; h < HB; ++h)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int32_t pos = sm_pos[nt * 8 + 2 * t + (e & 1)];
                                    const int32_t tok = tok0 + 16 * h + ka + (e < 2 ? 0 : 8);
                                    if (tok > pos || (S == KvSees::kCausal ? a.window > 0 && tok <= pos - a.window
                                                                           : tok < all_lo)) {
                                        x[h][nt][e] = -INFINITY;
                                        s[h][nt][e] = -INFINITY;
                                    }
                                }
                    }
#pragma unroll
                    for (int h = 0; h < HB; ++h)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                top = fmaxf(top, x[h][nt][e]);
                    if (__any_sync(0xFFFFFFFFu, top > kLift + kRaise)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                // a masked score stays at -inf whatever the factor
                                float most = -INFINITY;
#pragma unroll
                                for (int h = 0; h < HB; ++h)
#pragma unroll
                                    for (int y = e; y < 4; y += 2)
                                        if (s[h][nt][y] != -INFINITY)
                                            most = fmaxf(most, s[h][nt][y] * f[nt][e]);
                                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 4));
                                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 8));
                                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 16));
                                const float now = fmaxf(m[nt][e], most - kLift);
                                const float by = m[nt][e] == now ? 1.f : ex2(m[nt][e] - now);
                                m[nt][e] = now;
                                l[nt][e] *= by;
#pragma unroll
                                for (int k = 0; k < KS; ++k) {
                                    acc[nt][k][e] *= by;
                                    acc[nt][k][e + 2] *= by;
                                }
#pragma unroll
                                for (int h = 0; h < HB; ++h)
#pragma unroll
                                    for (int y = e; y < 4; y += 2)
                                        x[h][nt][y] = s[h][nt][y] == -INFINITY
                                                          ? -INFINITY
                                                          : fmaf(s[h][nt][y], f[nt][e], -now);
                            }
                    }
                    uint32_t pb[HB][C::kQTerms][NT][2];  // P^T as B fragments
#pragma unroll
                    for (int h = 0; h < HB; ++h)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float p[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                p[e] = ex2(x[h][nt][e]);
                            l[nt][0] += p[0] + p[2];
                            l[nt][1] += p[1] + p[3];
                            const uint32_t h0_ = pack_f16(p[0], p[1]), h1_ = pack_f16(p[2], p[3]);
                            pb[h][0][nt][0] = movm_trans(h0_);
                            pb[h][0][nt][1] = movm_trans(h1_);
                            if constexpr (SPLIT) {
                                pb[h][1][nt][0] = movm_trans(pack_rest(p[0], p[1], h0_));
                                pb[h][1][nt][1] = movm_trans(pack_rest(p[2], p[3], h1_));
                            }
                        }

                    // ---- O^T += V^T P^T: this lane's eighth of the head dim, tokens of rows 2t .. --
                    uint32_t vw[HB][4][D / 64], vs[HB][2];
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        const uint8_t* sv = st + (h0 + h) * code_half + v_part;
                        const uint8_t* ss = sk + (h0 + h) * scale_half + s_part;
                        uint32_t one[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int vt = v_tok + (k >> 1) * 8 + (k & 1) * v_odd;
                            if constexpr (D == 128) {
                                const uint2 v = *reinterpret_cast<const uint2*>(sv + vt * 64 + 8 * g);
                                vw[h][k][0] = v.x, vw[h][k][1] = v.y;
                                one[k] = ss[vt * 8 + g];
                            } else {
                                vw[h][k][0] = *reinterpret_cast<const uint32_t*>(sv + vt * 32 + 4 * g);
                                one[k] = ss[vt * 4 + (g >> 1)];
                            }
                        }
                        if (edge) {  // past the end and before the window may be anything
                            const int32_t key0 = Work::first_key(a, it);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int32_t tok = tok0 + 16 * h + v_tok + (k >> 1) * 8 + (k & 1) * v_odd;
                                if (tok >= it.q.seq || tok < key0) {
                                    one[k] = 0;
#pragma unroll
                                    for (int w = 0; w < D / 64; ++w)
                                        vw[h][k][w] = 0;
                                }
                            }
                        }
                        vs[h][0] = one[0] | (one[1] << 8);
                        vs[h][1] = one[2] | (one[3] << 8);
                    }
                    if (h0 + HB == kUnit / 16) {  // all read: the slot can be filled again
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(empty0 + 8 * slot);
                    }
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        const uint32_t s01 = e4m3x2_to_f16x2_bits(vs[h][0]);
                        const uint32_t s23 = e4m3x2_to_f16x2_bits(vs[h][1]);
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) {
                            constexpr uint32_t kLow = 0x0F0F0F0Fu;
                            const uint32_t x0 = vw[h][0][w], x1 = vw[h][1][w];
                            const uint32_t x2 = vw[h][2][w], x3 = vw[h][3][w];
                            uint32_t e0[4], e1[4], o0[4], o1[4];  // even / odd elements, token pairs
                            e2m1x8_to_f16((x0 & kLow) | ((x1 << 4) & ~kLow), e0);
                            e2m1x8_to_f16(((x0 >> 4) & kLow) | (x1 & ~kLow), o0);
                            e2m1x8_to_f16((x2 & kLow) | ((x3 << 4) & ~kLow), e1);
                            e2m1x8_to_f16(((x2 >> 4) & kLow) | (x3 & ~kLow), o1);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t a0 = f16x2_mul(e0[k], s01), a1 = f16x2_mul(o0[k], s01);
                                const uint32_t a2 = f16x2_mul(e1[k], s23), a3 = f16x2_mul(o1[k], s23);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float(&o)[4] = acc[nt][4 * w + k];
                                    if constexpr (SPLIT) {
                                        // the MMA's own sums are cut off, not rounded: these 16
                                        // tokens are summed alone and added in FP32
                                        float sum[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma_m16n8k16(sum, a0, a1, a2, a3, pb[h][1][nt][0], pb[h][1][nt][1]);
                                        mma_m16n8k16(sum, a0, a1, a2, a3, pb[h][0][nt][0], pb[h][0][nt][1]);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            o[e] += sum[e];
                                    } else {
                                        mma_m16n8k16(o, a0, a1, a2, a3, pb[h][0][nt][0], pb[h][0][nt][1]);
                                    }
                                }
                            }
                        }
                    }
                }
            } else if (lane == 0) {
                mbar_arrive(empty0 + 8 * slot);
            }
        }

        // ---- join the warps ---------------------------------------------------------------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
                if (g == 0) {
                    sm_m[warp][nt * 8 + 2 * t + e] = m[nt][e];
                    sm_l[warp][nt * 8 + 2 * t + e] = v;
                }
            }
        compute_sync();

        taken += u1 - u0;
        // the next item's queries are on their way during the join
        Item nx = it;
        more = Work::next(a, sh, nx);
        if (more) {
#pragma unroll
            for (int j = 0; j < QR; ++j)
                qv[j] = query(nx, warp + j * kWarps);
        }

        const bool whole = u0 == 0 && u1 == it.n;
        const int32_t slot = 2 * blockIdx.x + (u0 == 0 ? 1 : 0);
        constexpr int kFrag = KS * 32;  // float4 fragments of 8 rows
        constexpr int64_t kPart = (int64_t)NT * kFrag * 4 + 2 * R;  // floats of a partial result

        // (row, two elements) of a fragment entry to the output
        auto store2 = [&](int col, int fi, int fl, float v0, float v1, float ltot) {
            const int row = it.row0 + col;
            if (row >= it.row1)
                return;
            const int tok = kv_token(a, row);
            const float inv = ltot == 0.f ? 0.f : vg / ltot;
            const int64_t at = (it.q.base + tok) * a.out_stride +
                               (int64_t)(it.h * a.group + row - tok * a.group) * D +
                               (D / 8) * (fl >> 2) + 2 * fi;
            if (a.out_bf16) {
                *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) =
                    __floats2bfloat162_rn(v0 * inv, v1 * inv);
            } else {
                *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) =
                    make_float2(v0 * inv, v1 * inv);
            }
        };
        auto store_lse = [&](int col, float mtot, float ltot) {
            const int row = it.row0 + col;
            if (a.lse == nullptr || row >= it.row1)
                return;
            const int tok = kv_token(a, row);
            a.lse[(int64_t)(it.q.base + tok) * (a.c.heads * a.group) + it.h * a.group + row -
                  tok * a.group] =
                ltot == 0.f ? -INFINITY : 0.6931471805599453f * (mtot + log2f(ltot));
        };
        // a row's sums as they are, in the row's own place or in this CTA's part of the item
        const bool keep = S == KvSees::kBehind || (S == KvSees::kAll && a.keep.rows != nullptr);
        auto keep_stats = [&](int col, float mtot, float ltot) {
            const int row = it.row0 + col;
            if (row >= it.row1)
                return;
            const int tok = kv_token(a, row);
            const int64_t at = (int64_t)(it.q.base + tok) * (a.c.heads * a.group) + it.h * a.group + row -
                               tok * a.group;
            (whole ? a.keep.stats[at] : a.keep.part_stats[(int64_t)slot * R + col]) = make_float2(mtot, ltot);
            if (u0 == 0)
                a.keep.where[at] = (whole ? 0
                                          : (Work::last_cta(sh, it) - Work::first_cta(sh, it) + 1) << kKvPartBits |
                                                (slot * R + col)) |
                                   (S == KvSees::kBehind && it.q.low > 0 ? kKvSharesBit : 0);
        };
        auto keep2 = [&](int col, int fi, int fl, float v0, float v1) {
            const int row = it.row0 + col;
            if (row >= it.row1)
                return;
            const int tok = kv_token(a, row);
            const int64_t at = (int64_t)(it.q.base + tok) * (a.c.heads * a.group) + it.h * a.group + row -
                               tok * a.group;
            float* dst = whole ? a.keep.rows + at * D : a.keep.parts + ((int64_t)slot * R + col) * D;
            *reinterpret_cast<float2*>(dst + (D / 8) * (fl >> 2) + 2 * fi) = make_float2(v0, v1);
        };
        // a column's largest reference of the warps, by which all rescale
        auto column = [&](int col) {
            float mt = sm_m[0][col];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                mt = fmaxf(mt, sm_m[w][col]);
            return mt;
        };
        if (tid < R) {
            const float mt = column(tid);
            float lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                lt += sm_m[w][tid] == mt ? sm_l[w][tid] : sm_l[w][tid] * ex2(sm_m[w][tid] - mt);
            sm_sum[tid] = lt;
            if (keep) {
                keep_stats(tid, mt, lt);
            } else if (whole) {
                store_lse(tid, mt, lt);
            } else {
                float* ml = a.part + slot * kPart + (int64_t)NT * kFrag * 4;
                ml[tid] = mt;
                ml[R + tid] = lt;
            }
        }

#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float by[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mt = column(nt * 8 + 2 * t + e);
                by[e] = m[nt][e] == mt ? 1.f : ex2(m[nt][e] - mt);
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
                red[(warp * KS + i) * 32 + lane] =
                    make_float4(acc[nt][i][0] * by[0], acc[nt][i][1] * by[1],
                                acc[nt][i][2] * by[0], acc[nt][i][3] * by[1]);
            compute_sync();
            for (int e = tid; e < kFrag; e += kCompute) {
                float4 v = red[e];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 o = red[w * kFrag + e];
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                if (keep) {
                    const int col = nt * 8 + 2 * (e & 3);
                    keep2(col, e >> 5, e & 31, v.x, v.z);
                    keep2(col + 1, e >> 5, e & 31, v.y, v.w);
                } else if (whole) {
                    const int col = nt * 8 + 2 * (e & 3);
                    store2(col, e >> 5, e & 31, v.x, v.z, sm_sum[col]);
                    store2(col + 1, e >> 5, e & 31, v.y, v.w, sm_sum[col + 1]);
                } else {
                    reinterpret_cast<float4*>(a.part + slot * kPart)[nt * kFrag + e] = v;
                }
            }
            compute_sync();
        }
        if (S != KvSees::kBehind && !whole && !keep) {
            // ---- join the CTAs: the last to arrive sums all parts in CTA order ----------------
            const int ca = Work::first_cta(sh, it), cb = Work::last_cta(sh, it);
            if (tid == 0) {
                // releases the CTA's writes (the barrier above orders them before) and,
                // for the last to arrive, acquires the others'
                unsigned seen;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                             : "=r"(seen) : "l"(a.count + ca) : "memory");
                last_s = seen == (unsigned)(cb - ca);
                if (last_s)
                    a.count[ca] = 0u;
            }
            compute_sync();
            if (last_s) {
                // part c's entries, then references [R] and sums [R]
                auto part_of = [&](int c) { return a.part + (2 * c + (c == ca)) * kPart; };
                constexpr int64_t kMl = (int64_t)NT * kFrag * 4;
                // a thread a (column, part) of up to kStep parts at a time
                constexpr int kStep = kCompute / R;
                constexpr int kOwn = (NT * kFrag + kCompute - 1) / kCompute;
                float* scratch = reinterpret_cast<float*>(red);       // [kStep][R] references
                float* factor = scratch + kCompute;                   // [kStep][R] factors
                float* summed = factor + kCompute;                    // [kStep][R] sums
                static_assert(3 * kCompute * 4 <= C::kRedBytes, "the join's tables");
                const int col = tid % R, k0 = tid / R;
                float mt = -INFINITY, lt = 0.f;  // so far, of column col
                float4 v[kOwn];
#pragma unroll
                for (int j = 0; j < kOwn; ++j)
                    v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c0 = ca; c0 <= cb; c0 += kStep) {
                    const int n = min(kStep, cb - c0 + 1);
                    float mc = -INFINITY, lc = 0.f;
                    if (k0 < n) {
                        const float* ml = part_of(c0 + k0) + kMl + col;
                        mc = __ldcg(ml);
                        lc = __ldcg(ml + R);
                    }
                    scratch[tid] = mc;
                    compute_sync();
                    float top = mt;
                    for (int k = 0; k < n; ++k)
                        top = fmaxf(top, scratch[k * R + col]);
                    const float by = mc == top ? 1.f : ex2(mc - top);
                    factor[tid] = by;
                    summed[tid] = by * lc;
                    if (k0 == 0)  // what was joined so far, against the new reference
                        sm_f[col] = mt == top ? 1.f : ex2(mt - top);
                    compute_sync();
                    lt *= mt == top ? 1.f : ex2(mt - top);
                    for (int k = 0; k < n; ++k)
                        lt += summed[k * R + col];
                    mt = top;
#pragma unroll
                    for (int j = 0; j < kOwn; ++j) {
                        const int c2 = ((tid + j * kCompute) / kFrag) * 8 + 2 * (tid & 3);
                        const float o0 = c2 < R ? sm_f[c2] : 0.f, o1 = c2 < R ? sm_f[c2 + 1] : 0.f;
                        v[j].x *= o0, v[j].y *= o1, v[j].z *= o0, v[j].w *= o1;
                    }
                    // kAhead parts' entries on their way at once
                    constexpr int kAhead = kOwn <= 2 ? 8 : 2;
                    for (int k = 0; k < n; k += kAhead) {
                        float4 o[kAhead][kOwn];
#pragma unroll
                        for (int i = 0; i < kAhead; ++i)
#pragma unroll
                            for (int j = 0; j < kOwn; ++j) {
                                const int e = tid + j * kCompute;
                                o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (k + i < n && e < NT * kFrag)
                                    o[i][j] = __ldcg(
                                        reinterpret_cast<const float4*>(part_of(c0 + k + i)) + e);
                            }
#pragma unroll
                        for (int i = 0; i < kAhead; ++i)
#pragma unroll
                            for (int j = 0; j < kOwn; ++j) {
                                const int e = tid + j * kCompute;
                                if (k + i < n && e < NT * kFrag) {
                                    const float* by = factor + (k + i) * R + (e / kFrag) * 8 + 2 * (e & 3);
                                    v[j].x = fmaf(o[i][j].x, by[0], v[j].x);
                                    v[j].y = fmaf(o[i][j].y, by[1], v[j].y);
                                    v[j].z = fmaf(o[i][j].z, by[0], v[j].z);
                                    v[j].w = fmaf(o[i][j].w, by[1], v[j].w);
                                }
                            }
                    }
                    compute_sync();  // the tables are free
                }
                if (k0 == 0) {
                    sm_sum[col] = lt;
                    store_lse(col, mt, lt);
                }
                compute_sync();
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    const int e = tid + j * kCompute, f = e % kFrag;
                    if (e >= NT * kFrag)
                        break;
                    const int c2 = (e / kFrag) * 8 + 2 * (e & 3);
                    store2(c2, f >> 5, f & 31, v[j].x, v[j].z, sm_sum[c2]);
                    store2(c2 + 1, f >> 5, f & 31, v[j].y, v[j].w, sm_sum[c2 + 1]);
                }
            }
        }
        compute_sync();  // shared memory is free for the next item
        it = nx;
    }
    kv_pdl_end<S>();
}

template <KvSees S, int D, int NT, bool SPLIT, int W>
cudaError_t launch(const KvAttnArgs& a, cudaStream_t stream, bool pdl)
{
    using C = Cfg<D, NT, SPLIT, W>;
    const int dev = current_device();
    auto* kern = &kv_rows_kernel<S, D, NT, SPLIT, W>;
    const cudaError_t e = ensure_smem_limit(kern, C::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    // the workspace holds two partial results of kMaxCtas CTAs with items of kMaxRows rows
    constexpr int kMost = kMaxCtas * (kMaxRows / C::R) < kKvCountBytes / 4 ? kMaxCtas * (kMaxRows / C::R)
                                                                           : (int)(kKvCountBytes / 4);
    const int grid = device_sm_count(dev) * C::kCtas;
    return kv_launch(kern, grid > kMost ? kMost : grid, C::kThreads, C::kSmem, stream, pdl, a);
}

inline int item_rows(const KvAttnArgs& a)
{
    const int64_t rows = (int64_t)a.max_q * a.group;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

template <KvSees S, int D, bool SPLIT>
cudaError_t launch_rows(const KvAttnArgs& a, cudaStream_t stream, bool pdl)
{
    switch (item_rows(a)) {
    case 8:
        return launch<S, D, 1, SPLIT, S == KvSees::kBehind ? 3 : 7>(a, stream, pdl);
    case 16:
        return launch<S, D, 2, SPLIT, 7>(a, stream, pdl);
    default:
        return launch<S, D, 4, SPLIT, 7>(a, stream, pdl);
    }
}

}  // namespace

// One translation unit for each S (the twelve kernels of one take a minute to compile).
template <KvSees S>
cudaError_t launch_kv_rows(const KvAttnArgs& args, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl)
{
    KvAttnArgs a = args;
    a.count = nullptr;
    a.part = nullptr;
    if (a.keep.rows) {
        a.part = a.keep.parts;  // items may be cut
    } else if (workspace_bytes >= kv_rows_workspace_bytes(a.c.dim)) {
        a.count = static_cast<unsigned*>(workspace);
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kKvCountBytes);
    }
    const bool split = !a.q_bf16 || !a.out_bf16;
    if (a.c.dim == 128)
        return split ? launch_rows<S, 128, true>(a, stream, pdl) : launch_rows<S, 128, false>(a, stream, pdl);
    return split ? launch_rows<S, 64, true>(a, stream, pdl) : launch_rows<S, 64, false>(a, stream, pdl);
}

}  // namespace nvfp4

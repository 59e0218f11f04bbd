// kv_attention_rows.cu -- attention over the paged NVFP4 cache with few query
// rows a request: single tokens, drafted tokens, short prompts.
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
// f16 (outputs in BF16) or two (FP32), against exact values.
//
// Layout.  The query rows (token, head of the group) are the narrow side of
// m16n8k16 tiles, 8 NT of them: S^T = K Q^T and O^T = V^T P^T, so a single
// token of a group of 4 to 8 heads fills the tile and the 4-bit cache is
// decoded once for all of them.  A warp takes 16 tokens at a time: lane
// (g, t) = (lane / 4, lane % 4) reads K of token rows g, g + 8 -- its quarter
// of the head dim, one vector -- and V of four tokens -- its eighth -- so that
// every load is one contiguous vector and a lane meets one or two block scales
// a token.  V's codes of two tokens are interleaved as nibbles before they are
// converted, which gives the f16 pairs along the tokens that the MMA wants.
//
// Work.  One list of 16-token units for all requests (kv.cuh), equal shares a
// CTA, the units of an item dealt to the CTA's warps in turn; each warp feeds
// itself through its own ring of cp.async copies, no barrier in the loop.
// Warps join through shared memory at an item's end; items cut between CTAs
// are joined by the last of them to arrive, in CTA order.
//
// Bound by the cache's bytes for one token a request.
#include "../../include/nvfp4_kv.h"
#include "formats.cuh"
#include "kv.cuh"
#include "launch_cache.cuh"
#include "mma_frag.cuh"

namespace nvfp4 {

namespace {

constexpr int kUnit = 16;       // tokens a unit
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 512;   // workspace extent
constexpr int kMaxRows = 32;
constexpr float kRaise = 8.0f;  // log2 a score may pass the reference by
constexpr float kLift = 7.0f;   // p = 2^(s - m + kLift)

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t movm_trans(uint32_t v)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// What an f16 pair leaves of the two floats it came from, as another pair.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_f16(lo - f.x, hi - f.y);
}

// MMA row k of a unit holds this token: rows 2j are tokens 0..3, rows 2j + 1
// tokens 4..7 (paired j with j ^ 1), and the same eight further on; so the
// four lanes of a V load and the two rows of a K load phase fall on different
// banks as far as 64-byte rows allow.
__device__ __forceinline__ int token_of_row(int k)
{
    const int j = (k & 7) >> 1;
    return (k & 8) | ((k & 1) ? 4 + (j ^ 1) : j);
}

// The place of an item in the work list.
struct Item {
    int r, h, tile;
    KvReq q;
    int rows;       // query rows of the request (tokens * group)
    int row0, row1;
    int64_t begin;  // first unit in the list
    int32_t first, n;
};

template <int R>
__device__ __forceinline__ void item_units(const KvAttnArgs& a, Item& it)
{
    it.row0 = it.tile * R;
    it.row1 = min(it.row0 + R, it.rows);
    kv_tile_units<kUnit>(a, it.q, it.row0, it.row1, it.first, it.n);
}

// The first item of the first request at or after r that has rows.
template <int R>
__device__ __forceinline__ bool item_request(const KvAttnArgs& a, Item& it, int r)
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
    item_units<R>(a, it);
    return true;
}

template <int R>
__device__ __forceinline__ bool item_next(const KvAttnArgs& a, Item& it)
{
    it.begin += it.n;
    if ((it.tile + 1) * R < it.rows) {
        ++it.tile;
        item_units<R>(a, it);
        return true;
    }
    it.tile = 0;
    if (++it.h < a.c.heads) {
        item_units<R>(a, it);
        return true;
    }
    return item_request<R>(a, it, it.r + 1);
}

// Units of one kv head of a request.
template <int R>
__device__ __forceinline__ int64_t head_units(const KvAttnArgs& a, const KvReq& q)
{
    int64_t s = 0;
    const int rows = q.nq * a.group;
    for (int row0 = 0; row0 < rows; row0 += R) {
        int32_t first, n;
        kv_tile_units<kUnit>(a, q, row0, min(row0 + R, rows), first, n);
        s += n;
    }
    return s;
}

template <int D, int NT, bool SPLIT>
struct Cfg {
    static constexpr int R = 8 * NT;             // query rows a tile
    static constexpr int KS = D / 16;            // k16 steps of Q K, m16 tiles of V
    static constexpr int kCode = kUnit * D / 2;  // bytes of a unit's K (or V) codes
    static constexpr int kScale = kUnit * D / 16;
    static constexpr int kStageBytes = 2 * kCode + 2 * kScale;
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kQTerms = SPLIT ? 2 : 1;
    static constexpr int kQBytes = kQTerms * NT * KS * 32 * 8;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kRedBytes = kWarps * KS * 32 * 16;
    static constexpr int kMain = kRingBytes > kRedBytes ? kRingBytes : kRedBytes;
    static constexpr int kSmem = kMain + kQBytes;
    static constexpr bool kQRegs = NT * kQTerms <= 2;  // queries held in registers
};

template <int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kCtasPerSm : 1)
    kv_rows_kernel(const KvAttnArgs a)
{
    using C = Cfg<D, NT, SPLIT>;
    constexpr int R = C::R, KS = C::KS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t warp_sum[kWarps];
    __shared__ int64_t found_rem;
    __shared__ int found_r;
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R], sm_f[R];
    __shared__ int32_t sm_pos[R];
    __shared__ int last_s;
    uint2* sq = reinterpret_cast<uint2*>(smem + C::kMain);

    kv_pdl_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    // ---- this CTA's share of the list ------------------------------------------------
    const int per = (a.reqs + kThreads - 1) / kThreads;
    const int ra = min(tid * per, a.reqs), rb = min(ra + per, a.reqs);
    int64_t mine = 0;
    for (int r = ra; r < rb; ++r) {
        mine += a.c.heads * head_units<R>(a, kv_req(a, r));
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
        warp_sum[warp] = inc;
    __syncthreads();
    int64_t before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp)
            before += warp_sum[w];
        total += warp_sum[w];
    }
    // at least a unit a warp
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    share = share < kWarps ? kWarps : share;
    const int64_t lo = share * blockIdx.x, hi = min(lo + share, total);
    if (lo >= total)
        return;
    if (lo >= before && lo < before + mine) {
        int64_t at = before;
        for (int r = ra; r < rb; ++r) {
            const int64_t n = a.c.heads * head_units<R>(a, kv_req(a, r));
            if (lo < at + n) {
                found_r = r;
                found_rem = lo - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    Item it;
    it.begin = lo - found_rem;
    bool more = item_request<R>(a, it, found_r);
    if (more) {
        const int64_t hu = head_units<R>(a, it.q);
        it.h = (int)(found_rem / hu);
        it.begin += it.h * hu;
        while (it.begin + it.n <= lo) {
            it.begin += it.n;
            ++it.tile;
            item_units<R>(a, it);
        }
    }
    // without a workspace an item belongs to the CTA whose share it begins in
    const bool cut = a.part != nullptr;
    if (!cut && it.begin < lo)
        more = item_next<R>(a, it);

    const int64_t head_bytes = kv_head_bytes(a.c.page_shift, D);
    const float vg = a.c.v_g[0], qk = a.scale_log2 * a.c.k_g[0];
    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    const uint8_t* ring_gen = smem + warp * C::kStages * C::kStageBytes;
    const int code_part = (D / 2) << a.c.page_shift, scale_part = (D / 16) << a.c.page_shift;
    bool bad = false;

    while (more && it.begin < hi) {
        const int32_t u0 = cut ? (int32_t)max((int64_t)0, lo - it.begin) : 0;
        const int32_t u1 = cut ? (int32_t)min((int64_t)it.n, hi - it.begin) : it.n;
        const int32_t* row_table = a.table + it.r * a.table_stride;
        const int my_n = u1 - u0 > warp ? (u1 - u0 - warp + kWarps - 1) / kWarps : 0;
        const int32_t c0 = it.first + u0 + warp;  // this warp's units: c0, c0 + kWarps ..

        // copies of one unit into a ring slot; the page id was looked up one unit before
        auto page_of = [&](int i) {
            const int32_t b = ((c0 + i * kWarps) * kUnit) >> a.c.page_shift;
            return i < my_n && b < a.max_blocks ? row_table[b] : -1;
        };
        int32_t next_page = page_of(0);
        auto issue = [&](int i) {
            if (i < my_n) {
                const int32_t tok = (c0 + i * kWarps) * kUnit;
                bool ok = next_page >= 0 && next_page < a.c.num_pages;
                if (!ok && tok < it.q.seq)
                    bad = true;
                const int32_t off = tok & ((1 << a.c.page_shift) - 1);
                const uint8_t* src = a.c.pool + (ok ? next_page : 0) * a.c.page_stride +
                                     it.h * head_bytes;
                const uint32_t bytes = ok ? 16u : 0u;
                const uint32_t dst = ring + (i % C::kStages) * C::kStageBytes;
#pragma unroll
                for (int j = lane; j < C::kCode / 16; j += 32) {
                    cp16(dst + 16 * j, src + off * (D / 2) + 16 * j, bytes);
                    cp16(dst + C::kCode + 16 * j, src + code_part + off * (D / 2) + 16 * j, bytes);
                }
                if (lane < 2 * C::kScale / 16) {
                    const int v = lane >= C::kScale / 16, j = lane - v * (C::kScale / 16);
                    cp16(dst + 2 * C::kCode + 16 * lane,
                         src + 2 * code_part + v * scale_part + off * (D / 16) + 16 * j, bytes);
                }
                next_page = page_of(i + 1);
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i)
            issue(i);

        // queries of this item as B fragments, in f16 terms, rows scaled by powers of two
        for (int c = warp; c < R; c += kWarps) {
            const int row = it.row0 + c;
            const bool live = row < it.row1;
            const int tok = live ? row / a.group : 0;
            const int head = it.h * a.group + (live ? row - tok * a.group : 0);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const bool has = 4 * lane < D;
            if (live && has) {
                const int64_t at = (it.q.base + tok) * a.q_stride + (int64_t)head * D + 4 * lane;
                if (a.q_bf16) {
                    const uint2 w =
                        *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at);
                    v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
                } else {
                    v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                }
            }
            const float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
            const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));
            // 2^(14 - exponent of the largest), kept a normal number
            const int e = min(max(14 - ((int)(bits >> 23) - 127), -100), 100);
            const float up = bits ? __uint_as_float((uint32_t)(e + 127) << 23) : 1.0f;
            const float down = bits ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f;
            if (has) {
                v.x *= up, v.y *= up, v.z *= up, v.w *= up;
                const int at = ((c >> 3) * KS + lane % KS) * 32 + (c & 7) * 4 + lane / KS;
                const uint2 h = make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
                sq[at] = h;
                if constexpr (SPLIT)
                    sq[NT * KS * 32 + at] =
                        make_uint2(pack_rest(v.x, v.y, h.x), pack_rest(v.z, v.w, h.y));
            }
            if (lane == 0) {
                sm_f[c] = qk * down;
                sm_pos[c] = live ? it.q.seq - it.q.nq + tok : -1;
            }
        }
        __syncthreads();

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
        const int32_t p0 = it.q.seq - it.q.nq + it.row0 / a.group;
        const int32_t p1 = it.q.seq - it.q.nq + (it.row1 - 1) / a.group;
        const int32_t all_hi = p0, all_lo = a.window > 0 ? p1 - a.window + 1 : 0;

        for (int i = 0; i < my_n; ++i) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            const uint8_t* st = ring_gen + (i % C::kStages) * C::kStageBytes;
            const int32_t tok0 = (c0 + i * kWarps) * kUnit;

            // ---- S^T = K Q^T: 16 tokens x 8 NT rows ----------------------------------------
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[nt][e] = 0.f;
            const int ka = token_of_row(g), kb = ka + 8;
            uint32_t wa[D / 32], wb[D / 32];
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(st + ka * 64 + 16 * t);
                const uint4 y = *reinterpret_cast<const uint4*>(st + kb * 64 + 16 * t);
                wa[0] = x.x, wa[1] = x.y, wa[2] = x.z, wa[3] = x.w;
                wb[0] = y.x, wb[1] = y.y, wb[2] = y.z, wb[3] = y.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(st + ka * 32 + 8 * t);
                const uint2 y = *reinterpret_cast<const uint2*>(st + kb * 32 + 8 * t);
                wa[0] = x.x, wa[1] = x.y;
                wb[0] = y.x, wb[1] = y.y;
            }
            const uint8_t* sk = st + 2 * C::kCode;
            uint32_t sa[D / 64], sb[D / 64];  // this lane's block scales of the two rows, doubled
            if constexpr (D == 128) {
                const uint32_t x = e4m3x2_to_f16x2_bits(
                    *reinterpret_cast<const uint16_t*>(sk + ka * 8 + 2 * t));
                const uint32_t y = e4m3x2_to_f16x2_bits(
                    *reinterpret_cast<const uint16_t*>(sk + kb * 8 + 2 * t));
                sa[0] = f16x2_dup_lo(x), sa[1] = f16x2_dup_hi(x);
                sb[0] = f16x2_dup_lo(y), sb[1] = f16x2_dup_hi(y);
            } else {
                const uint32_t two = e4m3x2_to_f16x2_bits(sk[ka * 4 + t] | (sk[kb * 4 + t] << 8));
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
                            const uint2 b = C::kQRegs ? qf[C::kQRegs ? j : 0] : sq[j * 32 + lane];
                            mma_m16n8k16(s[nt], ha[2 * e], hb[2 * e], ha[2 * e + 1], hb[2 * e + 1],
                                         b.x, b.y);
                        }
            }

            // ---- softmax: rows of S^T are tokens ka, kb; columns 2t, 2t + 1 -----------------
            const bool edge = tok0 < all_lo || tok0 + kUnit - 1 > all_hi;
            bool raise = false;
            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[nt][e] = fmaf(s[nt][e], f[nt][e & 1], -m[nt][e & 1]);
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t pos = sm_pos[nt * 8 + 2 * t + (e & 1)];
                        const int32_t tok = tok0 + (e < 2 ? ka : kb);
                        if (tok > pos || (a.window > 0 && tok <= pos - a.window)) {
                            x[nt][e] = -INFINITY;
                            s[nt][e] = -INFINITY;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    raise |= x[nt][e] > kLift + kRaise;
            if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // a masked score stays at -inf whatever the factor
                        const float s0 = s[nt][e] == -INFINITY ? -INFINITY : s[nt][e] * f[nt][e];
                        const float s1 =
                            s[nt][e + 2] == -INFINITY ? -INFINITY : s[nt][e + 2] * f[nt][e];
                        float top = fmaxf(s0, s1);
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const float now = fmaxf(m[nt][e], top - kLift);
                        const float by = m[nt][e] == now ? 1.f : ex2(m[nt][e] - now);
                        m[nt][e] = now;
                        l[nt][e] *= by;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            acc[nt][k][e] *= by;
                            acc[nt][k][e + 2] *= by;
                        }
                        x[nt][e] = s0 == -INFINITY ? -INFINITY : fmaf(s[nt][e], f[nt][e], -now);
                        x[nt][e + 2] =
                            s1 == -INFINITY ? -INFINITY : fmaf(s[nt][e + 2], f[nt][e], -now);
                    }
            }
            uint32_t pb[C::kQTerms][NT][2];  // P^T as B fragments
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[e] = ex2(x[nt][e]);
                l[nt][0] += p[0] + p[2];
                l[nt][1] += p[1] + p[3];
                const uint32_t h0 = pack_f16(p[0], p[1]), h1 = pack_f16(p[2], p[3]);
                pb[0][nt][0] = movm_trans(h0);
                pb[0][nt][1] = movm_trans(h1);
                if constexpr (SPLIT) {
                    pb[1][nt][0] = movm_trans(pack_rest(p[0], p[1], h0));
                    pb[1][nt][1] = movm_trans(pack_rest(p[2], p[3], h1));
                }
            }

            // ---- O^T += V^T P^T: this lane's eighth of the head dim, tokens of rows 2t ..----
            const uint8_t* sv = st + C::kCode;
            const uint8_t* ss = sk + C::kScale;
            int vt[4];
            uint32_t vw[4][D / 64], vs[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                vt[k] = token_of_row((k >> 1) * 8 + 2 * t + (k & 1));
                if constexpr (D == 128) {
                    const uint2 v = *reinterpret_cast<const uint2*>(sv + vt[k] * 64 + 8 * g);
                    vw[k][0] = v.x, vw[k][1] = v.y;
                    vs[k] = ss[vt[k] * 8 + g];
                } else {
                    vw[k][0] = *reinterpret_cast<const uint32_t*>(sv + vt[k] * 32 + 4 * g);
                    vs[k] = ss[vt[k] * 4 + (g >> 1)];
                }
            }
            if (tok0 + kUnit > it.q.seq) {  // what lies past the end may be anything
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (tok0 + vt[k] >= it.q.seq) {
                        vs[k] = 0;
#pragma unroll
                        for (int w = 0; w < D / 64; ++w)
                            vw[k][w] = 0;
                    }
            }
            const uint32_t s01 = e4m3x2_to_f16x2_bits(vs[0] | (vs[1] << 8));
            const uint32_t s23 = e4m3x2_to_f16x2_bits(vs[2] | (vs[3] << 8));
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                constexpr uint32_t kLow = 0x0F0F0F0Fu;
                uint32_t e0[4], e1[4], o0[4], o1[4];  // even / odd elements of both token pairs
                e2m1x8_to_f16((vw[0][w] & kLow) | ((vw[1][w] << 4) & ~kLow), e0);
                e2m1x8_to_f16(((vw[0][w] >> 4) & kLow) | (vw[1][w] & ~kLow), o0);
                e2m1x8_to_f16((vw[2][w] & kLow) | ((vw[3][w] << 4) & ~kLow), e1);
                e2m1x8_to_f16(((vw[2][w] >> 4) & kLow) | (vw[3][w] & ~kLow), o1);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a0 = f16x2_mul(e0[k], s01), a1 = f16x2_mul(o0[k], s01);
                    const uint32_t a2 = f16x2_mul(e1[k], s23), a3 = f16x2_mul(o1[k], s23);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int y = 0; y < C::kQTerms; ++y)
                            mma_m16n8k16(acc[nt][4 * w + k], a0, a1, a2, a3, pb[y][nt][0],
                                         pb[y][nt][1]);
                }
            }
            __syncwarp();  // every lane has read the slot that the next copies overwrite
            issue(i + C::kStages - 1);
        }
        cp_wait<0>();

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
        __syncthreads();

        const bool whole = u0 == 0 && u1 == it.n;
        const int32_t slot = 2 * blockIdx.x + (u0 == 0 ? 1 : 0);
        constexpr int kFrag = KS * 32;  // float4 fragments of 8 rows
        constexpr int64_t kPart = (int64_t)NT * kFrag * 4 + 2 * R;  // floats of a partial result
        float4* red = reinterpret_cast<float4*>(smem);

        // (row, two elements) of a fragment entry to the output
        auto store2 = [&](int col, int fi, int fl, float v0, float v1, float ltot) {
            const int row = it.row0 + col;
            if (row >= it.row1)
                return;
            const float inv = ltot == 0.f ? 0.f : vg / ltot;
            const int tok = row / a.group;
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
            const int tok = row / a.group;
            a.lse[(int64_t)(it.q.base + tok) * (a.c.heads * a.group) + it.h * a.group + row -
                  tok * a.group] =
                ltot == 0.f ? -INFINITY : 0.6931471805599453f * (mtot + log2f(ltot));
        };
        // reference and sum of a column over the warps
        auto column = [&](int col, float& mtot, float& ltot) {
            mtot = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                mtot = fmaxf(mtot, sm_m[w][col]);
            ltot = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                ltot += sm_m[w][col] == mtot ? sm_l[w][col] : sm_l[w][col] * ex2(sm_m[w][col] - mtot);
        };

#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mt[2], lt[2], by[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                column(nt * 8 + 2 * t + e, mt[e], lt[e]);
                by[e] = m[nt][e] == mt[e] ? 1.f : ex2(m[nt][e] - mt[e]);
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
                red[(warp * KS + i) * 32 + lane] =
                    make_float4(acc[nt][i][0] * by[0], acc[nt][i][1] * by[1],
                                acc[nt][i][2] * by[0], acc[nt][i][3] * by[1]);
            __syncthreads();
            for (int e = tid; e < kFrag; e += kThreads) {
                float4 v = red[e];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 o = red[w * kFrag + e];
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                if (whole) {
                    store2(nt * 8 + 2 * t, e >> 5, e & 31, v.x, v.z, lt[0]);
                    store2(nt * 8 + 2 * t + 1, e >> 5, e & 31, v.y, v.w, lt[1]);
                } else {
                    reinterpret_cast<float4*>(a.part + slot * kPart)[nt * kFrag + e] = v;
                }
            }
            __syncthreads();
        }
        if (tid < R) {
            float mt, lt;
            column(tid, mt, lt);
            if (whole) {
                store_lse(tid, mt, lt);
            } else {
                float* ml = a.part + slot * kPart + (int64_t)NT * kFrag * 4;
                ml[tid] = mt;
                ml[R + tid] = lt;
            }
        }
        if (!whole) {
            // ---- join the CTAs: the last to arrive sums all parts in CTA order ----------------
            const int ca = (int)(it.begin / share), cb = (int)((it.begin + it.n - 1) / share);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned seen = atomicAdd(a.count + ca, 1u);
                last_s = seen == (unsigned)(cb - ca);
                if (last_s)
                    a.count[ca] = 0u;
                __threadfence();
            }
            __syncthreads();
            if (last_s) {
                for (int nt = 0; nt < NT; ++nt)
                    for (int e = tid; e < kFrag; e += kThreads) {
                        const int col = nt * 8 + 2 * (e & 3);
                        float mt[2] = {-INFINITY, -INFINITY}, lt[2] = {0.f, 0.f};
                        for (int c = ca; c <= cb; ++c) {
                            const float* ml = a.part + (2 * c + (c == ca)) * kPart +
                                              (int64_t)NT * kFrag * 4 + col;
                            mt[0] = fmaxf(mt[0], __ldcg(ml));
                            mt[1] = fmaxf(mt[1], __ldcg(ml + 1));
                        }
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int c = ca; c <= cb; ++c) {
                            const float* pc = a.part + (2 * c + (c == ca)) * kPart;
                            const float* ml = pc + (int64_t)NT * kFrag * 4 + col;
                            const float4 o =
                                __ldcg(reinterpret_cast<const float4*>(pc) + nt * kFrag + e);
                            const float m0 = __ldcg(ml), m1 = __ldcg(ml + 1);
                            const float b0 = m0 == mt[0] ? 1.f : ex2(m0 - mt[0]);
                            const float b1 = m1 == mt[1] ? 1.f : ex2(m1 - mt[1]);
                            lt[0] += b0 * __ldcg(ml + R);
                            lt[1] += b1 * __ldcg(ml + R + 1);
                            v.x = fmaf(o.x, b0, v.x), v.y = fmaf(o.y, b1, v.y);
                            v.z = fmaf(o.z, b0, v.z), v.w = fmaf(o.w, b1, v.w);
                        }
                        store2(col, e >> 5, e & 31, v.x, v.z, lt[0]);
                        store2(col + 1, e >> 5, e & 31, v.y, v.w, lt[1]);
                        if (e < 4) {  // one entry a column pair
                            store_lse(col, mt[0], lt[0]);
                            store_lse(col + 1, mt[1], lt[1]);
                        }
                    }
            }
        }
        __syncthreads();  // shared memory is free for the next item
        more = item_next<R>(a, it);
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
        atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
}

template <int D, int NT, bool SPLIT>
cudaError_t launch(const KvAttnArgs& a, cudaStream_t stream, bool pdl)
{
    using C = Cfg<D, NT, SPLIT>;
    const int dev = current_device();
    auto* kern = &kv_rows_kernel<D, NT, SPLIT>;
    const cudaError_t e = ensure_smem_limit(kern, C::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    const int grid = device_sm_count(dev) * (NT == 1 ? kCtasPerSm : 1);
    return kv_launch(kern, grid > kMaxCtas ? kMaxCtas : grid, kThreads, C::kSmem, stream, pdl, a);
}

template <int D, bool SPLIT>
cudaError_t launch_rows(const KvAttnArgs& a, cudaStream_t stream, bool pdl)
{
    const int64_t rows = (int64_t)a.max_q * a.group;
    if (rows <= 8)
        return launch<D, 1, SPLIT>(a, stream, pdl);
    if (rows <= 16)
        return launch<D, 2, SPLIT>(a, stream, pdl);
    return launch<D, 4, SPLIT>(a, stream, pdl);
}

constexpr int64_t kCountBytes = kMaxCtas * sizeof(unsigned);

}  // namespace

// Counters, then two partial results a CTA.
int64_t kv_rows_workspace_bytes(int dim)
{
    return kCountBytes + (int64_t)kMaxCtas * 2 * (kMaxRows * dim + 2 * kMaxRows) * sizeof(float);
}

cudaError_t launch_kv_rows(const KvAttnArgs& args, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl)
{
    KvAttnArgs a = args;
    a.count = nullptr;
    a.part = nullptr;
    if (workspace_bytes >= kv_rows_workspace_bytes(a.c.dim)) {
        a.count = static_cast<unsigned*>(workspace);
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCountBytes);
    }
    const bool split = !a.q_bf16 || !a.out_bf16;
    if (a.c.dim == 128)
        return split ? launch_rows<128, true>(a, stream, pdl) : launch_rows<128, false>(a, stream, pdl);
    return split ? launch_rows<64, true>(a, stream, pdl) : launch_rows<64, false>(a, stream, pdl);
}

}  // namespace nvfp4

// kv_attention_tile.cu -- attention over the paged NVFP4 cache with many query
// rows a request (chunks, whole prompts) on the fifth-generation tensor cores.
//
// Mathematics as in kv_attention_rows.cu: cached values sK cK and sV cV enter as
// exact f16, BF16 query rows scaled by powers of two as (practically) exact f16,
// scores and outputs accumulate in FP32 in tensor memory, the softmax runs online
// against a reference per row that is raised lazily, probabilities enter the
// second product as f16 (scaled by 2^7), row sums are FP32.
//
// One CTA an SM, 256 query rows (token, head of the group) of one kv head as two
// 128-row tiles, 128 keys at a time, warps in four groups:
//   warps 0..3, 4..7   softmax of tile 0, 1, a thread a row: the queries into
//                      shared memory, scores out of tensor memory, probabilities
//                      back into it over the scores, at the end the output
//   warps 8..11        decode the cache, a thread a token: codes and scales of
//                      the next block of keys are loaded while this block's are
//                      converted to f16 and written as 128-byte-swizzled tiles
//   warp 12            one thread issues the MMAs: S = Q K^T (both operands in
//                      shared memory) and O += P V (P in tensor memory, V in
//                      shared memory with the head dim contiguous)
// The two tiles alternate: while one's scores are in the softmax the other's
// products run, and both use each decoded block, so the decode costs one pass
// per 256 rows.  Keys of all items are one list cut into equal shares
// (kv_work.cuh); items cut between CTAs are joined by the last to arrive, in CTA
// order.  Bound by the tensor pipe and, close to it, the issue slots of the
// softmax.
//
// Waits have clock budgets; when one runs out NVFP4_DEVICE_WAIT_TIMEOUT is set,
// later waits are passed over, MMAs in flight are drained and tensor memory is
// freed.
#include <cuda_bf16.h>

#include "formats.cuh"
#include "kv_work.cuh"
#include "launch_cache.cuh"
#include "mma_frag.cuh"

namespace nvfp4 {

namespace {

constexpr int kRowsTile = 128;             // query rows of an MMA tile
constexpr int kRows = 2 * kRowsTile;       // of an item
constexpr int kKeys = 128;                 // keys of a block
constexpr int kItemCost = 2;               // blocks that an item's start and end cost
constexpr int kThreads = 512;
constexpr float kRaise = 8.0f;             // log2 a score may pass the reference by
constexpr float kLift = 7.0f;              // p = 2^(s - m + kLift)
constexpr uint32_t kColS = 0, kColO = 256;  // scores and outputs, 128 columns a tile
// probabilities lie over the second half of the scores: that half is in
// registers when they are written, the first is read once more
constexpr uint32_t kColP = 64;

using Work = KvWork<kRows, kKeys, kItemCost>;

template <int D>
struct Cfg {
    static constexpr int kTile = kKeys * D * 2;                  // bytes of a K, V or Q tile
    static constexpr size_t kSmem = (size_t)6 * kTile + 1024;    // Q 2, K 2, V 2, alignment
    static constexpr int64_t kPart = (int64_t)(D + 2) * kRowsTile;  // floats of a partial tile
};

// K-major operand tile with 128-byte swizzle: 8-row atoms of 1024 bytes.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// N-major operand (rows of 64 consecutive N, one a K index): the next 64 of N
// lie a half tile further, the next 8 of K 1024 bytes further.
__device__ __forceinline__ uint64_t desc_n(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)((kKeys * 128) >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, FP32 accumulator, f16 operands, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_n_major)
{
    return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kRowsTile >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}
__device__ __forceinline__ void fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

// 32 columns of this warp's 32 rows, a thread a row (call tmem_wait_ld before use).
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(t));
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 64 columns of scores, those outside [first, last] as -inf.
__device__ __forceinline__ void load_scores(uint32_t t, uint32_t (&s)[64], bool edge, int32_t first,
                                            int32_t last)
{
    tmem_ld32(t, s);
    tmem_ld32(t + 32, s + 32);
    tmem_wait_ld();
    if (edge) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (i > last || i < first)
                s[i] = 0xFF800000u;  // -inf
    }
}

struct Barriers {
    uint64_t qfull[2];                // a tile's queries are in shared memory
    uint64_t kfull[2], kempty[2];     // decoded K blocks
    uint64_t vfull[2], vempty[2];
    uint64_t sfull[2];                // a tile's scores are in tensor memory
    uint64_t pfull[2];                // its probabilities are
    uint64_t ofull[2];                // an item's output of a tile is complete
    uint64_t drain;
};

// ---- warps 8..11: the cache to f16 ----------------------------------------------------
template <int D>
struct RawToken {
    uint4 k[D / 32], v[D / 32];
    uint32_t ks[D / 64], vs[D / 64];
};

template <int D>
__device__ __forceinline__ void load_token(RawToken<D>& x, const KvAttnArgs& a, int32_t page,
                                           int32_t tok, int h)
{
    if (page < 0) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            x.k[i] = x.v[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            x.ks[i] = x.vs[i] = 0u;
        return;
    }
    const int P = a.c.page_shift;
    const int32_t off = tok & ((1 << P) - 1);
    const uint8_t* p = a.c.pool + page * a.c.page_stride + h * kv_head_bytes(P, D);
    const uint4* k = reinterpret_cast<const uint4*>(p + off * (D / 2));
    const uint4* v = reinterpret_cast<const uint4*>(p + ((D / 2) << P) + off * (D / 2));
    const uint32_t* ks = reinterpret_cast<const uint32_t*>(p + (D << P) + off * (D / 16));
    const uint32_t* vs =
        reinterpret_cast<const uint32_t*>(p + (D << P) + ((D / 16) << P) + off * (D / 16));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        x.k[i] = __ldg(k + i);
        x.v[i] = __ldg(v + i);
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        x.ks[i] = __ldg(ks + i);
        x.vs[i] = __ldg(vs + i);
    }
}

// A token's row as f16 into a swizzled tile (row r of 128-byte rows, a half a
// 64 elements): eight 16-byte pieces of a row, piece c at c XOR (r mod 8).
template <int D>
__device__ __forceinline__ void store_token(uint8_t* tile, int r, const uint4 (&c)[D / 32],
                                            const uint32_t (&s)[D / 64])
{
    uint8_t* row = tile + r * 128;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {  // 32 elements: two blocks, four pieces
        const uint32_t two = e4m3x2_to_f16x2_bits(s[i / 2] >> (16 * (i % 2)));
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t sc = j < 2 ? f16x2_dup_lo(two) : f16x2_dup_hi(two);
            uint32_t f[4];
            e2m1x8_to_f16(w[j], f);
            const int piece = (i * 4 + j) & 7, half = (i * 4 + j) >> 3;
            *reinterpret_cast<uint4*>(row + half * (kKeys * 128) + ((piece ^ (r & 7)) << 4)) =
                make_uint4(f16x2_mul(f[0], sc), f16x2_mul(f[1], sc), f16x2_mul(f[2], sc),
                           f16x2_mul(f[3], sc));
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_tile_kernel(const KvAttnArgs a)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Barriers bars;
    __shared__ typename Work::Smem work_sm;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, last_s[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_flag = &abort_s;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sQ = smem_u32(smem), sK = sQ + 2 * C::kTile, sV = sK + 2 * C::kTile;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.qfull[i]), kRowsTile);
            mbar_init(smem_u32(&bars.kfull[i]), kKeys);
            mbar_init(smem_u32(&bars.kempty[i]), 1);
            mbar_init(smem_u32(&bars.vfull[i]), kKeys);
            mbar_init(smem_u32(&bars.vempty[i]), 1);
            mbar_init(smem_u32(&bars.sfull[i]), 1);
            mbar_init(smem_u32(&bars.pfull[i]), kRowsTile);
            mbar_init(smem_u32(&bars.ofull[i]), 1);
        }
        mbar_init(smem_u32(&bars.drain), 1);
        abort_s = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    kv_pdl_begin();

    KvShare sh;
    KvItem it;
    bool more = Work::start<kThreads>(a, work_sm, kItemCost + 1, sh, it);
    if (sh.lo >= sh.hi)
        return;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base_s)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base_s;

    if (warp < 8) {
        // ---- softmax: thread = row of tile st -------------------------------------------------
        const int st = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes
        const uint32_t tS = tmem + lanes + kColS + st * 128, tO = tmem + lanes + kColO + st * 128;
        const uint32_t qfull = smem_u32(&bars.qfull[st]), sfull = smem_u32(&bars.sfull[st]),
                       pfull = smem_u32(&bars.pfull[st]), ofull = smem_u32(&bars.ofull[st]);
        uint8_t* q_row = smem + st * C::kTile + r * 128;
        // a negative factor goes into the queries' signs, so that larger scores are
        // larger throughout
        const float vg = a.c.v_g[0], signed_qk = a.scale_log2 * a.c.k_g[0], qk = fabsf(signed_qk);
        const uint32_t flip = signed_qk < 0.f ? 0x80008000u : 0u;
        uint32_t blocks = 0, items = 0;  // this tile's so far
        for (; more; more = Work::next(a, sh, it)) {
            __syncwarp();
            const int row = it.row0 + st * kRowsTile + r;
            if (it.row0 + st * kRowsTile >= it.row1)
                continue;  // the item has no second tile
            const bool live = row < it.row1;
            const int tok = live ? row / a.group : 0;
            const int head = it.h * a.group + (live ? row - tok * a.group : 0);

            // the row's queries, scaled by a power of two, as f16
            float f;
            {
                uint2 w[D / 4];
                const uint2* src = reinterpret_cast<const uint2*>(
                    static_cast<const __nv_bfloat16*>(a.q) +
                    (int64_t)(it.q.base + tok) * a.q_stride + (int64_t)head * D);
                uint32_t top = 0;  // BF16 magnitudes order like their bits
#pragma unroll
                for (int i = 0; i < D / 4; ++i) {
                    w[i] = live ? __ldg(src + i) : make_uint2(0u, 0u);
                    top = __vmaxu2(top, __vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu));
                }
                top = max(top & 0xFFFFu, top >> 16);
                if (top > 0x7F80u)
                    top = 0x7F80u;  // NaN: any finite factor keeps it
                const int e = min(max(14 - ((int)(top >> 7) - 127), -100), 100);
                const float up = top ? __uint_as_float((uint32_t)(e + 127) << 23) : 1.0f;
                f = qk * (top ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f);
                // a factor of 0 (a zero scale) would make -inf of a masked score NaN
                f = f == 0.f ? 1e-38f : f;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = j & 1 ? w[2 * c + j / 2].y : w[2 * c + j / 2].x;
                        o[j] = pack_f16(__uint_as_float(x << 16) * up,
                                        __uint_as_float(x & 0xFFFF0000u) * up) ^
                               flip;
                    }
                    *reinterpret_cast<uint4*>(q_row + (c >> 3) * (kKeys * 128) +
                                              (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fence_before();  // the last item's reads of the output come before this item's products
            mbar_arrive(qfull);

            const int32_t pos = live ? it.q.seq - it.q.nq + tok : -1;
            float m = -INFINITY, l = 0.f;  // reference minus kLift, and the sum
            for (int32_t u = it.u0; u < it.u1; ++u, ++blocks) {
                mbar_wait(sfull, blocks & 1, abort_flag, a.status);
                fence_after();
                // columns [first, last] are seen
                const int32_t k0 = (it.first + u) * kKeys;
                const int32_t last = pos - k0;
                const int32_t first = a.window > 0 ? last - a.window + 1 : 0;
                const bool edge = last < kKeys - 1 || first > 0;
                // scores 64 at a time: both halves for the maximum, then the second
                // half (still in registers) and the first again for the exponentials
                uint32_t s[64];
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int h = 0; h < kKeys; h += 64) {
                    load_scores(tS + h, s, edge, first - h, last - h);
#pragma unroll
                    for (int i = 0; i < 64; i += 8)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            top[j] = fmaxf(top[j], fmaxf(__uint_as_float(s[i + 2 * j]),
                                                         __uint_as_float(s[i + 2 * j + 1])));
                }
                const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
                if (__any_sync(0xFFFFFFFFu, best > m + (kLift + kRaise))) {
                    const float now = fmaxf(m, best - kLift);
                    const float by = m == now ? 1.f : ex2(m - now);
                    m = now;
                    l *= by;
                    // earlier products are complete: this block's scores were issued
                    // after them, and their commit covers both
                    if (u > it.u0) {
#pragma unroll 1
                        for (int i = 0; i < D; i += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * by);
                            tmem_st32(tO + i, o);
                        }
                    }
                }
                // no key seen yet: every score is -inf, against any finite reference
                const float ref = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = kKeys - 64; h >= 0; h -= 64) {
                    if (h == 0)
                        load_scores(tS, s, edge, first, last);
                    uint32_t p16[32];
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        float p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            p[j] = ex2(fmaf(__uint_as_float(s[i + j]), f, -ref));
                            sum[j] += p[j];
                        }
                        p16[i / 2] = pack_f16(p[0], p[1]);
                        p16[i / 2 + 1] = pack_f16(p[2], p[3]);
                    }
                    tmem_st32(tS + kColP + h / 2, p16);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                fence_before();
                mbar_arrive(pfull);
            }

            // ---- the item's output ----------------------------------------------------------
            mbar_wait(ofull, items & 1, abort_flag, a.status);
            ++items;
            fence_after();
            const bool whole = it.u0 == 0 && it.u1 == it.n;
            const int64_t out_at = (int64_t)(it.q.base + tok) * a.out_stride + (int64_t)head * D;
            const int64_t lse_at = (int64_t)(it.q.base + tok) * (a.c.heads * a.group) + head;
            auto write32 = [&](int i, const float* o, float scale) {
                uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + out_at + i);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(o[j] * scale, o[j + 1] * scale);
                    const __nv_bfloat162 y = __floats2bfloat162_rn(o[j + 2] * scale, o[j + 3] * scale);
                    dst[j / 4] = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                            *reinterpret_cast<const uint32_t*>(&y));
                }
            };
            auto write_lse = [&](float mt, float lt) {
                if (a.lse != nullptr)
                    a.lse[lse_at] = lt == 0.f ? -INFINITY : 0.6931471805599453f * (mt + log2f(lt));
            };
            float* part = a.part + (4 * blockIdx.x + 2 * (it.u0 == 0 ? 1 : 0) + st) * C::kPart + r;
            const float scale = l == 0.f ? 0.f : vg / l;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld32(tO + i, o);
                tmem_wait_ld();
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = __uint_as_float(o[j]);
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        part[(i + j) * kRowsTile] = x[j];
                } else if (live) {
                    write32(i, x, scale);
                }
            }
            if (whole) {
                if (live)
                    write_lse(m, l);
                continue;
            }
            part[D * kRowsTile] = m;
            part[(D + 1) * kRowsTile] = l;
            // the last CTA of the item to arrive joins the parts in CTA order
            const int ca = Work::first_cta(sh, it), cb = Work::last_cta(sh, it);
            __threadfence();
            asm volatile("bar.sync %0, 128;" ::"r"(1 + st) : "memory");
            if (r == 0) {
                const unsigned seen = atomicAdd(a.count + 2 * ca + st, 1u);
                last_s[st] = seen == (unsigned)(cb - ca);
                if (last_s[st])
                    a.count[2 * ca + st] = 0u;
                __threadfence();
            }
            asm volatile("bar.sync %0, 128;" ::"r"(1 + st) : "memory");
            if (!last_s[st] || !live)
                continue;
            auto part_of = [&](int c) {
                return a.part + (4 * c + 2 * (c == ca ? 1 : 0) + st) * C::kPart + r;
            };
            float mt = -INFINITY, lt = 0.f;
            for (int c = ca; c <= cb; ++c)
                mt = fmaxf(mt, __ldcg(part_of(c) + D * kRowsTile));
            for (int c = ca; c <= cb; ++c) {
                const float mc = __ldcg(part_of(c) + D * kRowsTile);
                lt += __ldcg(part_of(c) + (D + 1) * kRowsTile) * (mc == mt ? 1.f : ex2(mc - mt));
            }
            const float all = lt == 0.f ? 0.f : vg / lt;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = 0.f;
                for (int c = ca; c <= cb; ++c) {
                    const float* pc = part_of(c);
                    const float mc = __ldcg(pc + D * kRowsTile);
                    const float by = mc == mt ? 1.f : ex2(mc - mt);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        x[j] = fmaf(__ldcg(pc + (i + j) * kRowsTile), by, x[j]);
                }
                write32(i, x, all);
            }
            write_lse(mt, lt);
        }
    } else if (warp < 12) {
        // ---- decode: thread = token of a block -------------------------------------------------
        const int r = tid & 127;
        bool bad = false;
        auto page_of = [&](const KvItem& x, int32_t u) {
            const int32_t tok = (x.first + u) * kKeys + r, b = tok >> a.c.page_shift;
            if (tok >= x.q.seq || b >= a.max_blocks)
                return -1;
            const int32_t page = a.table[x.r * a.table_stride + b];
            if (page >= 0 && page < a.c.num_pages)
                return page;
            bad = true;
            return -1;
        };
        RawToken<D> x;
        int32_t u = 0;
        KvItem nx = it;
        int32_t npage = -1;
        // the block after (it, u): its token is loaded a block ahead, its page two
        auto advance = [&](KvItem& w, int32_t& v) {
            if (v + 1 < w.u1) {
                ++v;
                return true;
            }
            if (!Work::next(a, sh, w))
                return false;
            v = w.u0;
            return true;
        };
        uint32_t n = 0;
        bool have_next = more;
        int32_t nu = 0;
        if (more) {
            u = it.u0;
            load_token<D>(x, a, page_of(it, u), (it.first + u) * kKeys + r, it.h);
            nu = u;
            have_next = advance(nx, nu);
            npage = have_next ? page_of(nx, nu) : -1;
        }
        while (more) {
            const uint32_t b = n & 1, turn = n >> 1;
            if (n >= 2)
                mbar_wait(smem_u32(&bars.kempty[b]), (turn - 1) & 1, abort_flag, a.status);
            store_token<D>(smem + (2 + b) * C::kTile, r, x.k, x.ks);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(smem_u32(&bars.kfull[b]));
            if (n >= 2)
                mbar_wait(smem_u32(&bars.vempty[b]), (turn - 1) & 1, abort_flag, a.status);
            store_token<D>(smem + (4 + b) * C::kTile, r, x.v, x.vs);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(smem_u32(&bars.vfull[b]));
            ++n;
            more = have_next;
            if (more) {
                load_token<D>(x, a, npage, (nx.first + nu) * kKeys + r, nx.h);
                have_next = advance(nx, nu);
                npage = have_next ? page_of(nx, nu) : -1;
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
            atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
    } else {
        // ---- warp 12: the MMAs --------------------------------------------------------------------
        if (warp == 12 && lane == 0) {
            constexpr uint32_t id_s = idesc(kKeys, false), id_o = idesc(D, true);
            uint32_t n = 0, items = 0, items1 = 0, blocks1 = 0;  // blocks and items (tile 1: its own)
            auto scores = [&](int st, uint32_t b) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k >> 2) * (kKeys * 128) + (k & 3) * 32;
                    mma_ss(tmem + kColS + st * 128, desc_k(sQ + st * C::kTile + at),
                           desc_k(sK + b * C::kTile + at), id_s, k > 0);
                }
                commit(smem_u32(&bars.sfull[st]));
            };
            auto outputs = [&](int st, uint32_t b, bool acc) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(tmem + kColO + st * 128, tmem + kColS + kColP + st * 128 + k * 8,
                           desc_n(sV + b * C::kTile + k * 2048), id_o, acc || k > 0);
            };
            bool ok = true;
            for (; more && ok; more = Work::next(a, sh, it)) {
                const int tiles = it.row1 - it.row0 > kRowsTile ? 2 : 1;
                const int32_t count = it.u1 - it.u0;
                for (int st = 0; st < tiles && ok; ++st)
                    ok = mbar_wait(smem_u32(&bars.qfull[st]), (st ? items1 : items) & 1, abort_flag,
                                   a.status);
                ok = ok && mbar_wait(smem_u32(&bars.kfull[n & 1]), (n >> 1) & 1, abort_flag, a.status);
                if (!ok)
                    break;
                fence_after();
                for (int st = 0; st < tiles; ++st)
                    scores(st, n & 1);
                commit(smem_u32(&bars.kempty[n & 1]));
                for (int32_t j = 0; j < count && ok; ++j, ++n) {
                    const uint32_t b = n & 1, nb = (n + 1) & 1;
                    ok = mbar_wait(smem_u32(&bars.vfull[b]), (n >> 1) & 1, abort_flag, a.status);
                    for (int st = 0; st < tiles && ok; ++st) {
                        ok = mbar_wait(smem_u32(&bars.pfull[st]), (st ? blocks1 : n) & 1, abort_flag,
                                       a.status);
                        if (!ok)
                            break;
                        fence_after();
                        outputs(st, b, j > 0);
                        if (st == tiles - 1)
                            commit(smem_u32(&bars.vempty[b]));
                        if (j + 1 < count) {
                            if (st == 0)
                                ok = mbar_wait(smem_u32(&bars.kfull[nb]), ((n + 1) >> 1) & 1,
                                               abort_flag, a.status);
                            if (!ok)
                                break;
                            fence_after();
                            scores(st, nb);
                            if (st == tiles - 1)
                                commit(smem_u32(&bars.kempty[nb]));
                        } else {
                            commit(smem_u32(&bars.ofull[st]));
                        }
                    }
                    if (tiles == 2)
                        ++blocks1;
                }
                ++items;
                if (tiles == 2)
                    ++items1;
            }
            // what was issued must be complete before tensor memory is freed
            commit(smem_u32(&bars.drain));
            const long long t0 = clock64();
            while (!mbar_test(smem_u32(&bars.drain), 0) && clock64() - t0 < kKvWaitBudget) {
            }
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

template <int D>
cudaError_t launch(const KvAttnArgs& a, cudaStream_t stream, bool pdl)
{
    const int dev = current_device();
    const cudaError_t e = ensure_smem_limit(kv_tile_kernel<D>, Cfg<D>::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    return kv_launch(kv_tile_kernel<D>, device_sm_count(dev), kThreads, Cfg<D>::kSmem, stream, pdl, a);
}

}  // namespace

// Counters (one a CTA and tile), then four partial tiles a CTA.
int64_t kv_tile_workspace_bytes(int dim)
{
    const int64_t ctas = device_sm_count(current_device());
    return kKvCountBytes + ctas * 4 * (dim + 2) * kRowsTile * (int64_t)sizeof(float);
}

cudaError_t launch_kv_tile(const KvAttnArgs& args, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl)
{
    KvAttnArgs a = args;
    a.count = nullptr;
    a.part = nullptr;
    if (workspace_bytes >= kv_tile_workspace_bytes(a.c.dim)) {
        a.count = static_cast<unsigned*>(workspace);
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kKvCountBytes);
    }
    return a.c.dim == 128 ? launch<128>(a, stream, pdl) : launch<64>(a, stream, pdl);
}

}  // namespace nvfp4

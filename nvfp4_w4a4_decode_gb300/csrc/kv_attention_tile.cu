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
// 128-row tiles, 128 keys at a time:
//   warps 0..3, 4..7   softmax of tile 0, 1, a thread a row: the queries into
//                      shared memory, scores out of tensor memory, probabilities
//                      back into it over the scores, at the end the output.  The
//                      exponentials of 64 scores are taken against the reference
//                      at hand, with their maximum as a by-product; only where
//                      that passes the reference by 2^8 is it raised, by a power of
//                      two, what was accumulated rescaled (exactly, so that a
//                      probability is rounded to f16 once) and the 64 scores done again
//   warps 8..11        decode the cache, 32 tokens each: codes and scales of
//                      the next block of keys are loaded while this block's are
//                      converted to f16 and written as 128-byte-swizzled tiles
//   warp 12            one lane issues the MMAs: S = Q K^T (both operands in
//                      shared memory) and O += P V (P in tensor memory, V in
//                      shared memory with the head dim contiguous)
// The two tiles alternate: while one's scores are in the softmax the other's
// products run, and both use each decoded block, so the decode costs one pass
// per 256 rows.  Keys of all items are one list cut into equal shares
// (kv_work.cuh); items cut between CTAs are joined by the last to arrive, in CTA
// order.
//
// What bounds it: the chain scores -> exponentials -> probabilities of a tile
// (about 2600 cycles a block beside the 1024 of its products, of which the other
// tile's run meanwhile) and shared memory, which the products of both tiles and the
// decode's stores read and write 192 KB of a block, 1536 of its 2048 tensor
// cycles.  2048 queries of 32 heads on 32049 keys: 768 us, 1.36 PFLOP/s; four prompts of
// 2185..3879 tokens and 64 heads: 723 us, 0.94 PFLOP/s (an item's queries, first
// block, masked last block and output add about 9 us to its keys).
//
// Waits have clock budgets; when one runs out NVFP4_DEVICE_WAIT_TIMEOUT is set,
// later waits are passed over, MMAs in flight are drained and tensor memory is
// freed.
#include <cuda_bf16.h>

#include <type_traits>

#include "formats.cuh"
#include "kv_work.cuh"
#include "launch_cache.cuh"
#include "mma_frag.cuh"

namespace nvfp4 {

namespace {

constexpr int kRowsTile = 128;             // query rows of an MMA tile
constexpr int kRows = 2 * kRowsTile;       // of an item
constexpr int kKeys = 128;                 // keys of a block
// Blocks that an item's start and end cost (us for four prompts of 2185..3879 tokens of 64
// heads / six of 32 heads / 16 requests of 3..6 tokens on a window of 1024: 3 704 392 28.8,
// 4 724 384 27.1, 5 716 401 27.0, 7 753 413 27.8).
constexpr int kItemCost = 5;
constexpr int kDecodeWarp = 8, kMmaWarp = 12;
constexpr int kDecodeRows = kKeys / (kMmaWarp - kDecodeWarp);  // tokens a decoding warp
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kSpan = 64;                  // keys between two looks at the reference
constexpr float kRaise = 8.0f;             // log2 a score may pass the reference by
constexpr float kLift = 7.0f;              // p = 2^(s - m + kLift)
constexpr uint32_t kColS = 0, kColO = 256;  // scores and outputs, 128 columns a tile

using Work = KvWork<kRows, kKeys, kItemCost, 2>;

template <int D>
struct Cfg {
    static constexpr int kTile = kKeys * D * 2;                  // bytes of a K, V or Q tile
    static constexpr int kStage = kRows * 64;                    // 32 outputs a row on their way
    static constexpr size_t kSmem = (size_t)6 * kTile + kStage + 1024;  // Q 2, K 2, V 2, alignment
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

// The MMA warp runs its loop with all lanes, so that descriptors stay in uniform
// registers (from a branch of one lane each MMA took 80 cycles to issue, more
// than it takes to run); `one` is set in the lane that issues.
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       bool acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(one)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       bool acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(one)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
                     "r"(bar), "r"(one)
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

// 16 or 32 columns of this warp's 32 rows, a thread a row; complete on return.
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
        "}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%"
        "21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
        "}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
        "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
        "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
        "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
        "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
        "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Packed pairs of FP32 operations.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(x), "l"(y), "l"(z));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
    return v;
}

// One arrival for the warp.
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
}

// Barrier of a tile's softmax threads.
__device__ __forceinline__ void tile_sync(int st)
{
    asm volatile("bar.sync %0, %1;" ::"r"(1 + st), "n"(kRowsTile) : "memory");
}

// Byte of 16-byte piece `piece` (8 elements) of row r in a swizzled tile.
__device__ __forceinline__ int piece_at(int r, int piece)
{
    return (piece >> 3) * (kKeys * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
}

struct Barriers {
    uint64_t qfull[2];                // a tile's queries are in shared memory (an arrival a
                                      // warp, here and below)
    uint64_t kfull[2], kempty[2];     // decoded K blocks
    uint64_t vfull[2], vempty[2];
    uint64_t sfull[2];                // a tile's scores are in tensor memory
    uint64_t pfull[2];                // its probabilities are
    uint64_t ofull[2];                // an item's output of a tile is complete
    uint64_t drain;
};

// ---- warps 8..11: the cache to f16 ----------------------------------------------------
// 32 tokens of a block a warp: a lane takes 32 elements (16 bytes of codes, two
// scales) of every kRpi-th row, neighbouring lanes neighbouring bytes.
template <int D>
struct Raw {
    static constexpr int kLanes = D / 32;        // lanes a row
    static constexpr int kRpi = 32 / kLanes;     // rows at a time
    static constexpr int kIters = kDecodeRows / kRpi;
    uint4 c[kIters];
    uint32_t s[kIters];
};

// The K or V rows of a warp's tokens in [key0, seq) (key0 is 0 without a window),
// zeros for others; page[i] holds the i-th 16 of them (-1: nothing there).
template <int D, bool WINDOW>
__device__ __forceinline__ void load_rows(Raw<D>& x, const KvAttnArgs& a,
                                          const int32_t (&page)[kDecodeRows / 16], int32_t tok0,
                                          int32_t key0, int32_t seq, int h, bool is_v)
{
    using X = Raw<D>;
    const int P = a.c.page_shift, lane = threadIdx.x & 31;
    const int64_t part = h * kv_head_bytes(P, D);
    const int64_t codes = part + (is_v ? (D / 2) << P : 0) + lane * 16;
    const int64_t scales = part + (D << P) + (is_v ? (D / 16) << P : 0) + lane * 2;
#pragma unroll
    for (int i = 0; i < X::kIters; ++i) {
        const int row0 = i * X::kRpi;  // rows row0 .. row0 + kRpi - 1 lie in one page
        const int32_t pg = page[row0 / 16], off = (tok0 + row0) & ((1 << P) - 1);
        x.c[i] = make_uint4(0u, 0u, 0u, 0u);
        x.s[i] = 0u;
        const int32_t tok = tok0 + row0 + lane / X::kLanes;
        if (pg >= 0 && tok < seq && (!WINDOW || tok >= key0)) {
            const uint8_t* p = a.c.pool + pg * a.c.page_stride;
            x.c[i] = __ldg(reinterpret_cast<const uint4*>(p + codes + off * (D / 2)));
            x.s[i] = __ldg(reinterpret_cast<const uint16_t*>(p + scales + off * (D / 16)));
        }
    }
}

// The same rows as f16 into a swizzled tile (rows row0 ..).  Lanes of the second
// half of a row write their pieces in another order, so that a store's lanes fall
// on different banks.
template <int D>
__device__ __forceinline__ void store_rows(uint8_t* tile, int row0, const Raw<D>& x)
{
    using X = Raw<D>;
    const int lane = threadIdx.x & 31, t = lane % X::kLanes;
    const bool turn = t >= 2;
#pragma unroll
    for (int i = 0; i < X::kIters; ++i) {
        const int r = row0 + i * X::kRpi + lane / X::kLanes;
        const uint32_t two = e4m3x2_to_f16x2_bits(x.s[i]);
        const uint32_t lo = f16x2_dup_lo(two), hi = f16x2_dup_hi(two);
        const uint32_t w[4] = {turn ? x.c[i].z : x.c[i].x, turn ? x.c[i].w : x.c[i].y,
                               turn ? x.c[i].x : x.c[i].z, turn ? x.c[i].y : x.c[i].w};
        const uint32_t sc[2] = {turn ? hi : lo, turn ? lo : hi};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t f[4];
            e2m1x8_to_f16(w[j], f);
            *reinterpret_cast<uint4*>(tile + piece_at(r, 4 * t + (turn ? j ^ 2 : j))) =
                make_uint4(f16x2_mul(f[0], sc[j / 2]), f16x2_mul(f[1], sc[j / 2]),
                           f16x2_mul(f[2], sc[j / 2]), f16x2_mul(f[3], sc[j / 2]));
        }
    }
}

// A kernel of its own without a window: with the window's first key in the decoding
// warps of the one kernel four prompts took 735 us instead of 716, a chunk 769 instead of 762.
template <int D, bool WINDOW>
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
            mbar_init(smem_u32(&bars.qfull[i]), kRowsTile / 32);
            mbar_init(smem_u32(&bars.kfull[i]), kKeys / kDecodeRows);
            mbar_init(smem_u32(&bars.kempty[i]), 1);
            mbar_init(smem_u32(&bars.vfull[i]), kKeys / kDecodeRows);
            mbar_init(smem_u32(&bars.vempty[i]), 1);
            mbar_init(smem_u32(&bars.sfull[i]), 1);
            mbar_init(smem_u32(&bars.pfull[i]), kRowsTile / 32);
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
    constexpr int kDecodeThreads = 32 * (kMmaWarp - kDecodeWarp);
    const bool decodes = warp >= kDecodeWarp && warp < kMmaWarp;
    if (sh.lo >= sh.hi) {
        if (a.all_rows && decodes)
            kv_write_other_rows(a, tid - 32 * kDecodeWarp, kDecodeThreads);
        return;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base_s)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base_s;

    if (warp < kDecodeWarp) {
        // ---- softmax: thread = row of tile st -------------------------------------------------
        const int st = warp >> 2, r = tid & 127, wrow = r & ~31;  // the warp's first row
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // its 32 lanes
        const uint32_t tS = tmem + lanes + kColS + st * 128, tO = tmem + lanes + kColO + st * 128;
        const uint32_t qfull = smem_u32(&bars.qfull[st]), sfull = smem_u32(&bars.sfull[st]),
                       pfull = smem_u32(&bars.pfull[st]), ofull = smem_u32(&bars.ofull[st]);
        uint8_t* tile = smem + st * C::kTile;                    // the queries
        uint8_t* staged = smem + 6 * C::kTile + warp * (32 * 64);  // the warp's outputs
        // rows move in pieces of 16 bytes, a lane each, where their alignment allows it
        // (halves of 8 bytes: four prompts 726 us instead of 701).  What runs once an item
        // is kept in short loops: unrolled to 20 KB, the queries' part spent 18000 cycles
        // an item on fetching its instructions.
        constexpr int kPieces = D / 8;
        const bool q_wide = ((uintptr_t)a.q | (uintptr_t)(2 * a.q_stride)) % 16 == 0;
        const bool out_wide = ((uintptr_t)a.out | (uintptr_t)(2 * a.out_stride)) % 16 == 0;
        // a negative factor goes into the queries' signs, so that larger scores are
        // larger throughout
        const float vg = a.c.v_g[0], signed_qk = a.scale_log2 * a.c.k_g[0], qk = fabsf(signed_qk);
        const uint32_t flip = signed_qk < 0.f ? 0x80008000u : 0u;
        uint32_t blocks = 0, items = 0;  // this tile's so far
        // a thread's row of an item's tile (past the item's end: its last row again, which
        // keeps the thread off the masked path; never written)
        struct Row {
            bool live;
            int tok, head, rows;  // token and head; rows of the warp's 32 in the item
        };
        auto row_of = [&](const KvItem& x) {
            const int row = x.row0 + st * kRowsTile + r;
            Row y;
            y.live = row < x.row1;
            const int at = min(row, x.row1 - 1);
            y.tok = kv_token(a, at);
            y.head = x.h * a.group + at - y.tok * a.group;
            y.rows = min(x.row1 - (row - lane), 32);
            return y;
        };
        // on to the next item that has this tile
        auto advance = [&](KvItem& x) {
            do {
                __syncwarp();
                if (!Work::next(a, sh, x))
                    return false;
            } while (x.row0 + st * kRowsTile >= x.row1);
            return true;
        };
        // the warp's 32 rows of queries as they are into the tile, a row's lanes reading
        // neighbouring bytes
        auto fetch = [&](const KvItem& x) {
            const Row y = row_of(x);
            const int64_t at = (x.q.base + y.tok) * a.q_stride + (int64_t)y.head * D;
#pragma unroll 2
            for (int i = 0; i < 32; i += 32 / kPieces) {
                const int z = i + lane / kPieces, c = lane % kPieces;
                const int64_t from = __shfl_sync(0xFFFFFFFFu, at, z);
                const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + from + 8 * c;
                const uint32_t dst = smem_u32(tile + piece_at(wrow + z, c));
                if (q_wide) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                                 "r"(z < y.rows ? 16u : 0u)
                                 : "memory");
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + 8 * k),
                                     "l"(src + 4 * k), "r"(z < y.rows ? 8u : 0u)
                                     : "memory");
                }
            }
        };
        // then a thread a row scales its own by a power of two and leaves it as f16;
        // returns the factor of the row's scores
        auto convert = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            uint32_t top = 0;  // BF16 magnitudes order like their bits
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(tile + piece_at(r, c));
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                             __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
            }
            top = max(top & 0xFFFFu, top >> 16);
            top = min(top, 0x7F80u);  // NaN: any finite factor keeps it
            const int e = min(max(14 - ((int)(top >> 7) - 127), -100), 100);
            const float up = top ? __uint_as_float((uint32_t)(e + 127) << 23) : 1.0f;
            const float f = qk * (top ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f);
#pragma unroll 2
            for (int c = 0; c < D / 8; ++c) {
                uint4* place = reinterpret_cast<uint4*>(tile + piece_at(r, c));
                const uint4 x = *place;
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = pack_f16(__uint_as_float(w[j] << 16) * up,
                                    __uint_as_float(w[j] & 0xFFFF0000u) * up) ^ flip;
                *place = make_uint4(o[0], o[1], o[2], o[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            warp_arrive(qfull);
            // a factor of 0 (a zero scale) would make -inf of a masked score NaN
            return f == 0.f ? 1e-38f : f;
        };

        if (more && it.row0 + st * kRowsTile >= it.row1)
            more = advance(it);
        float f = 0.f, next_f = 0.f;
        if (more) {
            fetch(it);
            f = convert();
        }
        KvItem nx;
        for (; more; it = nx, f = next_f) {
            const Row mine = row_of(it);
            const bool live = mine.live;
            const int tok = mine.tok, head = mine.head;

            // the next item, while this one's first scores are made: its query rows to L2
            nx = it;
            more = advance(nx);
            if (more) {
                const Row y = row_of(nx);
                if (y.live) {
                    const char* q = reinterpret_cast<const char*>(
                        static_cast<const __nv_bfloat16*>(a.q) +
                        (nx.q.base + y.tok) * a.q_stride + (int64_t)y.head * D);
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
                    if constexpr (D > 64)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 128));
                }
            }

            const int32_t pos = it.q.seq - it.q.nq + tok;
            float m = -INFINITY, l = 0.f;  // reference minus kLift, and the sum
            const uint64_t f2 = pair(f, f);
            for (int32_t u = it.u0; u < it.u1; ++u, ++blocks) {
                // columns [first, last] are seen
                const int32_t last = pos - (it.first + u) * kKeys;
                const int32_t first = a.window > 0 ? last - a.window + 1 : 0;
                const bool edge = last < kKeys - 1 || first > 0;
                mbar_wait(sfull, blocks & 1, abort_flag, a.status);
                __syncwarp();  // lanes poll each for itself; the loads below want a whole warp
                fence_after();
                // scores outside [first, last] of the 32 from c on become -inf
                auto hide = [&](int c, uint32_t* s) {
                    int lo = first - c, hi = last - c + 1;
                    asm volatile("" : "+r"(lo), "+r"(hi));  // not computed where it is not needed
                    lo = min(max(lo, 0), 32);
                    hi = min(max(hi, 0), 32);
                    const uint32_t seen = __funnelshift_lc(0u, 0xFFFFFFFFu, lo) &
                                          ~__funnelshift_lc(0u, 0xFFFFFFFFu, hi);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        s[i] = seen >> i & 1 ? s[i] : 0xFF800000u;
                };
                if (mine.rows > 0 && u == it.u0) {  // the first reference: the block's largest score
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t s[32];
                        tmem_ld32(tS + c, s);
                        if (edge)
                            hide(c, s);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                top[j] = fmaxf(top[j], fmaxf(__uint_as_float(s[i + 2 * j]),
                                                             __uint_as_float(s[i + 2 * j + 1])));
                    }
                    m = fmaxf(top[0], top[1]);
                    m = m == -INFINITY ? m : m * f - kLift;
                }
                // kSpan keys at a time (with a look at the reference every 32 a chunk of
                // 2048 rows on 30000 keys took 858 us, every 64 776, every 128 784);
                // blocks that every row of the warp sees whole skip the masks
                auto exponentials = [&](auto masked) {
#pragma unroll
                    for (int h = 0; h < kKeys; h += kSpan) {
                        uint32_t p16[kSpan / 2];
                        float sum;
                        // usually once; a second time when the reference had to be raised
#pragma unroll 1
                        for (int pass = 0;; ++pass) {
                            // no key seen yet: every score is -inf, against any finite reference
                            const float ref = m == -INFINITY ? 0.f : m;
                            const uint64_t neg = pair(-ref, -ref);
                            float top[2] = {-INFINITY, -INFINITY};
                            uint64_t sums[2] = {0ull, 0ull};
#pragma unroll
                            for (int c = 0; c < kSpan; c += 32) {
                                uint32_t s[32];
                                tmem_ld32(tS + h + c, s);
                                if constexpr (masked)
                                    hide(h + c, s);
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    const uint64_t x = fma2(pair(__uint_as_float(s[i]),
                                                                 __uint_as_float(s[i + 1])), f2, neg);
                                    float p0, p1;
                                    unpair(x, p0, p1);
                                    top[(i >> 1) & 1] = fmaxf(top[(i >> 1) & 1], fmaxf(p0, p1));
                                    p0 = ex2(p0);
                                    p1 = ex2(p1);
                                    sums[(i >> 1) & 1] = add2(sums[(i >> 1) & 1], pair(p0, p1));
                                    p16[(c + i) / 2] = pack_f16(p0, p1);
                                }
                            }
                            float x0, x1;
                            unpair(add2(sums[0], sums[1]), x0, x1);
                            sum = x0 + x1;
                            const float best = fmaxf(top[0], top[1]);  // against ref
                            // (a row that has seen no key takes its first reference too)
                            const bool raise =
                                best > kLift + kRaise || (m == -INFINITY && best > -INFINITY);
                            if (pass == 1 || !__any_sync(0xFFFFFFFFu, raise))
                                break;
                            // The first reference as it comes; then a whole number of powers of
                            // two at a time, which takes nothing from probabilities already f16.
                            float by = 0.f;
                            if (m == -INFINITY) {
                                m = best - kLift;
                            } else {
                                const float steps = floorf(fmaxf(best - kLift, 0.f));
                                m += steps;
                                if (steps < 127.f)
                                    by = __int_as_float((127 - (int)steps) << 23);
                            }
                            l *= by;
                            // The output so far (its products are complete: this block's scores
                            // were issued after them, and their commit covers both) and the
                            // probabilities of the first half, over scores already used.
                            tmem_wait_st();
                            if (u > it.u0) {
#pragma unroll 1
                                for (int i = 0; i < D; i += 16) {
                                    uint32_t o[16];
                                    tmem_ld16(tO + i, o);
#pragma unroll
                                    for (int j = 0; j < 16; ++j)
                                        o[j] = __float_as_uint(__uint_as_float(o[j]) * by);
                                    tmem_st16(tO + i, o);
                                }
                            }
                            const uint32_t by16 = pack_f16(by, by);
#pragma unroll 1
                            for (int i = 0; i < h / 2; i += 16) {
                                uint32_t o[16];
                                tmem_ld16(tS + i, o);
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    o[j] = f16x2_mul(o[j], by16);
                                tmem_st16(tS + i, o);
                            }
                        }
                        l += sum;
#pragma unroll
                        for (int i = 0; i < kSpan / 2; i += 32)
                            tmem_st32(tS + h / 2 + i, p16 + i);
                    }
                };
                if (mine.rows <= 0) {
                    // no row of the warp is in the item: whatever the products take for it
                    // stays in rows that are never written
                } else if (__any_sync(0xFFFFFFFFu, edge))
                    exponentials(std::true_type{});
                else
                    exponentials(std::false_type{});
                tmem_wait_st();
                fence_before();
                warp_arrive(pfull);
            }

            // the next item's queries, during the last products: its first scores are made
            // during the output below (its own products wait for its probabilities)
            if (more) {
                fetch(nx);
                next_f = convert();
            }

            // ---- the item's output ----------------------------------------------------------
            mbar_wait(ofull, items & 1, abort_flag, a.status);
            __syncwarp();
            ++items;
            fence_after();
            const bool whole = it.u0 == 0 && it.u1 == it.n;
            auto write_lse = [&](float mt, float lt) {
                if (a.lse != nullptr && live)
                    a.lse[(int64_t)(it.q.base + tok) * (a.c.heads * a.group) + head] =
                        lt == 0.f ? -INFINITY : 0.6931471805599453f * (mt + log2f(lt));
            };
            // 32 outputs of each of the warp's rows, over shared memory: a row's lanes write
            // neighbouring bytes
            const int64_t row_out = (it.q.base + tok) * a.out_stride + (int64_t)head * D;
            auto write = [&](int i, const float* o, float scale) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(
                            o[8 * j + 2 * k] * scale, o[8 * j + 2 * k + 1] * scale);
                        v[k] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                    *reinterpret_cast<uint4*>(staged + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                }
                __syncwarp();
                const int c = lane & 3;
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    const int x = j + (lane >> 2);
                    const int64_t to = __shfl_sync(0xFFFFFFFFu, row_out, x);
                    const uint4 v =
                        *reinterpret_cast<const uint4*>(staged + x * 64 + ((c ^ (x >> 1 & 3)) << 4));
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + to + i + 8 * c;
                    if (x < mine.rows) {
                        if (out_wide) {
                            *reinterpret_cast<uint4*>(dst) = v;
                        } else {
                            reinterpret_cast<uint2*>(dst)[0] = make_uint2(v.x, v.y);
                            reinterpret_cast<uint2*>(dst)[1] = make_uint2(v.z, v.w);
                        }
                    }
                }
            };
            // a partial tile: [D] columns of 128 rows, then references, then sums
            float* part = a.part + (4 * blockIdx.x + 2 * (it.u0 == 0 ? 1 : 0) + st) * C::kPart + r;
            const float scale = l == 0.f ? 0.f : vg / l;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld32(tO + i, o);
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] = __uint_as_float(o[j]);
                if (whole) {
                    write(i, x, scale);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        part[(i + j) * kRowsTile] = x[j];
                }
            }
            if (whole) {
                write_lse(m, l);
                continue;
            }
            part[D * kRowsTile] = m;
            part[(D + 1) * kRowsTile] = l;
            // the last CTA of the item to arrive joins the parts in CTA order
            const int ca = Work::first_cta(sh, it), cb = Work::last_cta(sh, it);
            __threadfence();
            tile_sync(st);
            if (r == 0) {
                const unsigned seen = atomicAdd(a.count + 2 * ca + st, 1u);
                last_s[st] = seen == (unsigned)(cb - ca);
                if (last_s[st])
                    a.count[2 * ca + st] = 0u;
                __threadfence();
            }
            tile_sync(st);
            if (!last_s[st])
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
                write(i, x, all);
            }
            write_lse(mt, lt);
        }
    } else if (warp < kMmaWarp) {
        // ---- decode: 32 tokens of a block a warp -------------------------------------------------
        const int row0 = kDecodeRows * (warp - kDecodeWarp);
        bool bad = false;
        // a block's rows are loaded a block ahead, their page two
        Raw<D> k, v;
        int32_t page[kDecodeRows / 16];
        auto first_key = [&](const KvItem& y) { return WINDOW ? Work::first_key(a, y) : 0; };
        auto look_up = [&](const KvItem& y, int32_t u) {
            const int32_t key0 = first_key(y);
#pragma unroll
            for (int i = 0; i < kDecodeRows / 16; ++i) {
                const int32_t tok = (y.first + u) * kKeys + row0 + 16 * i, b = tok >> a.c.page_shift;
                page[i] = -1;
                if (tok < y.q.seq && b < a.max_blocks && (!WINDOW || tok + 15 >= key0)) {
                    page[i] = a.table[y.r * a.table_stride + b];
                    if (page[i] < 0 || page[i] >= a.c.num_pages) {
                        bad = true;
                        page[i] = -1;
                    }
                }
            }
        };
        auto load = [&](const KvItem& y, int32_t u) {
            const int32_t tok0 = (y.first + u) * kKeys + row0, key0 = first_key(y);
            load_rows<D, WINDOW>(k, a, page, tok0, key0, y.q.seq, y.h, false);
            load_rows<D, WINDOW>(v, a, page, tok0, key0, y.q.seq, y.h, true);
        };
        int32_t u = 0;
        auto advance = [&]() {  // to the block after u of `it`
            if (u + 1 < it.u1) {
                ++u;
                return true;
            }
            if (!Work::next(a, sh, it))
                return false;
            u = it.u0;
            return true;
        };
        bool have_next = more;
        if (more) {
            u = it.u0;
            look_up(it, u);
            load(it, u);
            have_next = advance();
            if (have_next)
                look_up(it, u);
        }
        for (uint32_t n = 0; more; ++n) {
            const uint32_t b = n & 1, turn = n >> 1;
            if (n >= 2)
                mbar_wait(smem_u32(&bars.kempty[b]), (turn - 1) & 1, abort_flag, a.status);
            store_rows<D>(smem + (2 + b) * C::kTile, row0, k);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            warp_arrive(smem_u32(&bars.kfull[b]));
            if (n >= 2)
                mbar_wait(smem_u32(&bars.vempty[b]), (turn - 1) & 1, abort_flag, a.status);
            store_rows<D>(smem + (4 + b) * C::kTile, row0, v);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            warp_arrive(smem_u32(&bars.vfull[b]));
            more = have_next;
            if (more) {
                load(it, u);
                have_next = advance();
                if (have_next)
                    look_up(it, u);
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
            atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
        if (a.all_rows)
            kv_write_other_rows(a, tid - 32 * kDecodeWarp, kDecodeThreads);
    } else {
        // ---- warp 12: the MMAs --------------------------------------------------------------------
        uint32_t one;
        asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
        constexpr uint32_t id_s = idesc(kKeys, false), id_o = idesc(D, true);
        const uint64_t q_desc = desc_k(sQ), k_desc = desc_k(sK), v_desc = desc_n(sV);
        constexpr uint32_t kTileStep = C::kTile >> 4;  // of a descriptor's address
        uint32_t n = 0, items = 0, items1 = 0, blocks1 = 0;  // blocks and items (tile 1: its own)
        auto scores = [&](int st, uint32_t b) {
            const uint64_t qd = q_desc + st * kTileStep, kd = k_desc + b * kTileStep;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                mma_ss(one, tmem + kColS + st * 128, qd + at, kd + at, id_s, k > 0);
            }
            commit(one, smem_u32(&bars.sfull[st]));
        };
        auto outputs = [&](int st, uint32_t b, bool acc) {
            const uint64_t vd = v_desc + b * kTileStep;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
                mma_ts(one, tmem + kColO + st * 128, tmem + kColS + st * 128 + k * 8,
                       vd + k * (2048 >> 4), id_o, acc || k > 0);
        };
        bool ok = true;
        auto wait = [&](uint64_t& bar, uint32_t parity) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bar), parity & 1, abort_flag, a.status));
            return ok;
        };
        for (; more && ok; more = Work::next(a, sh, it)) {
            const int tiles = it.row1 - it.row0 > kRowsTile ? 2 : 1;
            const int32_t count = it.u1 - it.u0;
            if (!wait(bars.kfull[n & 1], n >> 1))
                break;
            for (int st = 0; st < tiles; ++st) {
                if (!wait(bars.qfull[st], st ? items1 : items))
                    break;
                fence_after();
                scores(st, n & 1);
            }
            commit(one, smem_u32(&bars.kempty[n & 1]));
            for (int32_t j = 0; j < count && ok; ++j, ++n) {
                const uint32_t b = n & 1, nb = (n + 1) & 1;
                if (!wait(bars.vfull[b], n >> 1))
                    break;
                for (int st = 0; st < tiles; ++st) {
                    if (!wait(bars.pfull[st], st ? blocks1 : n))
                        break;
                    fence_after();
                    outputs(st, b, j > 0);
                    if (st == tiles - 1)
                        commit(one, smem_u32(&bars.vempty[b]));
                    if (j + 1 < count) {
                        if (st == 0 && !wait(bars.kfull[nb], (n + 1) >> 1))
                            break;
                        fence_after();
                        scores(st, nb);
                        if (st == tiles - 1)
                            commit(one, smem_u32(&bars.kempty[nb]));
                    } else {
                        commit(one, smem_u32(&bars.ofull[st]));
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
        commit(one, smem_u32(&bars.drain));
        const long long t0 = clock64();
        while (!mbar_test(smem_u32(&bars.drain), 0) && clock64() - t0 < kKvWaitBudget) {
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

template <int D, bool WINDOW>
cudaError_t launch(const KvAttnArgs& a, cudaStream_t stream, bool pdl)
{
    const int dev = current_device();
    const cudaError_t e = ensure_smem_limit(kv_tile_kernel<D, WINDOW>, Cfg<D>::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    return kv_launch(kv_tile_kernel<D, WINDOW>, device_sm_count(dev), kThreads, Cfg<D>::kSmem, stream, pdl, a);
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
    if (a.window > 0)
        return a.c.dim == 128 ? launch<128, true>(a, stream, pdl) : launch<64, true>(a, stream, pdl);
    return a.c.dim == 128 ? launch<128, false>(a, stream, pdl) : launch<64, false>(a, stream, pdl);
}

}  // namespace nvfp4

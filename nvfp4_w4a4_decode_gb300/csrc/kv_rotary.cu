// kv_rotary.cu -- the append with the position rotation on the way: queries and keys are
// turned by their token's angles, keys and values quantised into the paged cache.
//
// Mathematics.  The first `rot` elements of a head are rot / 2 pairs (a, b), at i and
// i + rot / 2 or, interleaved, at 2 i and 2 i + 1.  With (c, s) the cosine and sine of the
// token's angle i, a float32 table's row,
//     a' = a c - b s,   b' = b c + a s,
// the two products and their sum rounded to float32 each (no fused step), so that every
// bit of a' and b' has one right value, and with it every byte of the cache: keys go from
// here into the block recipe without a rounding between.  Queries are rounded once, to
// their own type.
//
// Layout.  A thread takes 8 pairs of U query heads, which share their angles, or two
// 16-element blocks of one head of K or V: the two that the rotation pairs (neighbours
// where the pairs are interleaved, or nothing is turned).  Its units are neighbouring
// pieces of a head, so that a warp's loads and stores are runs of whole sectors.
//
// What bounds it: memory (16103 tokens of 32/8 heads of 128 in BF16: 357 MB in 60.2 us, 5.9 TB/s,
// 88 % of the copy rate) once enough loads are on their way; few tokens the launch (8 tokens: 2.5 us).
#include "../../include/nvfp4_kv.h"
#include "kv.cuh"
#include "kv_quantise.cuh"
#include "launch_cache.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 128;
// With many tokens a thread turns four query heads by the angles it has loaded (two in FP32, whose
// elements take twice the registers), seven CTAs an SM.  Measured, 32/8 heads of 128: 16103 tokens in
// BF16, 60.2 us; with eight heads 88, two 69, one 114; six CTAs an SM 64, eight 63, nine 80, as many as come
// of themselves (five) 71.  19583 tokens in FP32, 124.7 us, 6.7 TB/s; with four heads 178, one 166; six, five
// or as many as come of themselves 129.4, eight 128.5.
template <bool BF16>
constexpr int kManyHeads = BF16 ? 4 : 2;
template <int U>
constexpr int kCtas = U == 1 ? 1 : 7;

// (a, b) turned by (c, s), each operation rounded.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s)
{
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

template <int N>
__device__ __forceinline__ void load_angles(const float* p, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
}

// Eight elements as they lie in memory.  Plain loads: queries may be turned in place.
template <bool BF16>
struct Eight {
    uint4 w[BF16 ? 1 : 2];
};

template <bool BF16, bool WIDE>
__device__ __forceinline__ Eight<BF16> load_eight(const void* p)
{
    Eight<BF16> x;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
        if constexpr (WIDE) {
            x.w[i] = static_cast<const uint4*>(p)[i];
        } else {
            const uint2 a = static_cast<const uint2*>(p)[2 * i], b = static_cast<const uint2*>(p)[2 * i + 1];
            x.w[i] = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    return x;
}

template <bool BF16, bool WIDE>
__device__ __forceinline__ void store_eight(void* p, const Eight<BF16>& x)
{
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
        if constexpr (WIDE) {
            static_cast<uint4*>(p)[i] = x.w[i];
        } else {
            static_cast<uint2*>(p)[2 * i] = make_uint2(x.w[i].x, x.w[i].y);
            static_cast<uint2*>(p)[2 * i + 1] = make_uint2(x.w[i].z, x.w[i].w);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Eight<BF16>& x, float (&v)[8])
{
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x.w);
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
        if constexpr (BF16) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            v[i] = __uint_as_float(w[i]);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ Eight<BF16> pack(const float (&v)[8])
{
    Eight<BF16> x;
    uint32_t* w = reinterpret_cast<uint32_t*>(x.w);
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
        if constexpr (BF16)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        else
            w[i] = __float_as_uint(v[i]);
    }
    return x;
}

// Units of a token: U query heads' pieces of 8 pairs (q_units), then pairs of blocks of K
// and of V.
template <bool BF16, bool WIDE, int U>
__global__ void __launch_bounds__(kThreads, kCtas<U>)
    kv_rotary_kernel(const KvRotaryArgs a, uint32_t per, uint32_t q_units, int q_groups)
{
    kv_pdl_begin();
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = (at >> 32) == 0 ? (int64_t)((uint32_t)at / per) : at / per;
    if (t >= a.tokens)
        return;
    const uint32_t unit = (uint32_t)(at - t * per);
    constexpr int kItem = BF16 ? 2 : 4;
    const int32_t pos = __ldg(a.positions + t);
    const bool known = pos >= 0 && pos < a.rotary_rows;
    const float* angles = a.rotary + pos * a.rotary_stride;  // followed only where the row is known
    const int half = a.rot / 2;

    if (unit < q_units) {
        const int pieces = a.c.dim / 16;
        const int g = unit / pieces, j = unit - g * pieces;
        const bool turned = 8 * j < half;
        const bool split = turned && !a.interleaved;
        const int lo = split ? 8 * j : 16 * j, hi = split ? lo + half : lo + 8;
        const char* src = static_cast<const char*>(a.q) + t * a.q_stride * kItem;
        char* dst = static_cast<char*>(a.q_out) + t * a.q_out_stride * kItem;
        Eight<BF16> x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = g + u * q_groups;
            if (h < a.q_heads) {
                x[u] = load_eight<BF16, WIDE>(src + (h * a.c.dim + lo) * kItem);
                y[u] = load_eight<BF16, WIDE>(src + (h * a.c.dim + hi) * kItem);
            }
        }
        float c[8], s[8];
        if (turned && known) {
            load_angles(angles + 8 * j, c);
            load_angles(angles + half + 8 * j, s);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = g + u * q_groups;
            if (h >= a.q_heads)
                break;
            if (turned && known) {
                float p[8], q[8];
                unpack(x[u], p);
                unpack(y[u], q);
                if (split) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        turn(p[i], q[i], c[i], s[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        turn(p[2 * i], p[2 * i + 1], c[i], s[i]);
                        turn(q[2 * i], q[2 * i + 1], c[4 + i], s[4 + i]);
                    }
                }
                x[u] = pack<BF16>(p);
                y[u] = pack<BF16>(q);
            }
            if (!known)
                x[u] = y[u] = Eight<BF16>{};
            store_eight<BF16, WIDE>(dst + (h * a.c.dim + lo) * kItem, x[u]);
            store_eight<BF16, WIDE>(dst + (h * a.c.dim + hi) * kItem, y[u]);
        }
        return;
    }

    const int nb = a.c.dim / 16, pairs = nb / 2;
    const int i = unit - q_units;
    const bool is_v = i >= pairs * a.c.heads;
    const int k = is_v ? i - pairs * a.c.heads : i;
    const int h = k / pairs, j = k - h * pairs;
    const bool turned = !is_v && 16 * j < half;
    const bool split = turned && !a.interleaved;
    const int b0 = split ? j : 2 * j, b1 = split ? j + half / 16 : b0 + 1;
    const char* src = static_cast<const char*>(is_v ? a.v : a.k) +
                      (t * (is_v ? a.v_stride : a.k_stride) + h * a.c.dim) * kItem;
    const RawBlock<BF16> x = load_block<BF16, WIDE>(src + b0 * 16 * kItem);
    const RawBlock<BF16> y = load_block<BF16, WIDE>(src + b1 * 16 * kItem);
    const int64_t slot = __ldg(a.slots + t);
    if (slot == -1)
        return;
    if (slot < 0 || (slot >> a.c.page_shift) >= a.c.num_pages || !known) {
        if (i == 0)
            atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
        return;
    }
    const float g = __ldg(is_v ? a.c.v_g : a.c.k_g);
    float p[16], q[16];
    values<BF16>(x, p);
    values<BF16>(y, q);
    if (turned) {
        float c[16], s[16];
        load_angles(angles + 16 * j, c);
        load_angles(angles + half + 16 * j, s);
        if (split) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                turn(p[e], q[e], c[e], s[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                turn(p[2 * e], p[2 * e + 1], c[e], s[e]);
                turn(q[2 * e], q[2 * e + 1], c[8 + e], s[8 + e]);
            }
        }
    }
    const int32_t off = (int32_t)slot & ((1 << a.c.page_shift) - 1);
    uint8_t* base = a.c.pool + (slot >> a.c.page_shift) * a.c.page_stride +
                    h * kv_head_bytes(a.c.page_shift, a.c.dim);
    const int code_part = (a.c.dim / 2) << a.c.page_shift, scale_part = nb << a.c.page_shift;
    uint8_t* codes = base + (is_v ? code_part : 0) + off * (a.c.dim / 2);
    uint8_t* scales = base + 2 * code_part + (is_v ? scale_part : 0) + off * nb;
    uint2 w;
    scales[b0] = (uint8_t)quantise(p, g, w);
    *reinterpret_cast<uint2*>(codes + b0 * 8) = w;
    scales[b1] = (uint8_t)quantise(q, g, w);
    *reinterpret_cast<uint2*>(codes + b1 * 8) = w;
}

template <bool BF16, bool WIDE, int U>
cudaError_t launch_units(const KvRotaryArgs& a, cudaStream_t stream, bool pdl)
{
    const int groups = (a.q_heads + U - 1) / U;
    const uint32_t q_units = (uint32_t)groups * (a.c.dim / 16);
    const uint32_t per = q_units + 2 * a.c.heads * (a.c.dim / 32);
    const int64_t ctas = (a.tokens * per + kThreads - 1) / kThreads;
    if (ctas > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    return kv_launch(kv_rotary_kernel<BF16, WIDE, U>, (unsigned)ctas, kThreads, 0, stream, pdl, a, per,
                     q_units, groups);
}

template <bool BF16, bool WIDE>
cudaError_t launch(const KvRotaryArgs& a, cudaStream_t stream, bool pdl)
{
    // several heads a thread once that still leaves every SM a few CTAs
    constexpr int kMany = kManyHeads<BF16>;
    const int64_t units = a.tokens * ((int64_t)(a.q_heads + kMany - 1) / kMany * (a.c.dim / 16) +
                                      a.c.heads * (a.c.dim / 16));
    return units >= (int64_t)8 * kThreads * device_sm_count(current_device())
               ? launch_units<BF16, WIDE, kMany>(a, stream, pdl)
               : launch_units<BF16, WIDE, 1>(a, stream, pdl);
}

}  // namespace

cudaError_t launch_kv_rotary(const KvRotaryArgs& a, bool bf16, cudaStream_t stream, bool pdl)
{
    if (!bf16)
        return launch<false, true>(a, stream, pdl);
    // 16-byte loads and stores where pointers and rows allow them
    const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                        reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out)) & 15) == 0 &&
                      ((a.k_stride | a.v_stride | a.q_stride | a.q_out_stride) & 7) == 0;
    return wide ? launch<true, true>(a, stream, pdl) : launch<true, false>(a, stream, pdl);
}

}  // namespace nvfp4

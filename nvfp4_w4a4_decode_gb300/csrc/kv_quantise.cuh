// kv_quantise.cuh -- one block of 16 elements on its way into the paged cache: wide
// loads, the block's scale and its E2M1 codes (shared by the plain and the rotating
// append, so that both write the same bytes for the same values).
#pragma once

#include "formats.cuh"

namespace nvfp4 {

// 16 elements as they lie in memory.
template <bool BF16>
struct RawBlock {
    uint4 w[BF16 ? 2 : 4];
};

template <bool BF16, bool WIDE>
__device__ __forceinline__ RawBlock<BF16> load_block(const void* p)
{
    RawBlock<BF16> x;
    constexpr int n = BF16 ? 2 : 4;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            x.w[i] = __ldg(static_cast<const uint4*>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint2 a = __ldg(static_cast<const uint2*>(p) + 2 * i);
            const uint2 b = __ldg(static_cast<const uint2*>(p) + 2 * i + 1);
            x.w[i] = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    return x;
}

template <bool BF16>
__device__ __forceinline__ void values(const RawBlock<BF16>& x, float (&v)[16])
{
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[4 * i] = __uint_as_float(x.w[i].x);
            v[4 * i + 1] = __uint_as_float(x.w[i].y);
            v[4 * i + 2] = __uint_as_float(x.w[i].z);
            v[4 * i + 3] = __uint_as_float(x.w[i].w);
        }
    }
}

// Eight values to eight E2M1 codes, element 0 in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float* q)
{
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return w;
}

__device__ __forceinline__ uint32_t quantise(float (&v)[16], float g, uint2& codes)
{
    float bmax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        bmax = fmaxf(bmax, fabsf(v[i]));
    float S;
    const uint32_t sc = block_scale(bmax, g, S);
    const BlockDivisor d = make_divisor(S);
    if (d.fast && bmax <= 0x1p+100f) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            // two quotients in packed FP32: q0 = t r, q = q0 + (t - S q0) r
            uint64_t t2, r2, s2, q;
            asm("mov.b64 %0, {%1, %2};" : "=l"(t2) : "f"(v[i]), "f"(v[i + 1]));
            asm("mov.b64 %0, {%1, %1};" : "=l"(r2) : "f"(d.r));
            asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(-d.S));
            asm("{\n\t.reg .b64 q0, e;\n\t"
                "mul.rn.f32x2 q0, %1, %2;\n\t"
                "fma.rn.f32x2 e, %3, q0, %1;\n\t"
                "fma.rn.f32x2 %0, e, %2, q0;\n\t}"
                : "=l"(q)
                : "l"(t2), "l"(r2), "l"(s2));
            float q0, q1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(q0), "=f"(q1) : "l"(q));
            // the sign is the element's (the correction of a zero is +0)
            v[i] = copysignf(q0, v[i]);
            v[i + 1] = copysignf(q1, v[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = S == 0.0f ? copysignf(0.0f, v[i]) : __fdiv_rn(v[i], S);
    }
    codes = make_uint2(e2m1x8(v), e2m1x8(v + 8));
    return sc;
}

}  // namespace nvfp4

// kv_append.cu -- quantise a step's keys and values into the paged cache.
//
// A thread takes one 16-element block of one head of K or V of one token: its
// block maximum, the E4M3 scale relative to the tensor scale, the 16 E2M1
// codes (the library's one recipe, formats.cuh), 8 code bytes and 1 scale byte
// stored.  Blocks of a head row are neighbouring threads, so a warp reads
// contiguous rows and writes contiguous codes.  Bound by the bytes read.
#include "../../include/nvfp4_kv.h"
#include "formats.cuh"
#include "kv.cuh"
#include "launch_cache.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void load16(const void* p, float (&v)[16])
{
    if constexpr (BF16) {
        const uint2* s = static_cast<const uint2*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 w = __ldg(s + i);
            v[4 * i] = __uint_as_float(w.x << 16);
            v[4 * i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
            v[4 * i + 2] = __uint_as_float(w.y << 16);
            v[4 * i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
        }
    } else {
        const float4* s = static_cast<const float4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 w = __ldg(s + i);
            v[4 * i] = w.x;
            v[4 * i + 1] = w.y;
            v[4 * i + 2] = w.z;
            v[4 * i + 3] = w.w;
        }
    }
}

// `per` blocks a token (K's, then V's), `tpc` tokens a CTA.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a, int per, int tpc)
{
    kv_pdl_begin();
    const int nb = a.c.dim / 16;
    const int tl = per <= kThreads ? threadIdx.x / per : 0;
    const int64_t t = (int64_t)blockIdx.x * tpc + tl;
    if (tl >= tpc || t >= a.tokens)
        return;
    const int64_t slot = a.slots[t];
    if (slot < 0 || (slot >> a.c.page_shift) >= a.c.num_pages) {
        if (slot != -1 && threadIdx.x == tl * per)
            atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
        return;
    }
    const int64_t head_bytes = kv_head_bytes(a.c.page_shift, a.c.dim);
    const int32_t off = (int32_t)slot & ((1 << a.c.page_shift) - 1);
    uint8_t* page = a.c.pool + (slot >> a.c.page_shift) * a.c.page_stride;
    const int code_part = (a.c.dim / 2) << a.c.page_shift, scale_part = nb << a.c.page_shift;
    for (int i = threadIdx.x - tl * per; i < per; i += kThreads) {
        const bool is_v = i >= per / 2;
        const int j = is_v ? i - per / 2 : i;  // head * nb + block
        const int h = j / nb, b = j - h * nb;
        float v[16];
        const int64_t at = t * (is_v ? a.v_stride : a.k_stride) + j * 16;
        load16<BF16>(static_cast<const char*>(is_v ? a.v : a.k) + at * (BF16 ? 2 : 4), v);
        uint32_t w0, w1;
        const uint32_t sc = quantize_block16(v, __ldg(is_v ? a.c.v_g : a.c.k_g), w0, w1);
        uint8_t* base = page + h * head_bytes;
        *reinterpret_cast<uint2*>(base + (is_v ? code_part : 0) + off * (a.c.dim / 2) + b * 8) =
            make_uint2(w0, w1);
        base[2 * code_part + (is_v ? scale_part : 0) + off * nb + b] = (uint8_t)sc;
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool bf16, cudaStream_t stream, bool pdl)
{
    const int per = 2 * a.c.heads * (a.c.dim / 16);
    const int tpc = per >= kThreads ? 1 : kThreads / per;
    const int64_t grid = (a.tokens + tpc - 1) / tpc;
    return kv_launch(bf16 ? kv_append_kernel<true> : kv_append_kernel<false>, (unsigned)grid,
                     kThreads, 0, stream, pdl, a, per, tpc);
}

}  // namespace nvfp4

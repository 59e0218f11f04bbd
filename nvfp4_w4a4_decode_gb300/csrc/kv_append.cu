// kv_append.cu -- quantise a step's keys and values into the paged cache.
//
// A thread takes one 16-element block of one head of K or V of one token: its
// block maximum, the E4M3 scale relative to the tensor scale, the 16 E2M1
// codes, 8 code bytes and 1 scale byte stored.  Blocks of a head row are
// neighbouring threads, so a warp reads contiguous rows and writes contiguous
// codes.  The recipe is the library's (formats.cuh) to the bit: the quotient
// t / S comes from the block's reciprocal with one correction, correctly rounded
// in its domain and by division outside it, and the conversion to E2M1 is the
// hardware's (round to nearest even, saturating, sign kept), two elements an
// instruction instead of seven comparisons an element.
//
// 16384 tokens of 8 heads of 128 in BF16: 20.4 us for 86 MB, 4.2 TB/s.  No unit is full
// then (issue active 55 %, ALU 55 %, DRAM 41 % of its peak; a warp waits most for its
// loads): it is bound by the latency of loads and of the chain from block maximum to
// codes, with 28 warps an SM.  So the loads of a thread's blocks (of several tokens,
// when there are enough of them to fill the SMs) are issued before its slots are
// looked up.
#include "../../include/nvfp4_kv.h"
#include "kv.cuh"
#include "kv_quantise.cuh"
#include "launch_cache.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 128;
// Blocks a thread when there are many (16384 tokens of 8 heads of 128: 20.6 us
// with two; with one 23.6, four 27.8, eight 29.5).
constexpr int kManyTokens = 2;

// `per` blocks a token (K's, then V's), `tpc` tokens a CTA at a time, U times.
template <bool BF16, bool WIDE, int U>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a, int per, int tpc)
{
    kv_pdl_begin();
    const int nb = a.c.dim / 16;
    const int tl = per <= kThreads ? threadIdx.x / per : 0;
    const int64_t t0 = (int64_t)blockIdx.x * tpc * U + tl;
    if (tl >= tpc || t0 >= a.tokens)
        return;
    const int64_t head_bytes = kv_head_bytes(a.c.page_shift, a.c.dim);
    const int code_part = (a.c.dim / 2) << a.c.page_shift, scale_part = nb << a.c.page_shift;
    for (int i = threadIdx.x - tl * per; i < per; i += kThreads) {
        const bool is_v = i >= per / 2;
        const int j = is_v ? i - per / 2 : i;  // head * nb + block
        const int h = j / nb, b = j - h * nb;
        const char* src = static_cast<const char*>(is_v ? a.v : a.k);
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        RawBlock<BF16> x[U];
        int64_t slot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * tpc;
            slot[u] = -1;
            if (t < a.tokens) {
                x[u] = load_block<BF16, WIDE>(src + (t * stride + j * 16) * (BF16 ? 2 : 4));
                slot[u] = __ldg(a.slots + t);
            }
        }
        const float g = __ldg(is_v ? a.c.v_g : a.c.k_g);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (slot[u] < 0 || (slot[u] >> a.c.page_shift) >= a.c.num_pages) {
                if (slot[u] != -1 && i == 0)
                    atomicOr(a.status, NVFP4_DEVICE_KV_RANGE);
                continue;
            }
            const int32_t off = (int32_t)slot[u] & ((1 << a.c.page_shift) - 1);
            uint8_t* base = a.c.pool + (slot[u] >> a.c.page_shift) * a.c.page_stride + h * head_bytes;
            float v[16];
            values<BF16>(x[u], v);
            uint2 codes;
            const uint32_t sc = quantise(v, g, codes);
            *reinterpret_cast<uint2*>(base + (is_v ? code_part : 0) + off * (a.c.dim / 2) + b * 8) =
                codes;
            base[2 * code_part + (is_v ? scale_part : 0) + off * nb + b] = (uint8_t)sc;
        }
    }
}

template <bool BF16, bool WIDE>
cudaError_t launch(const KvAppendArgs& a, cudaStream_t stream, bool pdl)
{
    const int per = 2 * a.c.heads * (a.c.dim / 16);
    const int tpc = per >= kThreads ? 1 : kThreads / per;
    // several tokens a thread once that still leaves every SM a few CTAs
    const int64_t ctas = (a.tokens + tpc - 1) / tpc;
    const bool many = ctas >= (int64_t)kManyTokens * 4 * device_sm_count(current_device());
    const int u = many ? kManyTokens : 1;
    return kv_launch(many ? kv_append_kernel<BF16, WIDE, kManyTokens> : kv_append_kernel<BF16, WIDE, 1>,
                     (unsigned)((ctas + u - 1) / u), kThreads, 0, stream, pdl, a, per, tpc);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool bf16, cudaStream_t stream, bool pdl)
{
    if (!bf16)
        return launch<false, true>(a, stream, pdl);
    // 16-byte loads where pointers and rows allow them
    const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0 &&
                      ((a.k_stride | a.v_stride) & 7) == 0;
    return wide ? launch<true, true>(a, stream, pdl) : launch<true, false>(a, stream, pdl);
}

}  // namespace nvfp4

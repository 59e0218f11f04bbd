// kv_join.cu -- the outputs of rows whose keys were taken in two passes (a shared prefix, a
// request's own keys), from the parts that these left: with M the largest reference,
//     L = sum l_k 2^(m_k - M),  out = v_g / L sum o_k 2^(m_k - M),  lse = ln L + M ln 2,
// added up in one order, first the prefix's parts, then the own ones.
//
// A warp a row, and a CTA: its lanes take the parts' references and sums, 32 at a time, then four
// elements each of all parts, sixteen loads on their way at once.  What bounds it: three loads that
// wait for one another (where the parts lie, their statistics, the parts), and L2 (64 tokens of 32
// heads, 17 parts each of a prefix and one or two of the own keys: 20 MB, 4 us behind the passes); its
// launch is hidden by them.  The call took 41.6 us with eight loads and four warps a CTA, 40.6 with
// sixteen loads, and two requests on 60000 tokens 29.9, 28.9 and with a warp a CTA 27.4.  (With the prefix's
// parts added up by the other pass at its items' starts a call of two tokens behind 1030 took 17.7 us
// instead of 14.5.)
#include <cuda_bf16.h>

#include "kv.cuh"
#include "kv_work.cuh"

namespace nvfp4 {

namespace {

template <int D>
__global__ void __launch_bounds__(32) kv_join_kernel(const KvAttnArgs a)
{
    kv_pdl_begin();
    const int lane = threadIdx.x, heads = a.c.heads * a.group;
    const int64_t at = blockIdx.x;
    const int64_t t = kv_divide(at, heads);
    // rows of no request are the second pass's to write
    int32_t begin = 0, end = a.tokens;
    if (a.q_start) {
        begin = a.q_start[0];
        end = min(a.q_start[a.reqs], a.tokens);
    }
    if (t < begin || t >= end)
        return;
    const bool shares = (a.keep.where[at] & kKvSharesBit) != 0;
    int parts[2] = {0, 0};
    int32_t where[2] = {0, 0};
    if (shares)
        where[0] = kv_where(a.prefix, at, parts[0]);
    where[1] = kv_where(a.keep, at, parts[1]);

    constexpr int kPieces = D / 4, kAbreast = 32 / kPieces;  // float4s of a row; rows at a time
    const int piece = lane % kPieces, first = lane / kPieces;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY, total = 0.f;
    const int all = parts[0] + parts[1];
    for (int k0 = 0; k0 < all; k0 += 32) {
        const int n = min(32, all - k0);
        // this lane's part
        const int k = k0 + lane, own = k >= parts[0], w = where[own];
        const KvParts& s = own ? a.keep : a.prefix;
        const int64_t row = w ? kv_part_row(w, own ? k - parts[0] : k, s.item_rows) : at;
        const float* src = (w ? s.parts : s.rows) + row * D;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n)
            ml = __ldcg((w ? s.part_stats : s.stats) + row);
        constexpr int kAhead = 16 / kAbreast;
        float4 x[kAhead];
        auto load = [&](int z0) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int z = z0 + i * kAbreast + first;
                const float* p = reinterpret_cast<const float*>(
                    __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), z & 31));
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (z < n)
                    x[i] = __ldcg(reinterpret_cast<const float4*>(p) + piece);
            }
        };
        load(0);
        float now = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, d));
        now = fmaxf(now, top);
        const float by = top == now ? 1.f : ex2(top - now);
        const float mine = ml.x == now ? 1.f : ex2(ml.x - now);
        float l = ml.y * mine;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        total = fmaf(total, by, l);
        top = now;
        sum.x *= by, sum.y *= by, sum.z *= by, sum.w *= by;
        for (int z0 = 0; z0 < n; z0 += kAhead * kAbreast) {
            if (z0)
                load(z0);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float f = __shfl_sync(0xFFFFFFFFu, mine, (z0 + i * kAbreast + first) & 31);
                sum.x = fmaf(x[i].x, f, sum.x);
                sum.y = fmaf(x[i].y, f, sum.y);
                sum.z = fmaf(x[i].z, f, sum.z);
                sum.w = fmaf(x[i].w, f, sum.w);
            }
        }
    }
    if constexpr (kAbreast == 2) {
        sum.x += __shfl_xor_sync(0xFFFFFFFFu, sum.x, 16);
        sum.y += __shfl_xor_sync(0xFFFFFFFFu, sum.y, 16);
        sum.z += __shfl_xor_sync(0xFFFFFFFFu, sum.z, 16);
        sum.w += __shfl_xor_sync(0xFFFFFFFFu, sum.w, 16);
    }
    const float scale = total == 0.f ? 0.f : a.c.v_g[0] / total;
    if (first == 0) {
        const int64_t to = t * a.out_stride + (at - t * heads) * D + 4 * piece;
        if (a.out_bf16) {
            __nv_bfloat162 v[2] = {__floats2bfloat162_rn(sum.x * scale, sum.y * scale),
                                   __floats2bfloat162_rn(sum.z * scale, sum.w * scale)};
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) = *reinterpret_cast<const uint2*>(v);
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) =
                make_float4(sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale);
        }
    }
    if (a.lse != nullptr && lane == 0)
        a.lse[at] = total == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(total));
}

}  // namespace

cudaError_t launch_kv_join(const KvAttnArgs& a, cudaStream_t stream)
{
    const int64_t rows = (int64_t)a.tokens * a.c.heads * a.group;
    return kv_launch(a.c.dim == 128 ? kv_join_kernel<128> : kv_join_kernel<64>, (unsigned)rows, 32, 0, stream, true,
                     a);
}

}  // namespace nvfp4

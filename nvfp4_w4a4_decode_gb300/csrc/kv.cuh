// kv.cuh -- the paged NVFP4 key/value cache: layout, launchers and the
// device-side work list of the attention kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4_kv.h"

namespace nvfp4 {

// nvfp4_kv_cache as the kernels take it.  Bytes of one (page, kv head), P
// tokens of D elements: K codes [P][D/2], V codes [P][D/2], K scales
// [P][D/16], V scales [P][D/16].  16 tokens of each part are contiguous, and a
// page is a multiple of 16 tokens, so a chunk of 16 tokens is four contiguous
// pieces and never leaves its page.
struct KvCache {
    uint8_t* pool;
    const float* k_g;
    const float* v_g;
    int64_t num_pages;
    int64_t page_stride;
    int32_t page_shift;  // log2 of the tokens a page
    int32_t heads;
    int32_t dim;
};

__host__ __device__ __forceinline__ int64_t kv_head_bytes(int page_shift, int dim)
{
    return ((int64_t)dim * 9 / 8) << page_shift;
}

constexpr int kKvMaxReqs = 16384;
constexpr int kKvMaxGroup = 64;

struct KvTablesArgs {
    const int32_t* kv_len;
    const int32_t* q_len;
    int32_t reqs;
    int32_t page_shift;
    const int32_t* free_pages;
    int64_t num_free;
    const int32_t* free_head;
    int32_t* table;
    int64_t table_stride;
    int32_t max_blocks;
    int32_t* seq_len;
    int32_t* q_start;
    int64_t* slots;
    int32_t* positions;
    int32_t tokens;
    int32_t* free_next;
    unsigned* status;
};

cudaError_t launch_kv_tables(const KvTablesArgs& a, cudaStream_t stream, bool pdl);

struct KvAppendArgs {
    KvCache c;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;  // elements
    const int64_t* slots;
    int64_t tokens;
    unsigned* status;
};

cudaError_t launch_kv_append(const KvAppendArgs& a, bool bf16, cudaStream_t stream, bool pdl);

struct KvRotaryArgs {
    KvCache c;
    const void* q;
    void* q_out;
    const void* k;
    const void* v;
    int64_t q_stride, q_out_stride, k_stride, v_stride;  // elements
    int32_t q_heads;
    const int64_t* slots;
    const int32_t* positions;
    int64_t tokens;
    const float* rotary;  // rows of rot / 2 cosines, then rot / 2 sines
    int64_t rotary_rows, rotary_stride;
    int32_t rot;  // a multiple of 32, at most dim
    int32_t interleaved;
    unsigned* status;
};

cudaError_t launch_kv_rotary(const KvRotaryArgs& a, bool bf16, cudaStream_t stream, bool pdl);

// Which keys a query row of a request sees (position p of the row, seq keys in all).
enum class KvSees {
    kCausal,  // j <= p, with a window j > p - W
    kAll,     // j < seq: cross attention, and the prefix that a group's requests share
    kBehind,  // KvShared::first of its request <= j <= p: a request's own keys
};

// What a pass over some of a row's keys leaves of it: the sum of p V, the reference (log2)
// and the sum of p.  An item cut between CTAs is not joined by the pass (one SM would read the
// parts of 256 rows while the others wait): whoever reads the row adds up its parts.
struct KvParts {
    float* rows;         // [tokens][query heads][D]: of items that were not cut
    float2* stats;       // [tokens][query heads]
    float* parts;        // [total][D]: of the cut ones, two places of an item's rows a CTA
    float2* part_stats;  // [total]
    int32_t* where;      // [tokens][query heads]: 0, or parts << kKvPartBits | row of the first in
                         // `parts`; with kKvSharesBit where the prefix's sums belong to the row
    int64_t total;       // rows of `parts`
    int32_t item_rows;   // query rows of an item of the pass
};

// Rows of KvParts::parts: two items of 256 rows on each SM, or of 32 rows for 512 CTAs.
constexpr int kKvPartBits = 17;
constexpr int32_t kKvSharesBit = 1 << 30;
constexpr int64_t kv_part_total(int sms)
{
    return (int64_t)(sms > 64 ? sms : 64) * 512;
}

// Devices of more SMs, whose rows `where` has no bits for, are refused.
constexpr int kKvMostSms = 256;
static_assert(kv_part_total(kKvMostSms) <= (int64_t)1 << kKvPartBits);

// Part k's row of the parts that `where` names: the first lies in its CTA's second place, the
// others in the first places of the CTAs behind.
__device__ __forceinline__ int64_t kv_part_row(int32_t where, int k, int item_rows)
{
    return (where & ((1 << kKvPartBits) - 1)) + (k ? (int64_t)(2 * k - 1) * item_rows : 0);
}

// What a pass has written for a row, and the number of its parts.  Starts that go back
// (the rows of a request are then not those of its group) may leave anything there: such an
// entry is not followed.
__device__ __forceinline__ int32_t kv_where(const KvParts& s, int64_t row, int& parts)
{
    int32_t w = s.where[row] & ~kKvSharesBit;
    parts = w >> kKvPartBits;
    if (w < 0 || (parts > 0 && kv_part_row(w, parts - 1, s.item_rows) >= s.total))
        w = parts = 0;
    if (parts == 0)
        w = 0, parts = 1;
    return w;
}

// Requests that share prefixes take two passes.  The first (kAll) takes a group for a request:
// its rows are those of the group's requests, its table the prefix's.  The second (kBehind)
// takes the requests' own keys; with many rows a request it joins the two itself, else both leave
// their parts to launch_kv_join.
struct KvGroups {
    const int32_t* start;       // first request of each group, or null: one group of all
    const int32_t* prefix_len;  // tokens of each group's prefix
    int32_t count, reqs;
    int64_t cap;                // keys that a row of the prefixes' table has room for
};

struct KvAttnArgs {
    KvCache c;
    const void* q;
    int64_t q_stride;
    const int32_t* table;
    int64_t table_stride;
    int32_t max_blocks;
    const int32_t* seq_len;
    const int32_t* q_start;  // or null: q_per_req rows each
    int32_t q_per_req;
    int32_t reqs;
    int32_t tokens;
    int32_t max_q;
    int32_t group;  // query heads per kv head
    uint32_t group_magic;  // floor(2^32 / group) + 1
    float scale_log2;
    int32_t window;  // 0: none
    void* out;
    int64_t out_stride;
    float* lse;
    int32_t q_bf16, out_bf16;
    int32_t all_rows;  // rows of no request are written too
    KvGroups groups;
    KvParts keep;     // where the pass leaves its rows (rows null: it writes outputs)
    KvParts prefix;   // what the first pass left
    float* part;      // partial results of items cut between CTAs (null: none is cut)
    unsigned* count;  // arrival counters, zero between calls
    unsigned* status;
};

// The workspace's arrival counters (zero between calls; both kernels' lie
// here), then partial results.
constexpr int64_t kKvCountBytes = NVFP4_KV_WORKSPACE_ZERO;

// Few query rows a request, any dtype.
int64_t kv_rows_workspace_bytes(int dim);
int kv_rows_item_rows(const KvAttnArgs& a);  // query rows of an item of the launch for these arguments
template <KvSees S>
cudaError_t launch_kv_rows(const KvAttnArgs& a, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl);

// Many query rows a request (tcgen05); BF16 queries and outputs only.
int64_t kv_tile_workspace_bytes(int dim);
int kv_tile_item_rows();
template <KvSees S>
cudaError_t launch_kv_tile(const KvAttnArgs& a, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl);

// The outputs of rows whose sums lie in a.prefix and a.keep (the second pass's).
cudaError_t launch_kv_join(const KvAttnArgs& a, cudaStream_t stream);

// Launch with or without programmatic dependent launch (every kernel of the
// cache waits for the previous one before its first access).
template <typename... P, typename... A>
inline cudaError_t kv_launch(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem,
                             cudaStream_t stream, bool pdl, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

__device__ __forceinline__ void kv_pdl_launch()
{
    asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void kv_pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void kv_pdl_begin()
{
    kv_pdl_launch();
    kv_pdl_wait();
}
// Of the two passes of shared prefixes the first lets the second start only when what came
// before it is complete; so the second waits for nothing but the first's results, if and when
// it reads them.  Its last CTA waits for the first pass before it ends, so that what follows the
// second pass follows both (if every CTA did, those that found no room beside the first pass's would
// come after it: 64 tokens behind 8003 41.6 us).
template <KvSees S>
__device__ __forceinline__ void kv_pdl_begin(const KvParts& keep)
{
    if constexpr (S == KvSees::kBehind) {
        kv_pdl_launch();
    } else if (S == KvSees::kAll && keep.rows != nullptr) {
        kv_pdl_wait();
        kv_pdl_launch();
    } else {
        kv_pdl_begin();
    }
}

template <KvSees S>
__device__ __forceinline__ void kv_pdl_end()
{
    if (S == KvSees::kBehind && blockIdx.x == gridDim.x - 1)
        kv_pdl_wait();
}

}  // namespace nvfp4

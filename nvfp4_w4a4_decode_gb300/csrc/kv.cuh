// kv.cuh -- the paged NVFP4 key/value cache: layout, launchers and the
// device-side work list of the attention kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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
    float scale_log2;
    int32_t window;  // 0: none
    void* out;
    int64_t out_stride;
    float* lse;
    int32_t q_bf16, out_bf16;
    float* part;      // partial results of items cut between CTAs (null: none is cut)
    unsigned* count;  // arrival counters, zero between calls
    unsigned* status;
};

int64_t kv_rows_workspace_bytes(int dim);
cudaError_t launch_kv_rows(const KvAttnArgs& a, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl);

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

__device__ __forceinline__ void kv_pdl_begin()
{
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- the attention kernels' work list ------------------------------------------
// An item is (request, kv head, tile of query rows): rows token * group + head,
// tiles of `R` of them.  Its units are the blocks of UT tokens that any of its
// rows sees (one unit when it sees none, so that its rows are written).  Items
// are ordered request, head, tile; the units of all items form one list, cut
// into equal shares, one a CTA.

struct KvReq {
    int32_t seq;   // tokens in the cache
    int32_t base;  // first query row
    int32_t nq;    // query rows (tokens)
};

__device__ __forceinline__ KvReq kv_req(const KvAttnArgs& a, int r)
{
    KvReq q;
    int32_t b, e;
    if (a.q_start) {
        b = a.q_start[r];
        e = a.q_start[r + 1];
    } else {
        b = r * a.q_per_req;
        e = b + a.q_per_req;
    }
    b = min(max(b, 0), a.tokens);
    e = min(max(e, b), a.tokens);
    q.base = b;
    q.nq = e - b;
    const int64_t cap = (int64_t)a.max_blocks << a.c.page_shift;
    q.seq = (int32_t)min((int64_t)max(a.seq_len[r], 0), cap);
    return q;
}

// Whether a request is longer than its table (its end is then cut off).
__device__ __forceinline__ bool kv_too_long(const KvAttnArgs& a, int r)
{
    return (int64_t)a.seq_len[r] > (int64_t)a.max_blocks << a.c.page_shift;
}

// Units [first, first + n) of a tile of rows [row0, row0 + rows).
template <int UT>
__device__ __forceinline__ void kv_tile_units(const KvAttnArgs& a, const KvReq& q, int row0,
                                              int row1, int32_t& first, int32_t& n)
{
    const int32_t i0 = row0 / a.group, i1 = (row1 - 1) / a.group;
    const int32_t p0 = q.seq - q.nq;
    const int32_t hi = p0 + i1 + 1;  // keys [lo, hi)
    const int32_t lo = a.window > 0 ? max(0, p0 + i0 - a.window + 1) : 0;
    if (hi <= lo) {
        first = 0;
        n = 1;
        return;
    }
    first = lo / UT;
    n = (hi + UT - 1) / UT - first;
}

}  // namespace nvfp4

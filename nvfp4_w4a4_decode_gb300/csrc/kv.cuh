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
    float* part;      // partial results of items cut between CTAs (null: none is cut)
    unsigned* count;  // arrival counters, zero between calls
    unsigned* status;
};

// The workspace's arrival counters (zero between calls; both kernels' lie
// here), then partial results.
constexpr int64_t kKvCountBytes = NVFP4_KV_WORKSPACE_ZERO;

// Few query rows a request, any dtype.
int64_t kv_rows_workspace_bytes(int dim);
cudaError_t launch_kv_rows(const KvAttnArgs& a, void* workspace, int64_t workspace_bytes,
                           cudaStream_t stream, bool pdl);

// Many query rows a request (tcgen05); BF16 queries and outputs only.
int64_t kv_tile_workspace_bytes(int dim);
cudaError_t launch_kv_tile(const KvAttnArgs& a, void* workspace, int64_t workspace_bytes,
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

}  // namespace nvfp4

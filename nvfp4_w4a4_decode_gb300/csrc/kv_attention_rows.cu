// kv_attention_rows.cu -- causal attention over the paged cache, few rows a request.
#include "kv_attention_rows.cuh"

namespace nvfp4 {

// Counters, then two partial results a CTA.
int64_t kv_rows_workspace_bytes(int dim)
{
    return kKvCountBytes + (int64_t)kMaxCtas * 2 * (kMaxRows * dim + 2 * kMaxRows) * sizeof(float);
}

int kv_rows_item_rows(const KvAttnArgs& a)
{
    return item_rows(a);
}

template cudaError_t launch_kv_rows<KvSees::kCausal>(const KvAttnArgs&, void*, int64_t, cudaStream_t, bool);

}  // namespace nvfp4

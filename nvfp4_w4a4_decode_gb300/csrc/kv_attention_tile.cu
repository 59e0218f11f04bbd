// kv_attention_tile.cu -- causal attention over the paged cache, many rows a request.
#include "kv_attention_tile.cuh"

namespace nvfp4 {

// Counters (one a CTA and tile), then four partial tiles a CTA.
int64_t kv_tile_workspace_bytes(int dim)
{
    const int64_t ctas = device_sm_count(current_device());
    return kKvCountBytes + ctas * 4 * (dim + 2) * kRowsTile * (int64_t)sizeof(float);
}

int kv_tile_item_rows()
{
    return kRows;
}

template cudaError_t launch_kv_tile<KvSees::kCausal>(const KvAttnArgs&, void*, int64_t, cudaStream_t, bool);

}  // namespace nvfp4

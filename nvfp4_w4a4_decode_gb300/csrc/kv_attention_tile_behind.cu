// kv_attention_tile_behind.cu -- attention over the paged cache, many rows a request:
// keys behind a shared prefix, joined with the prefix's results.
#include "kv_attention_tile.cuh"

namespace nvfp4 {

template cudaError_t launch_kv_tile<KvSees::kBehind>(const KvAttnArgs&, void*, int64_t, cudaStream_t, bool);

}  // namespace nvfp4

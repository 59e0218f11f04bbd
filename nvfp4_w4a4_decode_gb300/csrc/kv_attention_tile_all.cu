// kv_attention_tile_all.cu -- attention over the paged cache, many rows a request:
// every row sees all keys: cross attention, shared prefixes.
#include "kv_attention_tile.cuh"

namespace nvfp4 {

template cudaError_t launch_kv_tile<KvSees::kAll>(const KvAttnArgs&, void*, int64_t, cudaStream_t, bool);

}  // namespace nvfp4

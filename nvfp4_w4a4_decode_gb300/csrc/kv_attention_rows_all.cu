// kv_attention_rows_all.cu -- attention over the paged cache, few rows a request:
// every row sees all keys: cross attention, shared prefixes.
#include "kv_attention_rows.cuh"

namespace nvfp4 {

template cudaError_t launch_kv_rows<KvSees::kAll>(const KvAttnArgs&, void*, int64_t, cudaStream_t, bool);

}  // namespace nvfp4

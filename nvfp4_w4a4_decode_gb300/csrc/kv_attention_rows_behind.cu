// kv_attention_rows_behind.cu -- attention over the paged cache, few rows a request:
// keys behind a shared prefix, joined with the prefix's results.
#include "kv_attention_rows.cuh"

namespace nvfp4 {

template cudaError_t launch_kv_rows<KvSees::kBehind>(const KvAttnArgs&, void*, int64_t, cudaStream_t, bool);

}  // namespace nvfp4

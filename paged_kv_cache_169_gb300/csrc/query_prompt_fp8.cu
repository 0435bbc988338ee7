// paged_query_attention for many rows over FP8 pools.

#include "query_prompt.cuh"

namespace kvp {

int launch_query_prompt_fp8(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream) {
    return launch_prompt_pool<KV_FP8_E4M3>(pool, p, pdl, stream);
}

}  // namespace kvp

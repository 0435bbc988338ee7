// paged_query_attention for many rows over 4-bit pools.

#include "query_prompt.cuh"

namespace kvp {

int launch_query_prompt_int4(const kv_pool* pool, const PromptArgs& p, bool pdl, cudaStream_t stream) {
    return launch_prompt_pool<KV_INT4>(pool, p, pdl, stream);
}

}  // namespace kvp

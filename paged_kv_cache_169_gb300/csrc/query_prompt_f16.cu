// paged_query_attention for many rows over float16 pools, and the choice of the kernel by pool.

#include "query_prompt.cuh"

namespace kvp {

int launch_query_prompt(const kv_pool* pool, int layer, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    PromptArgs p{};
    p.a = a;
    p.tiles = prompt_tiles(a.max_queries, a.G);
    if (pool->desc.dtype == KV_FP8_E4M3) return launch_query_prompt_fp8(pool, p, pdl, stream);
    if (pool->desc.dtype == KV_INT4) return launch_query_prompt_int4(pool, p, pdl, stream);
    if (!pool->rmaps) return KV_ERR_UNSUPPORTED;
    p.kmap = pool->rmaps[2 * layer];
    p.vmap = pool->rmaps[2 * layer + 1];
    return launch_prompt_pool<KV_F16>(pool, p, pdl, stream);
}

}  // namespace kvp

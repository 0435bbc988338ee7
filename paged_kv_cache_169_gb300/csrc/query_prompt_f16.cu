// paged_query_attention for many rows over float16 pools.

#include "query_prompt.cuh"

namespace kvp {

int launch_query_prompt_f16(const kv_pool* pool, int layer, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    if (!pool->rmaps) return KV_ERR_UNSUPPORTED;
    PromptArgs p{};
    p.kmap = pool->rmaps[2 * layer];
    p.vmap = pool->rmaps[2 * layer + 1];
    p.a = a;
    p.tiles = prompt_tiles(a.max_queries, a.G);
    return pool->desc.head_dim == 128 ? launch_prompt_typed<PromptCfg<128, KV_F16>>(pool, p, pdl, stream)
                                      : launch_prompt_typed<PromptCfg<64, KV_F16>>(pool, p, pdl, stream);
}

}  // namespace kvp

// paged_query_attention for few rows: launch.

#include "query_few.cuh"

namespace kvp {

size_t few_space(const kv_pool* pool, size_t* counters) {
    const FewSpace space(pool->num_sms, pool->desc.head_dim);
    if (counters) *counters = space.ml;
    return space.bytes;
}

int launch_query_few(const kv_pool* pool, const QueryArgs& a, void* workspace, bool pdl, cudaStream_t stream) {
    const FewSpace space(pool->num_sms, pool->desc.head_dim);
    char* const ws = static_cast<char*>(workspace);
    FewArgs x{};
    x.a = a;
    x.done = reinterpret_cast<unsigned*>(ws);
    x.group_done = x.done + 2 * pool->num_sms;
    x.part_ml = reinterpret_cast<float2*>(ws + space.ml);
    x.part_o = reinterpret_cast<float*>(ws + space.o);
    switch (pool->desc.dtype) {
        case KV_F16: return launch_few_pool<KV_F16>(pool, x, pool->num_sms, pdl, stream);
        case KV_FP8_E4M3: return launch_few_pool<KV_FP8_E4M3>(pool, x, pool->num_sms, pdl, stream);
        default: return launch_few_pool<KV_INT4>(pool, x, pool->num_sms, pdl, stream);
    }
}

}  // namespace kvp

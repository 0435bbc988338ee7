// paged_query_attention for many rows over float16 pools, and the choice of the kernel by pool.

#include "query_prompt.cuh"

namespace kvp {

int launch_query_prompt(const kv_pool* pool, int layer, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    PromptArgs p{};
    p.a = a;
    p.items = static_cast<int>(prompt_items(a.batch, a.H, a.G, a.num_tokens, a.max_queries) * a.splits);
    // queries: rows of a token are D-element heads; a box is 64 elements of the G heads of 128 / G tokens
    const kv_pool_desc& d = pool->desc;
    const TensorMapEncode encode = reinterpret_cast<TensorMapEncode>(pool->encode);
    if (!encode) return KV_ERR_UNSUPPORTED;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(d.head_dim / 64), static_cast<cuuint64_t>(a.H) * a.G,
                                static_cast<cuuint64_t>(a.num_tokens)};
    const cuuint64_t strides[3] = {128, static_cast<cuuint64_t>(d.head_dim) * 2, static_cast<cuuint64_t>(a.q_stride)};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(128 / a.G)}, estr[4] = {1, 1, 1, 1};
    if (encode(&p.qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<char*>(a.q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return KV_ERR_CUDA;
    if (pool->desc.dtype == KV_FP8_E4M3) return launch_query_prompt_fp8(pool, p, pdl, stream);
    if (pool->desc.dtype == KV_INT4) return launch_query_prompt_int4(pool, p, pdl, stream);
    if (!pool->rmaps) return KV_ERR_UNSUPPORTED;
    p.kmap = pool->rmaps[2 * layer];
    p.vmap = pool->rmaps[2 * layer + 1];
    return launch_prompt_pool<KV_F16>(pool, p, pdl, stream);
}

}  // namespace kvp

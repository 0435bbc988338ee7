// What depends on a pool's element type outside the attention kernels: the bytes of a row and of
// a block, the element types a pool takes, and the choice between the decode kernels.
#pragma once

#include "kvp_internal.cuh"

namespace kvp {

// bytes of one token of one head in a pool (KV_INT4: 4-bit codes and a scale byte per 16 elements)
inline int row_bytes(const kv_pool_desc& d) {
    return d.dtype == KV_INT4 ? d.head_dim / 2 + d.head_dim / 16 : d.head_dim * elem_bytes(d.dtype);
}

// bytes of one physical block (every head) of a layer's K or V
inline int64_t block_bytes(const kv_pool_desc& d) {
    return static_cast<int64_t>(d.num_heads) * d.block_size * row_bytes(d);
}

// element types of new K/V that a pool takes: its own, or float16 / float32 where it quantises
inline bool valid_input(kv_dtype pool, kv_dtype in) {
    if (pool == KV_FP8_E4M3 || pool == KV_INT4) return in == KV_F16 || in == KV_F32;
    return in == pool;
}

// 4-bit pools (attention_int4.cu): plan and launch of a decode call, as plan_attention and
// launch_attention_append for the other pools.
int plan_attention_int4(const kv_pool* pool, int batch, int max_context, int partition_tokens, AttnPlan* plan,
                        int group, int window);
int launch_attention_int4(const kv_pool* pool, int layer, const void* q, const void* k_new, const void* v_new,
                          int in_bytes, void* out, const int32_t* block_tables, int max_blocks,
                          const int32_t* context_lens, int batch, int max_context, float scale, const AttnPlan& plan,
                          void* workspace, cudaStream_t stream);

inline int plan_decode(const kv_pool* pool, int batch, int max_context, int partition_tokens, AttnPlan* plan,
                       int group = 1, int window = 0) {
    return pool->desc.dtype == KV_INT4
               ? plan_attention_int4(pool, batch, max_context, partition_tokens, plan, group, window)
               : plan_attention(pool, batch, max_context, partition_tokens, plan, group, window);
}

inline int launch_decode(const kv_pool* pool, int layer, const void* q, const void* k_new, const void* v_new,
                         int in_bytes, void* out, const int32_t* block_tables, int max_blocks,
                         const int32_t* context_lens, int batch, int max_context, float scale, const AttnPlan& plan,
                         void* workspace, cudaStream_t stream) {
    return (pool->desc.dtype == KV_INT4 ? launch_attention_int4 : launch_attention_append)(
        pool, layer, q, k_new, v_new, in_bytes, out, block_tables, max_blocks, context_lens, batch, max_context,
        scale, plan, workspace, stream);
}

// kv_append into a 4-bit pool, kv_append_rope, kv_gather, kv_rope_table (append_rope.cu)
int launch_append_int4(const kv_pool* pool, int layer, const void* k, const void* v, kv_dtype in_dtype,
                       const int64_t* slot_mapping, int num_tokens, cudaStream_t stream);
int launch_append_rope(const kv_pool* pool, const kv_rope_args& args);
int launch_gather(const kv_pool* pool, int layer, const int64_t* slot_mapping, int num_tokens, void* k_out,
                  void* v_out, kv_dtype out_dtype, cudaStream_t stream);
int launch_rope_table(float* table, int num_positions, int rot_dim, double base, double position_scale,
                      cudaStream_t stream);

}  // namespace kvp

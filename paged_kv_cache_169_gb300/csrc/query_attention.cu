// paged_query_attention: host side (plan, workspace, choice of kernel) and the row kernel.

#include "query_attention.cuh"

namespace kvp {
namespace {

constexpr int kRowWarps = 8;

// A warp per (row, query head), in float32 from the definition.
template <int D, kv_dtype POOL>
__global__ void __launch_bounds__(kRowWarps * 32) query_rows_kernel(const __grid_constant__ QueryArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int heads = a.H * a.G;
    const int64_t per_seq = static_cast<int64_t>(a.max_queries) * heads, all = per_seq * a.batch;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowWarps;
    #pragma unroll 1
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); u < all; u += step) {
        const int s = static_cast<int>(u / per_seq);
        const int r = static_cast<int>(u - s * per_seq);
        const int i = r / heads, head = r - i * heads;
        const QuerySeq seq = query_seq(a, s, r == 0 && (threadIdx.x & 31) == 0);
        if (i < seq.n) attend_row<D, POOL>(a, s, seq, i, head);
    }
}

template <kv_dtype POOL>
int launch_rows_typed(const kv_pool* pool, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(a.batch) * a.max_queries * a.H * a.G;
    const int64_t want = (warps + kRowWarps - 1) / kRowWarps, most = static_cast<int64_t>(pool->num_sms) * 64;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    const cudaError_t rc = pool->desc.head_dim == 128 ? cudaLaunchKernelEx(&cfg, query_rows_kernel<128, POOL>, a)
                                                      : cudaLaunchKernelEx(&cfg, query_rows_kernel<64, POOL>, a);
    if (rc != cudaSuccess) {
        cudaGetLastError();
        return KV_ERR_CUDA;
    }
    return KV_OK;
}

}  // namespace

int launch_query_rows(const kv_pool* pool, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    switch (pool->desc.dtype) {
        case KV_F32: return launch_rows_typed<KV_F32>(pool, a, pdl, stream);
        case KV_F16: return launch_rows_typed<KV_F16>(pool, a, pdl, stream);
        case KV_FP8_E4M3: return launch_rows_typed<KV_FP8_E4M3>(pool, a, pdl, stream);
        default: return launch_rows_typed<KV_INT4>(pool, a, pdl, stream);
    }
}

int plan_query(const kv_pool* pool, const kv_query_args& x, QueryPlan* plan) {
    const kv_pool_desc& d = pool->desc;
    if (x.batch < 0 || x.batch > KV_MAX_DECODE_BATCH || x.num_tokens < 0 || x.num_tokens > kMaxQueryTokens ||
        x.max_queries < 0 || x.max_queries > x.num_tokens || x.max_context < 0 || x.max_context > kMaxQueryTokens ||
        x.window < 0 || x.num_q_heads < 1 || x.num_q_heads % d.num_heads != 0)
        return KV_ERR_INVALID_ARG;
    const int g = x.num_q_heads / d.num_heads;
    if (g != 1 && g != 2 && g != 4 && g != 8) return KV_ERR_INVALID_ARG;
    if (prompt_items(x.batch, d.num_heads, g, x.num_tokens, x.max_queries) > (int64_t{1} << 30))
        return KV_ERR_INVALID_ARG;
    // float32 pools: a warp per row and head; the others by what a K/V head's rows fill: one 16-row matrix
    // product over keys that are read once, or 128-row tiles of the tensor cores
    const int64_t rows = static_cast<int64_t>(x.max_queries) * g;
    plan->kind = d.dtype == KV_F32 ? QueryPlan::ROWS : rows <= kFewRows ? QueryPlan::FEW : QueryPlan::PROMPT;
    plan->ws_bytes = 256;
    plan->counter_bytes = 0;
    if (plan->kind == QueryPlan::FEW) {
        const int64_t seqs = x.batch < kFewSeqs ? x.batch : kFewSeqs;
        if (seqs * d.num_heads * (x.max_context / 16 + 40) > (int64_t{1} << 30)) return KV_ERR_INVALID_ARG;
        plan->ws_bytes = few_space(pool, &plan->counter_bytes);
    }
    return KV_OK;
}

int launch_query(const kv_pool* pool, const kv_query_args& x, const QueryPlan& plan) {
    const kv_pool_desc& d = pool->desc;
    const int es = d.dtype == KV_F32 ? 4 : 2;
    QueryArgs a{};
    a.q = static_cast<const char*>(x.q);
    a.out = static_cast<char*>(x.out);
    a.q_stride = x.q_stride * es;
    a.out_stride = x.out_stride * es;
    a.query_start = x.query_start;
    a.tables = x.block_tables;
    a.lens = x.context_lens;
    a.slopes = x.slopes;
    a.ranges = reinterpret_cast<const int2*>(x.ranges);
    a.kpool = static_cast<const char*>(pool->k_layers[x.layer]);
    a.vpool = static_cast<const char*>(pool->v_layers[x.layer]);
    a.kscale = pool->k_scales ? pool->k_scales[x.layer] : nullptr;
    a.vscale = pool->v_scales ? pool->v_scales[x.layer] : nullptr;
    a.num_tokens = x.num_tokens;
    a.max_queries = x.max_queries;
    a.max_blocks = x.max_blocks_per_seq;
    a.batch = x.batch;
    const int64_t table_tokens = static_cast<int64_t>(x.max_blocks_per_seq) * d.block_size;
    a.ctx_limit = static_cast<int>(table_tokens < x.max_context ? table_tokens : x.max_context);
    a.window = x.window;
    a.H = d.num_heads;
    a.G = x.num_q_heads / d.num_heads;
    a.B = d.block_size;
    a.log_b = d.block_size == 8 ? 3 : d.block_size == 16 ? 4 : 5;
    a.num_blocks = d.num_blocks;
    a.scale = x.scale;
    a.cap = x.score_cap;
    a.err = pool->d_err;
    const bool pdl = (x.flags & KV_DECODE_PDL) != 0;
    const cudaStream_t stream = static_cast<cudaStream_t>(x.stream);
    // (every launch leaves its counters zero)
    if (plan.counter_bytes && !(x.flags & KV_DECODE_WORKSPACE_ZEROED) &&
        cudaMemsetAsync(x.workspace, 0, plan.counter_bytes, stream) != cudaSuccess)
        return KV_ERR_CUDA;
    switch (plan.kind) {
        case QueryPlan::ROWS: return launch_query_rows(pool, a, pdl, stream);
        case QueryPlan::FEW: return launch_query_few(pool, a, x.workspace, pdl, stream);
        default: return launch_query_prompt(pool, x.layer, a, pdl, stream);
    }
}

}  // namespace kvp

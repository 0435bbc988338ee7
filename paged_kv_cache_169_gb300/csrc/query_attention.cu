// paged_query_attention: host side (plan, workspace, choice of kernel) and the row kernel.

#include "query_attention.cuh"

namespace kvp {
namespace {

constexpr int kRowWarps = 8;

// R rows of K/V head h (row r: token r / G, query head h G + r % G) from r0 on, by one warp, in float32 from the
// definition: only what a row sees is read for it.  Eight lanes share a key (lane t of them has the t-th 16 bytes of every
// 128), four keys go side by side with a softmax state each, joined at the end.
template <int D, int R>
__device__ __forceinline__ void attend_rows(const QueryArgs& a, int s, QuerySeq seq, int h, int r0) {
    constexpr int N = D / 8;
    const int lane = threadIdx.x & 31, part = lane & 7, which = lane >> 3;
    auto load_parts = [&](const char* row, float (&x)[N]) {
        #pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(row + part * 16 + e * 32);
            x[e] = f.x; x[e + 1] = f.y; x[e + 2] = f.z; x[e + 3] = f.w;
        }
    };
    int2 range[R];
    int lo = 1 << 30, hi = 0, pos[R];
    float q[R][N], o[R][N], m[R], l[R], slope[R];
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = (r0 + r) / a.G, head = h * a.G + (r0 + r) % a.G;
        const bool some = i < seq.n;
        range[r] = some ? row_range(a, seq, i) : make_int2(0, 0);
        if (range[r].x < range[r].y) {
            lo = min(lo, range[r].x);
            hi = max(hi, range[r].y);
        }
        pos[r] = seq.ctx - seq.n + i;
        slope[r] = a.slopes ? a.slopes[head] : 0.f;
        m[r] = -CUDART_INF_F;
        l[r] = 0.f;
        load_parts(a.q + static_cast<int64_t>(seq.first + (some ? i : 0)) * a.q_stride + head * (D * 4), q[r]);
        #pragma unroll
        for (int e = 0; e < N; ++e) o[r][e] = 0.f;
    }
    auto seen_by = [&](int r, int j) { return j >= range[r].x && j < range[r].y; };
    auto any_sees = [&](int j) {
        bool any = false;
        #pragma unroll
        for (int r = 0; r < R; ++r) any |= seen_by(r, j);
        return any;
    };
    // (a key's block is looked up an iteration ahead)
    auto look_up = [&](int j) { return any_sees(j) ? query_block(a, s, j) : -1; };
    int next = look_up(lo + which);
    #pragma unroll 1
    for (int j0 = lo; j0 < hi; j0 += 4) {
        const int j = j0 + which, id = next;
        next = look_up(j + 4);
        float x[N], v[N], dot[R];
        #pragma unroll
        for (int r = 0; r < R; ++r) dot[r] = 0.f;
        if (id >= 0) {
            const int64_t at = ((static_cast<int64_t>(id) * a.H + h) * a.B + (j & (a.B - 1))) * (D * 4);
            load_parts(a.kpool + at, x);
            load_parts(a.vpool + at, v);
            #pragma unroll
            for (int r = 0; r < R; ++r)
                #pragma unroll
                for (int e = 0; e < N; ++e) dot[r] = fmaf(q[r][e], x[e], dot[r]);
        }
        #pragma unroll
        for (int k = 1; k < 8; k *= 2)
            #pragma unroll
            for (int r = 0; r < R; ++r) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], k);
        #pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!seen_by(r, j)) continue;
            float t = dot[r] * a.scale;
            if (a.cap > 0.f) t = a.cap * tanhf(t / a.cap);
            if (a.slopes) t = fmaf(-slope[r], static_cast<float>(abs(pos[r] - j)), t);
            t *= kLog2e;
            if (t > m[r]) {                                    // (rare after the first keys; NaN: it reaches the weight)
                const float keep = ex2_approx(m[r] - t);
                m[r] = t;
                l[r] *= keep;
                #pragma unroll
                for (int e = 0; e < N; ++e) o[r][e] *= keep;
            }
            const float w = ex2_approx(t - (m[r] == -CUDART_INF_F ? 0.f : m[r]));
            l[r] += w;
            #pragma unroll
            for (int e = 0; e < N; ++e) o[r][e] = fmaf(w, v[e], o[r][e]);
        }
    }
    #pragma unroll
    for (int r = 0; r < R; ++r) {
        #pragma unroll
        for (int k = 8; k < 32; k *= 2) {
            const float other = __shfl_xor_sync(0xffffffffu, m[r], k);
            const float to = fmaxf(m[r], other), base = to == -CUDART_INF_F ? 0.f : to;
            const float mine = ex2_approx(m[r] - base), theirs = ex2_approx(other - base);
            l[r] = l[r] * mine + __shfl_xor_sync(0xffffffffu, l[r], k) * theirs;
            #pragma unroll
            for (int e = 0; e < N; ++e) o[r][e] = o[r][e] * mine + __shfl_xor_sync(0xffffffffu, o[r][e], k) * theirs;
            m[r] = to;
        }
        const int i = (r0 + r) / a.G;
        if (which != 0 || i >= seq.n) continue;
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        char* row = a.out + static_cast<int64_t>(seq.first + i) * a.out_stride + (h * a.G + (r0 + r) % a.G) * (D * 4) + part * 16;
        #pragma unroll
        for (int e = 0; e < N; e += 4)
            *reinterpret_cast<float4*>(row + e * 32) = make_float4(o[r][e] * inv, o[r][e + 1] * inv, o[r][e + 2] * inv, o[r][e + 3] * inv);
    }
}

// float32 pools: a warp per R rows of a K/V head, in float32 from the definition.  Bound: the FMA pipe, 4 D operations a
// pair, at 0.15 of its rate for the latency of the loads (4 prompts of 2048 tokens, 40 heads: 14.9 ms; a row per warp
// 41.9, four rows, whose registers leave one CTA per SM, 19.1).  R: 2, or 1 where a K/V head has a single row.
template <int D, int R>
__global__ void __launch_bounds__(kRowWarps * 32, 2) query_rows_kernel(const __grid_constant__ QueryArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per_head = (a.max_queries * a.G + R - 1) / R;
    const int64_t per_seq = static_cast<int64_t>(per_head) * a.H, all = per_seq * a.batch;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowWarps;
    #pragma unroll 1
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); u < all; u += step) {
        const int s = static_cast<int>(u / per_seq);
        const int64_t at = u - s * per_seq;
        const int h = static_cast<int>(at / per_head), r0 = static_cast<int>(at - static_cast<int64_t>(h) * per_head) * R;
        const QuerySeq seq = query_seq(a, s, at == 0 && (threadIdx.x & 31) == 0);
        if (r0 < seq.n * a.G) attend_rows<D, R>(a, s, seq, h, r0);
    }
}

template <int R>
int launch_rows(const kv_pool* pool, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(a.batch) * a.H * ((static_cast<int64_t>(a.max_queries) * a.G + R - 1) / R);
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
    const cudaError_t rc = pool->desc.head_dim == 128 ? cudaLaunchKernelEx(&cfg, query_rows_kernel<128, R>, a)
                                                      : cudaLaunchKernelEx(&cfg, query_rows_kernel<64, R>, a);
    if (rc != cudaSuccess) {
        cudaGetLastError();
        return KV_ERR_CUDA;
    }
    return KV_OK;
}

int launch_query_rows(const kv_pool* pool, const QueryArgs& a, bool pdl, cudaStream_t stream) {
    return static_cast<int64_t>(a.max_queries) * a.G > 1 ? launch_rows<2>(pool, a, pdl, stream)
                                                         : launch_rows<1>(pool, a, pdl, stream);
}

}  // namespace

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
    plan->splits = 1;
    plan->part_rows = 0;
    plan->part_by_sequence = false;
    size_t counters;
    const size_t few_bytes = few_space(pool, &counters);
    if (plan->kind == QueryPlan::PROMPT) {
        const QueryParts parts = query_parts(pool->num_sms, x.batch, d.num_heads, g, x.num_tokens, x.max_queries, x.max_context,
                                             x.window);
        plan->splits = parts.splits;
        plan->part_rows = parts.rows;
        plan->part_by_sequence = parts.by_sequence;
        // Behind the few-row kernel's counters, which stay zero; and what that kernel needs, so that a workspace for many
        // rows serves the calls of few that come between.
        const size_t part_bytes = counters + static_cast<size_t>(parts.space) * (d.head_dim * 4 + 8);
        plan->ws_bytes = part_bytes > few_bytes ? part_bytes : few_bytes;
    }
    if (plan->kind == QueryPlan::FEW) {
        const int64_t seqs = x.batch < kFewSeqs ? x.batch : kFewSeqs;
        if (seqs * d.num_heads * (x.max_context / 16 + 40) > (int64_t{1} << 30)) return KV_ERR_INVALID_ARG;
        plan->ws_bytes = few_bytes;
        plan->counter_bytes = counters;
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
    a.window = x.window < 2 * kMaxQueryTokens ? x.window : 2 * kMaxQueryTokens;            // (a row may stand at -2^24)
    a.H = d.num_heads;
    a.G = x.num_q_heads / d.num_heads;
    a.B = d.block_size;
    a.log_b = d.block_size == 8 ? 3 : d.block_size == 16 ? 4 : 5;
    a.num_blocks = d.num_blocks;
    a.scale = x.scale;
    a.cap = x.score_cap;
    a.splits = plan.splits;
    size_t counters;
    few_space(pool, &counters);
    a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(x.workspace) + counters);
    a.part_o = reinterpret_cast<float*>(a.part_ml + plan.splits * plan.part_rows * x.num_q_heads);
    a.part_rows = plan.part_rows;
    a.part_by_sequence = plan.part_by_sequence;
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

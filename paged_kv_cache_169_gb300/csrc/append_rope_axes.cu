// kv_append_rope_axes: the rotated append for positions with several axes.

#include "append_rope_kernel.cuh"

namespace kvp {

int launch_rope_axes_any(const kv_pool* pool, kv_dtype in, const RopeArgs& a, bool pdl, cudaStream_t stream) {
    return launch_rope_types<true>(pool, in, a, pdl, stream);
}

}  // namespace kvp

// pa_decode_sinks.cu -- instances of the tile-ring decode kernel for
// pa_decode_sinks: a window and the first rows (bf16: up to 8 query columns, heads per
// KV head x query tokens; fp32: 1, 2, 4 or 8 heads per KV head, one query token).
#include "pa_decode_rows_ring.cuh"

namespace pa {

cudaError_t launch_decode_sinks(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                                pa_dtype dtype, int sm_count, cudaStream_t stream) {
    return launch_rows_ring<false>(tk, tv, p, dtype, sm_count, stream);
}

bool has_rows_instance(pa_dtype dtype, int head_dim, int group, int num_queries) {
    if (head_dim != 64 && head_dim != 128) return false;
    if (dtype == PA_DTYPE_BF16) return group * num_queries <= 8;
    return num_queries == 1 && (group == 1 || group == 2 || group == 4 || group == 8);
}

}  // namespace pa

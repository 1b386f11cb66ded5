// pa_decode_sinks.cu -- instances of the tile-ring decode kernel for
// pa_decode_sinks: a window and the first rows. Up to 8 heads per KV head; bf16: the query
// tokens of an item fill up to 8 columns, further ones are another item's, whose K and V
// tiles the first one has brought into L2; fp32: one query token.
//
// 128 sequences of 1,640 rows, 32 query heads over 8 KV heads of 128, window 1,024 and 4 first
// rows, bf16: 86 us with the merge, 465 MB, bound by memory (5.7 TB/s between the ring's
// start, 6 us, and the merge, 4); the plain kernel took 1,056.
#include "pa_decode_rows_ring.cuh"

namespace pa {

cudaError_t launch_decode_sinks(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                                pa_dtype dtype, int sm_count, cudaStream_t stream) {
    return launch_rows_ring<false>(tk, tv, p, dtype, sm_count, stream);
}

int rows_group_tokens(pa_dtype dtype, int head_dim, int group, int num_queries) {
    if ((head_dim != 64 && head_dim != 128) || group > 8) return 0;
    if (dtype != PA_DTYPE_BF16) return num_queries == 1 ? 1 : 0;
    const int tokens = 8 / group;
    return tokens < num_queries ? tokens : num_queries;
}

}  // namespace pa

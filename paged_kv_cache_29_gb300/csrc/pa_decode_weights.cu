// pa_decode_weights.cu -- instances of the tile-ring decode kernel for
// pa_decode_weights: the scores of every row go to the workspace (shapes as in
// pa_decode_sinks.cu).
//
// 128 sequences of 1,640 rows, 32 query heads over 8 KV heads of 128, bf16: 152 us (6.1 TB/s of
// DRAM traffic, bound by memory; 5 us of it for the stores of 27 MB of scores), 168 with the merge and
// row_weights_kernel.
#include "pa_decode_rows_ring.cuh"

namespace pa {

cudaError_t launch_decode_weights(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                                  pa_dtype dtype, int sm_count, cudaStream_t stream) {
    return launch_rows_ring<true>(tk, tv, p, dtype, sm_count, stream);
}

}  // namespace pa

// pa_decode_weights.cu -- instances of the tile-ring decode kernel for
// pa_decode_weights: the scores of every row go to the workspace (shapes as in
// pa_decode_sinks.cu).
#include "pa_decode_rows_ring.cuh"

namespace pa {

cudaError_t launch_decode_weights(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                                  pa_dtype dtype, int sm_count, cudaStream_t stream) {
    return launch_rows_ring<true>(tk, tv, p, dtype, sm_count, stream);
}

}  // namespace pa

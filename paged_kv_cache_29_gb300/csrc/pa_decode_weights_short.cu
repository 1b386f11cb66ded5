// pa_decode_weights_short.cu -- instances of the tile-ring decode kernel for
// pa_decode_weights where every sequence has one partition: each item's end adds its row
// weights (shapes as in pa_decode_sinks.cu).
#include "pa_decode_rows_ring.cuh"

namespace pa {

cudaError_t launch_decode_weights_short(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                                        pa_dtype dtype, int sm_count, cudaStream_t stream) {
    return launch_rows_ring<true, true>(tk, tv, p, dtype, sm_count, stream);
}

}  // namespace pa

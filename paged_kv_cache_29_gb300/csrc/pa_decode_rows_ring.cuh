// pa_decode_rows_ring.cuh -- choice of the tile-ring instance for pa_decode_sinks and
// pa_decode_weights by head dim and query columns.
#pragma once

#include "pa_decode_stream.cuh"
#include "pa_tile_math_rows.cuh"

namespace pa {

namespace {
constexpr int kWarps = 4;            // consumer warps and CTAs per SM as the plain decode
constexpr int kMinCtasPerSm = 4;     // kernels have them (pa_decode_mma.cu, pa_decode_simt.cu)

// Ring stages over bf16: 32 KB of tiles on their way to each CTA (8 KV heads, 210,000 rows of 64
// dims: 1, 4 and 8 heads each 95, 101, 110 us with eight stages, 108, 115, 124 with four).
template <int D>
constexpr int kMmaStages = (D == 64 ? 2 : 1) * kWarps;

// Ring stages over fp32. Where registers or 64 dims leave room for them more than a tile a warp is on its way
// (8 KV heads, 210,000 rows of 64 dims: 1, 2, 4 and 8 heads each 154, 165, 302, 483 us with 12
// stages, 186, 224, 447, 623 with four; 105,000 rows of 128 dims, 4 and 8 heads 282 and 556 with
// eight, 365 and 624 with four, but 1 and 2 heads 156 and 192 instead of 149 and 175).
template <int D, int G>
constexpr int kSimtStages = (D == 64 ? 3 : G >= 4 ? 2 : 1) * kWarps;

template <int D, int G, bool SCORES, bool ENDS>
cudaError_t run_mma(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, int sm_count,
                    cudaStream_t stream) {
    return launch_stream_instance<RowsMmaMath<D, G, SCORES, ENDS>, D, G, kWarps, kMmaStages<D>, kMinCtasPerSm, false>(
        tk, tv, p, sm_count, stream);
}

template <int D, int G, bool SCORES, bool ENDS>
cudaError_t run_simt(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, int sm_count,
                     cudaStream_t stream) {
    return launch_stream_instance<RowsSimtMath<D, G, SCORES, ENDS>, D, G, kWarps, kSimtStages<D, G>, 1, false>(
        tk, tv, p, sm_count, stream);
}

template <int D, bool SCORES, bool ENDS>
cudaError_t by_columns(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, pa_dtype dtype,
                       int sm_count, cudaStream_t stream) {
    const int cols = (p.num_heads / p.num_kv_heads) * p.group_tokens;
    const bool bf16 = dtype == PA_DTYPE_BF16;
    if (cols <= 1) return bf16 ? run_mma<D, 1, SCORES, ENDS>(tk, tv, p, sm_count, stream)
                               : run_simt<D, 1, SCORES, ENDS>(tk, tv, p, sm_count, stream);
    if (cols <= 2) return bf16 ? run_mma<D, 2, SCORES, ENDS>(tk, tv, p, sm_count, stream)
                               : run_simt<D, 2, SCORES, ENDS>(tk, tv, p, sm_count, stream);
    if (cols <= 4) return bf16 ? run_mma<D, 4, SCORES, ENDS>(tk, tv, p, sm_count, stream)
                               : run_simt<D, 4, SCORES, ENDS>(tk, tv, p, sm_count, stream);
    return bf16 ? run_mma<D, 8, SCORES, ENDS>(tk, tv, p, sm_count, stream)
                : run_simt<D, 8, SCORES, ENDS>(tk, tv, p, sm_count, stream);
}

template <bool SCORES, bool ENDS = false>
cudaError_t launch_rows_ring(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, pa_dtype dtype,
                             int sm_count, cudaStream_t stream) {
    return p.head_dim == 64 ? by_columns<64, SCORES, ENDS>(tk, tv, p, dtype, sm_count, stream)
                            : by_columns<128, SCORES, ENDS>(tk, tv, p, dtype, sm_count, stream);
}
}  // namespace

}  // namespace pa

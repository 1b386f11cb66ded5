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

// Ring stages and CTAs per SM over fp32, whose tiles take twice the room: bound by the consumers'
// latencies from four heads per KV head on, they need warps more than tiles on their way (8 KV
// heads, 105,000 rows of 128 dims: 1, 2, 4 and 8 heads 150, 169, 230, 377 us with four stages in two CTAs,
// 158, 182, 269, 498 with eight in one; 210,000 rows of 64 dims 153, 177, 246, 373 us as they stand here,
// 157, 197, 246, 381 with eight stages in three CTAs, 153, 216, 280, 390 with twelve in two).
template <int D, int G>
constexpr int kSimtStages = (D == 128 || G == 2 ? 1 : G == 1 ? 3 : 2) * kWarps;
template <int D, int G>
constexpr int kSimtCtas = D == 64 && (G == 2 || G == 4) ? 3 : 2;

template <int D, int G, bool SCORES, bool ENDS>
cudaError_t run_mma(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, int sm_count,
                    cudaStream_t stream) {
    return launch_stream_instance<RowsMmaMath<D, G, SCORES, ENDS>, D, G, kWarps, kMmaStages<D>, kMinCtasPerSm, false>(
        tk, tv, p, sm_count, stream);
}

template <int D, int G, bool SCORES, bool ENDS>
cudaError_t run_simt(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, int sm_count,
                     cudaStream_t stream) {
    return launch_stream_instance<RowsSimtMath<D, G, SCORES, ENDS>, D, G, kWarps, kSimtStages<D, G>, kSimtCtas<D, G>, false>(
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

// pa_tile_math_rows.cuh -- tile math of pa_decode_sinks and pa_decode_weights:
// the plain decode's products and softmax with a mask per query token.
//
// Query token j of a sequence of n rows sees row r when r <= last(j) = n - Q + j and
// r < num_sinks or r > last(j) - window. Nearly every tile is seen whole by all
// tokens; the others (the one that the window begins in, the last one, a last
// tile of first rows) mask scores, and take the products with V a token at a time, over
// the rows that it sees: 0 * NaN would reach the other tokens' sums. With SCORES every row's scores go
// to p.scores, for the row weights.
#pragma once

#include "pa_tile_math.cuh"

namespace pa {

// Bit i: token with last row `last` sees row row0 + i (16 rows).
__device__ __forceinline__ uint32_t rows_seen(int row0, int last, int window, int sinks) {
    auto below = [](int k) -> uint32_t { return k <= 0 ? 0u : k >= kTileRows ? 0xffffu : (1u << k) - 1u; };
    uint32_t seen = below(last + 1 - row0);
    if (window > 0) seen &= below(sinks - row0) | ~below(last + 1 - window - row0);
    return seen;
}

// bf16 tensor-core products, up to G query columns.
template <int D, int G, bool SCORES>
struct RowsMmaMath : MmaMath<D, G, true> {
    using Base = MmaMath<D, G, true>;
    static constexpr bool kRows = true;
    using Base::gid;
    using Base::t4;

    float* scores;                // of the item's sequence and KV head, [row][cols]
    int cols, tokens, window, sinks;

    __device__ __forceinline__ void begin_rows(const DecodeParams& p, int s, int h, int ncols) {
        cols = ncols;
        tokens = p.num_queries;
        window = p.window > 0 ? p.window - p.num_queries + 1 : 0;   // of one token
        sinks = p.num_sinks;
        if constexpr (SCORES)
            scores = p.scores + (static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows * ncols;
    }

    __device__ __forceinline__ void tile(uint32_t kbase, uint32_t vbase, int /*valid*/,
                                         float scale_log2, int lane, int row0, int limit0, int grp,
                                         int /*skip*/, uint32_t /*xb: none*/) {
        float c[4];
        Base::qk(kbase, scale_log2, lane, c);
        const bool whole = row0 + kTileRows - 1 <= limit0 &&
                           (window == 0 || row0 + kTileRows <= sinks || row0 > limit0 + tokens - 1 - window);
        if (!whole) {
            const uint32_t s0 = rows_seen(row0, limit0 + (2 * t4) / grp, window, sinks) >> gid;
            const uint32_t s1 = rows_seen(row0, limit0 + (2 * t4 + 1) / grp, window, sinks) >> gid;
            if (!(s0 & 1u)) c[0] = -INFINITY;
            if (!(s1 & 1u)) c[1] = -INFINITY;
            if (!(s0 & 256u)) c[2] = -INFINITY;
            if (!(s1 & 256u)) c[3] = -INFINITY;
        }
        if constexpr (SCORES) {
            // Rows past the sequence too: the scratch has whole tiles.
            if (G > 1 && cols == G) {
                float* at = scores + static_cast<size_t>(row0 + gid) * G + 2 * t4;
                if (2 * t4 < G) {
                    *reinterpret_cast<float2*>(at) = make_float2(c[0], c[1]);
                    *reinterpret_cast<float2*>(at + 8 * G) = make_float2(c[2], c[3]);
                }
            } else {
                float* at = scores + static_cast<size_t>(row0 + gid) * cols + 2 * t4;
                if (2 * t4 < cols) {
                    at[0] = c[0];
                    at[8 * cols] = c[2];
                }
                if (2 * t4 + 1 < cols) {
                    at[1] = c[1];
                    at[8 * cols + 1] = c[3];
                }
            }
        }
        uint32_t b0, b1;
        Base::softmax(c, b0, b1);
        if (whole) {
            Base::pv(vbase, lane, b0, b1);
        } else if (tokens == 1) {
            Base::pv_rows(vbase, lane, b0, b1, rows_seen(row0, limit0, window, sinks));
        } else {
            // Each token's columns with the rows that it sees.
            for (int j = 0; j < tokens; ++j) {
                const uint32_t seen = rows_seen(row0, limit0 + j, window, sinks);
                if (seen != 0u)
                    Base::template pv_rows<true>(vbase, lane, b0, b1, seen, (2 * t4) / grp == j, (2 * t4 + 1) / grp == j);
            }
        }
    }
};

// fp32 on the CUDA cores, G query heads of one token.
template <int D, int G, bool SCORES>
struct RowsSimtMath : SimtMath<float, D, G> {
    using Base = SimtMath<float, D, G>;
    static constexpr bool kRows = true;

    float* scores;
    int window, sinks;

    __device__ __forceinline__ void begin_rows(const DecodeParams& p, int s, int h, int /*ncols: G*/) {
        window = p.window;
        sinks = p.num_sinks;
        if constexpr (SCORES)
            scores = p.scores + (static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows * G;
    }

    __device__ __forceinline__ void tile(uint32_t kbase, uint32_t vbase, int /*valid*/,
                                         float /*scale_log2*/, int /*lane*/, int row0, int limit0,
                                         int /*grp*/, int /*skip*/, uint32_t /*xb: none*/) {
        Base::fold(kbase, vbase, rows_seen(row0, limit0, window, sinks), [&](int row, const float (&sc)[G]) {
            if constexpr (SCORES) {
                if (Base::ch == 0) {
#pragma unroll
                    for (int g = 0; g < G; ++g) scores[static_cast<size_t>(row0 + row) * G + g] = sc[g];
                }
            }
        });
    }
};

}  // namespace pa

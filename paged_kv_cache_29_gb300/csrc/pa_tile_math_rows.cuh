// pa_tile_math_rows.cuh -- tile math of pa_decode_sinks and pa_decode_weights:
// the plain decode's products and softmax with a mask per query token.
//
// Query token j of a sequence of n rows sees row r when r <= last(j) = n - Q + j and
// r < num_sinks or r > last(j) - window. Nearly every tile is seen whole by all
// tokens; the others (the one that the window begins in, the last one, a last
// tile of first rows) mask scores, and take the products with V a token at a time, over
// the rows that it sees: 0 * NaN would reach the other tokens' sums. With SCORES every row's scores go
// to p.scores, for the row weights; with ENDS too an item's end adds them.
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

// The row weights of a sequence of one partition, by the CTA's consumer warps at its
// item's end: the columns' maxima and sums are those of the CTA's W warps (states of STATE
// floats, maxima then sums of G columns, in `buf`), the scores its own. For calls
// whose sequences all have one partition: a sequence of 17 rows takes 8.5 us, 10.5 with
// row_weights_kernel behind the decode kernel. In an instance for longer sequences
// it costs registers that their tiles need (128 sequences of 1,640 rows: 182 us instead of 171).
template <int W, int STATE, int G>
__device__ __forceinline__ void item_row_weights(const DecodeParams& p, const float* buf, int s, int h, int n, int cols) {
    float M[G], R[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        M[g] = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M[g] = fmaxf(M[g], buf[w * STATE + g]);
        M[g] = g < cols && M[g] != -INFINITY ? M[g] : 0.f;
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) L = fmaf(fast_exp2(buf[w * STATE + g] - M[g]), buf[w * STATE + G + g], L);
        R[g] = 1.f / L;
    }
    const int bs = p.block_size, grp = p.num_heads / p.num_kv_heads;
    const int32_t* table = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    const float* scores = p.scores + (static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows * cols;
    for (int i = threadIdx.x; i < n; i += W * 32) {
        const int b = i / bs;
        float* at = p.row_weights + (static_cast<size_t>(__ldg(table + b)) * p.num_kv_heads + h) * bs + (i - b * bs);
        const int first = max(0, i - (n - p.num_queries)) * grp;   // column of a token that sees the row (another's sum may be NaN)
        float w = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (g < cols && g >= first) w = fmaf(fast_exp2(scores[static_cast<size_t>(i) * cols + g] - M[g]), R[g], w);
        if (i >= n - p.num_queries)
            *at = w;
        else
            atomicAdd(at, w);
    }
}

// bf16 tensor-core products, up to G query columns.
template <int D, int G, bool SCORES, bool ENDS>
struct RowsMmaMath : MmaMath<D, G, true> {
    using Base = MmaMath<D, G, true>;
    static constexpr bool kRows = true;
    static constexpr bool kScores = SCORES;       // every row's scores are stored
    static constexpr bool kEnds = ENDS;           // an item's end adds its row weights
    using Base::gid;
    using Base::t4;

    float* scores;                // of the item's sequence, KV head and first column, [row][all columns]
    int cols, all_cols, tokens, window, sinks;

    // q of an item (head: with its column group), up to all its columns.
    __device__ __forceinline__ void stage_q(const DecodeParams& p, int s, int head, int /*all columns*/, int grp,
                                            uint32_t qbuf, int lane) const {
        const int h = head / p.col_groups, token0 = (head - h * p.col_groups) * p.group_tokens;
        stage_q_rows<D, Base::kQRowBytes>(p, s, h, grp * min(p.group_tokens, p.num_queries - token0), grp, qbuf, lane,
                                          token0 * grp);
    }

    template <int W, int STATE>
    __device__ __forceinline__ void end_rows(const DecodeParams& p, const float* buf, int s, int h, int n, int ncols) const {
        item_row_weights<W, STATE, G>(p, buf, s, h, n, ncols);
    }

    __device__ __forceinline__ void begin_rows(const DecodeParams& p, int s, int h, int token0, int ncols, int grp, float* /*scratch*/) {
        cols = ncols;
        if constexpr (!SCORES) {                  // (pa_decode_weights has no window)
            window = p.window > 0 ? p.window - p.num_queries + 1 : 0;   // of one token
            sinks = p.num_sinks;
            tokens = ncols / grp;
        } else {
            all_cols = grp * p.num_queries;
            scores = p.scores + (static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows * all_cols + token0 * grp;
        }
    }

    __device__ __forceinline__ void tile(uint32_t kbase, uint32_t vbase, int /*valid*/,
                                         float scale_log2, int lane, int row0, int limit0, int grp,
                                         int /*skip*/, uint32_t /*xb: none*/) {
        float c[4];
        Base::qk(kbase, scale_log2, lane, c);
        const bool whole = row0 + kTileRows - 1 <= limit0 &&
                           (SCORES || window == 0 || row0 + kTileRows <= sinks || row0 > limit0 + tokens - 1 - window);
        auto seen_by = [&](int last) { return SCORES ? rows_seen(row0, last, 0, 0) : rows_seen(row0, last, window, sinks); };
        if (!whole) {
            const uint32_t s0 = seen_by(limit0 + (2 * t4) / grp) >> gid;
            const uint32_t s1 = seen_by(limit0 + (2 * t4 + 1) / grp) >> gid;
            if (!(s0 & 1u)) c[0] = -INFINITY;
            if (!(s1 & 1u)) c[1] = -INFINITY;
            if (!(s0 & 256u)) c[2] = -INFINITY;
            if (!(s1 & 256u)) c[3] = -INFINITY;
        }
        if constexpr (SCORES) {
            // Rows past the sequence too: the scratch has whole tiles.
            if (G > 1 && all_cols == G) {
                float* at = scores + static_cast<size_t>(row0 + gid) * G + 2 * t4;
                if (2 * t4 < G) {
                    *reinterpret_cast<float2*>(at) = make_float2(c[0], c[1]);
                    *reinterpret_cast<float2*>(at + 8 * G) = make_float2(c[2], c[3]);
                }
            } else {
                float* at = scores + static_cast<size_t>(row0 + gid) * all_cols + 2 * t4;
                if (2 * t4 < cols) {
                    at[0] = c[0];
                    at[8 * all_cols] = c[2];
                }
                if (2 * t4 + 1 < cols) {
                    at[1] = c[1];
                    at[8 * all_cols + 1] = c[3];
                }
            }
        }
        uint32_t b0, b1;
        Base::softmax(c, b0, b1);
        if (whole) {
            Base::pv(vbase, lane, b0, b1);
        } else if (cols == grp) {
            Base::pv_rows(vbase, lane, b0, b1, seen_by(limit0));
        } else {
            // Each token's columns with the rows that it sees.
            for (int j = 0; j * grp < cols; ++j) {
                const uint32_t seen = seen_by(limit0 + j);
                if (seen != 0u)
                    Base::template pv_rows<true>(vbase, lane, b0, b1, seen, (2 * t4) / grp == j, (2 * t4 + 1) / grp == j);
            }
        }
    }
};

// fp32 on the CUDA cores, up to G query heads of one token.
//
// A row is split over LPR lanes, 16 bytes each; a warp takes RPP rows a pass. The lanes' parts of LPR
// scores (of S passes and G heads) are added up by halves: each step a lane hands over half of its
// scores and adds the other half's, so that every lane ends with one score (a butterfly for each
// score took five times the shuffles). Maxima and sums are kept by the lanes of a head's scores, weights
// pass through shared memory to the products with V.
template <int D, int G, bool SCORES, bool ENDS>
struct RowsSimtMath {
    using T = float;
    static constexpr bool kRows = true;
    static constexpr bool kScores = SCORES;
    static constexpr bool kEnds = ENDS;
    static constexpr bool kCausal = true;         // columns are the item's, not G of them
    static constexpr bool kQuantAppend = false;
    static constexpr int kExtraStageBytes = 0;
    static constexpr bool kQInSmem = false;
    static constexpr int kQBufBytes = 0;
    using Geom = TileGeom<T, D>;
    static constexpr int kLpr = D / 4;            // lanes per row
    static constexpr int kRpp = 32 / kLpr;        // rows per pass
    static constexpr int kPasses = kTileRows / kRpp;
    static constexpr int kSub = kPasses < kLpr / G ? kPasses : kLpr / G;   // passes of a sum by halves
    static constexpr int kSubs = kPasses / kSub;
    static constexpr int kScoresOf = kSub * G;    // scores of one
    static constexpr int kTwins = kLpr / kScoresOf;   // lanes with the same score

    struct QRegs {
        float f[G][4];
    };

    float qf[G][4], o[G][4];
    float m, l;                   // of the lane's head; l: of the lane's scores
    int rr, ch, own;              // row of a pass, chunk, the lane's score of a sum: pass own / G, head own % G
    float* scores;                // of the item's sequence and KV head
    float* weights;               // [row][head] of the warp's tile, in shared memory
    int cols, window, sinks;

    __device__ __forceinline__ void setup(int lane, const DecodeParams&) {
        rr = lane / kLpr;
        ch = lane % kLpr;
        own = ch / kTwins;
    }

    // The group's q rows; a column past them is zero.
    __device__ __forceinline__ void load_q(const DecodeParams& p, int s, int h, QRegs& r) const {
        const int grp = p.num_heads / p.num_kv_heads;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (g < grp)
                x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (static_cast<size_t>(s) * p.num_heads + h * grp + g) * D) + ch);
            r.f[g][0] = x.x * p.scale_log2;
            r.f[g][1] = x.y * p.scale_log2;
            r.f[g][2] = x.z * p.scale_log2;
            r.f[g][3] = x.w * p.scale_log2;
        }
    }

    __device__ __forceinline__ void begin(const DecodeParams&, const QRegs& r) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                qf[g][e] = r.f[g][e];
                o[g][e] = 0.f;
            }
        m = -INFINITY;
        l = 0.f;
    }

    template <int W, int STATE>
    __device__ __forceinline__ void end_rows(const DecodeParams& p, const float* buf, int s, int h, int n, int ncols) const {
        item_row_weights<W, STATE, G>(p, buf, s, h, n, ncols);
    }

    __device__ __forceinline__ void begin_rows(const DecodeParams& p, int s, int h, int /*token0: 0*/, int ncols, int /*grp*/, float* scratch) {
        cols = ncols;
        window = p.window;
        sinks = p.num_sinks;
        weights = scratch;
        if constexpr (SCORES)
            scores = p.scores + (static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows * ncols;
    }

    __device__ __forceinline__ void tile(uint32_t kbase, uint32_t vbase, int /*valid*/,
                                         float /*scale_log2*/, int /*lane*/, int row0, int limit0,
                                         int /*grp*/, int /*skip*/, uint32_t /*xb: none*/) {
        const uint32_t kbox = kbase + (ch >> 3) * kBoxBytes;
        const uint32_t vbox = vbase + (ch >> 3) * kBoxBytes;
        const int cc = ch & 7;
        const uint32_t seen = rows_seen(row0, limit0, window, sinks);
        float sc[kSubs];
        float mx = -INFINITY;
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) {
            float part[kScoresOf];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                const uint4 raw = lds128(swizzled(kbox, (sub * kSub + j) * kRpp + rr, cc));
                const float k[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w)};
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float acc = qf[g][0] * k[0];
#pragma unroll
                    for (int e = 1; e < 4; ++e) acc = fmaf(qf[g][e], k[e], acc);
                    part[j * G + g] = acc;
                }
            }
#pragma unroll
            for (int n = kScoresOf / 2, off = kLpr / 2; off > 0; n /= 2, off /= 2) {
                if (n > 0) {
                    const bool high = (ch & off) != 0;
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float give = high ? part[i] : part[i + n];
                        part[i] = (high ? part[i + n] : part[i]) + __shfl_xor_sync(0xffffffffu, give, off);
                    }
                } else {
                    part[0] += __shfl_xor_sync(0xffffffffu, part[0], off);
                }
            }
            const int row = (sub * kSub + own / G) * kRpp + rr;
            sc[sub] = (seen >> row) & 1u ? part[0] : -INFINITY;
            mx = fmaxf(mx, sc[sub]);
            if constexpr (SCORES) {
                if (ch % kTwins == 0 && own % G < cols) scores[static_cast<size_t>(row0 + row) * cols + own % G] = sc[sub];
            }
        }
        // Over the lanes of a head: those that differ in the pass, then in the row of a pass.
#pragma unroll
        for (int off = kTwins * G; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx);
        // (A whole tile can be masked while the maximum is still -inf: weights 0 then.)
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float al = fast_exp2(m - ref);
        m = mn;
        l *= al;
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) {
            const float w = fast_exp2(sc[sub] - ref);
            l += w;
            if (ch % kTwins == 0) weights[((sub * kSub + own / G) * kRpp + rr) * G + own % G] = w;
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float a = __shfl_sync(0xffffffffu, al, g * kTwins);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[g][e] *= a;
            }
        }
        auto add = [&](int row) {
            const uint4 raw = lds128(swizzled(vbox, row, cc));
            const float v[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w)};
            float w[G];
            if constexpr (G % 4 == 0) {
#pragma unroll
                for (int g = 0; g < G; g += 4)
                    *reinterpret_cast<float4*>(w + g) = *reinterpret_cast<const float4*>(weights + row * G + g);
            } else if constexpr (G == 2) {
                *reinterpret_cast<float2*>(w) = *reinterpret_cast<const float2*>(weights + row * G);
            } else {
                w[0] = weights[row];
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[g][e] = fmaf(w[g], v[e], o[g][e]);
        };
        if (seen == 0xffffu) {
#pragma unroll
            for (int j = 0; j < kPasses; ++j) add(j * kRpp + rr);
        } else {                                  // (0 * NaN would stay in the sums)
            for (int j = 0; j < kPasses; ++j)
                if ((seen >> (j * kRpp + rr)) & 1u) add(j * kRpp + rr);
        }
    }

    // State layout as SimtMath's.
    __device__ __forceinline__ void write_state(float* st, int lane, int /*ncols*/) {
        __syncwarp();                             // the weights were in its place
#pragma unroll
        for (int off = kTwins * G; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
        for (int off = kLpr; off < 32; off <<= 1)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[g][e] += __shfl_xor_sync(0xffffffffu, o[g][e], off);
        if (lane % kTwins == 0 && lane / kTwins < G) {
            st[own] = m;
            st[G + own] = l;
        }
        if (rr == 0) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[2 * G + g * D + ch * 4 + e] = o[g][e];
        }
    }
};

}  // namespace pa

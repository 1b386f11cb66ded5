// pa_decode_rows.cu -- pa_decode_sinks and pa_decode_weights beside the tile
// ring: the plain decode kernel for the shapes that the ring has no instance
// for (bound by its loads a row at a time: some 12 times the ring's time where both can run),
// and the kernel that turns the scores of pa_decode_weights into row weights.
//
// A query token j of a sequence of n rows sits at row r = n - Q + j. With a window it
// sees the rows i <= r with i < num_sinks or i > r - window (p.window counts the
// rows of all Q tokens, window + Q - 1). Partitions cover the rows that some token
// may see: the first rows, then those from the window's tile on, without the rows
// between them (seq_gap).
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;
constexpr int kCols = 8;              // query columns that the plain kernel takes at a time

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// The plain kernel: one CTA per (sequence, KV head, partition), the scores of up
// to kCols query columns (a query token's head of the group each) at a time in shared
// memory. Rows that a column does not see are left out of its sums, whatever they hold.
// Not tuned.
template <typename T>
__global__ void __launch_bounds__(kThreads) decode_rows_kernel(const DecodeParams p) {
    using E = ElemTraits<T>;
    extern __shared__ float sm[];
    const int D = p.head_dim, PS = p.partition_size;
    float* qf = sm;                           // [kCols][D]
    float* sc = qf + kCols * D;               // [kCols][PS]; -1 in place of the weight of an unseen row
    float* red = sc + kCols * PS;             // [kCols][2]: max, sum
    long long* rows = reinterpret_cast<long long*>(red + 2 * kCols);   // [PS] pool row of each row
    __shared__ int bad;

    const int bh = p.num_seqs * p.num_kv_heads;
    const int part = blockIdx.x / bh;
    const int rem = blockIdx.x - part * bh;
    const int s = rem / p.num_kv_heads;
    const int h = rem - s * p.num_kv_heads;
    const int Q = p.num_queries;
    const int grp = p.num_heads / p.num_kv_heads;
    const int n = __ldg(p.context_lens + s);
    if (n < 0 || n > p.context_cap || (n > 0 && n < Q)) {
        if (threadIdx.x == 0 && part == 0 && h == 0) raise_error(p.error_word, PA_DEVERR_CONTEXT);
        return;
    }
    // Query column c: token c / grp, head h * grp + c % grp.
    const int cols = grp * Q;
    auto out_row = [&](int c) {
        return (static_cast<size_t>(s) * Q + c / grp) * p.num_heads + h * grp + c % grp;
    };
    if (n == 0) {
        if (part == 0)
            for (int i = threadIdx.x; i < cols * D; i += kThreads)
                E::store(static_cast<T*>(p.out) + out_row(i / D) * D + i % D, 0.f);
        return;
    }
    const int gap = seq_gap(p, n), head = sink_rows(p);
    const int span = n - gap;
    const int lo = part * PS;
    if (lo >= span) return;
    const int len = min(span - lo, PS);
    const int nparts = (span + PS - 1) / PS;
    const int bs = p.block_size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto row_at = [&](int i) {                // the sequence's row of the partition's row i
        const int v = lo + i;
        return gap > 0 && v >= head ? v + gap : v;
    };

    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < len; i += kThreads) {
        const int r = row_at(i);
        const int id = __ldg(p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq + r / bs);
        if (id < 0 || id >= p.num_blocks) bad = 1;
        rows[i] = (static_cast<long long>(id) * p.num_kv_heads + h) * bs + r % bs;
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) raise_error(p.error_word, PA_DEVERR_BLOCK_ID);
        if (p.scores != nullptr)
            for (int c = threadIdx.x; c < cols; c += kThreads) p.part_ml[2 * (out_row(c) * p.max_parts + part) + 1] = kNoSum;
        return;
    }
    const T* kc = static_cast<const T*>(p.k_cache);
    const T* vc = static_cast<const T*>(p.v_cache);
    const int window = p.window > 0 ? p.window - Q + 1 : 0;   // of one token
    auto sees = [&](int c, int r) {
        const int last = n - Q + c / grp;
        return r <= last && (window == 0 || r < p.num_sinks || r > last - window);
    };
    for (int c0 = 0; c0 < cols; c0 += kCols) {
        const int nc = min(kCols, cols - c0);
        for (int i = threadIdx.x; i < nc * D; i += kThreads)
            qf[i] = E::load(static_cast<const T*>(p.q) + out_row(c0 + i / D) * D + i % D) * p.scale_log2;
        __syncthreads();
        for (int i = warp; i < len; i += kThreads / 32) {
            const T* krow = kc + rows[i] * D;
            const int r = row_at(i);
            for (int c = 0; c < nc; ++c) {
                float acc = 0.f;
                for (int d = lane; d < D; d += 32) acc = fmaf(qf[c * D + d], E::load(krow + d), acc);
                acc = warp_sum(acc);
                if (!sees(c0 + c, r)) acc = -INFINITY;
                if (lane == 0) {
                    sc[c * PS + i] = acc;
                    if (p.scores != nullptr)
                        p.scores[((static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows + r) * cols + c0 + c] = acc;
                }
            }
        }
        __syncthreads();
        for (int c = warp; c < nc; c += kThreads / 32) {
            float mx = -INFINITY;
            for (int i = lane; i < len; i += 32) mx = fmaxf(mx, sc[c * PS + i]);
            mx = warp_max(mx);
            const float ref = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f;
            for (int i = lane; i < len; i += 32) {
                const bool see = sees(c0 + c, row_at(i));
                const float e = see ? fast_exp2(sc[c * PS + i] - ref) : 0.f;
                sc[c * PS + i] = see ? e : -1.f;
                sum += e;
            }
            sum = warp_sum(sum);
            if (lane == 0) {
                red[2 * c] = mx;
                red[2 * c + 1] = sum;
            }
        }
        __syncthreads();
        for (int idx = threadIdx.x; idx < nc * D; idx += kThreads) {
            const int c = idx / D, d = idx - c * D;
            float acc = 0.f;
            for (int i = 0; i < len; ++i) {
                const float w = sc[c * PS + i];
                if (!(w < 0.f)) acc = fmaf(w, E::load(vc + rows[i] * D + d), acc);
            }
            const size_t row = out_row(c0 + c);
            const size_t slot = row * p.max_parts + part;
            if (nparts == 1)
                E::store(static_cast<T*>(p.out) + row * D + d, acc / red[2 * c + 1]);
            else
                p.part_o[slot * D + d] = acc;
            if (d == 0 && (nparts > 1 || p.scores != nullptr)) {
                p.part_ml[2 * slot] = red[2 * c];
                p.part_ml[2 * slot + 1] = red[2 * c + 1];
            }
        }
        __syncthreads();
    }
}

// Row weights: with the final maximum and sum of every query column (of a merged sequence
// the merge's, else its only partition's)
//   w = sum_c 2^(score_c - M_c) / L_c
// for every row, stored for the rows of this call's tokens, added for the others
// (atomically: sequences may share a block). A partition with a block outside the pool, or that the
// decode kernel gave up before its end, both flagged, has the sum kNoSum: its sequence keeps its weights.
//
// A warp takes 128 rows of a partition under one KV head, four a lane; all that it loads
// (states, scores, block ids) is on the way together, so that the time is some three
// latencies of memory, in 1.5 rounds of warps for 128 sequences of 1,640 rows, 13 us (a CTA
// per partition, which found its columns' states from all partitions first, took
// three times as long).
constexpr int kWeightThreads = 256;
constexpr int kWeightRows = 4;                // of a lane
constexpr int kWeightUnit = 32 * kWeightRows;
constexpr int kWeightSplit = kDefaultPartition / kWeightUnit;   // warps of a partition
constexpr int kWeightItems = kWeightThreads / 32 / kWeightSplit;   // partitions of a CTA at a time
static_assert(kDefaultPartition % kWeightUnit == 0 && kWeightThreads / 32 % kWeightSplit == 0, "whole warps");

// LISTED: the partitions are those of the tile ring's work list, item_count[0] of them; else
// (the plain kernel has no list) all that there may be.
// TOKENS: there may be several query tokens, and rows that not all of them see.
template <bool LISTED, bool TOKENS>
__global__ void __launch_bounds__(kWeightThreads) row_weights_kernel(const DecodeParams p, const int32_t* item_count,
                                                                     int most_items, const Divisor by_block) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int grp = p.num_heads / p.num_kv_heads, Q = p.num_queries;
    const int cols = grp * Q;
    const int bs = p.block_size;
    const int warp = threadIdx.x >> 5, sub = warp % kWeightSplit;
    const int items = LISTED ? item_count[0] : most_items;
    for (int k = blockIdx.x * kWeightItems + warp / kWeightSplit; k < items; k += gridDim.x * kWeightItems) {
        int s, h, part, n;
        if constexpr (LISTED) {
            const int4 it = p.items[k];
            s = it.x;
            h = it.y / p.col_groups;
            if (it.y != h * p.col_groups) continue;                          // (the first column group takes them all)
            part = it.z;
            n = it.w;
        } else {
            const int bh = p.num_seqs * p.num_kv_heads;
            part = k / bh;
            s = (k - part * bh) / p.num_kv_heads;
            h = k - part * bh - s * p.num_kv_heads;
            n = __ldg(p.context_lens + s);
            if (n > p.context_cap || n < Q) continue;                        // flagged or empty
        }
        const int i0 = part * kDefaultPartition + sub * kWeightUnit + lane;
        const int end = min(n, (part + 1) * kDefaultPartition);
        if (i0 - lane >= end) continue;
        const int nparts = (n + kDefaultPartition - 1) / kDefaultPartition;
        const size_t row0 = static_cast<size_t>(s) * Q * p.num_heads + h * grp;   // of column 0
        const float2* states = reinterpret_cast<const float2*>(p.part_ml);
        bool no_sum = false;
        for (int i = lane; i < nparts; i += 32) no_sum |= states[row0 * p.max_parts + i].y == kNoSum;
        if (LISTED && p.col_groups > 1)           // (an item of a further column group may have no sums of its own)
            for (int j = p.group_tokens; j < Q; j += p.group_tokens)
                for (int i = lane; i < nparts; i += 32)
                    no_sum |= states[(row0 + static_cast<size_t>(j) * p.num_heads) * p.max_parts + i].y == kNoSum;
        const int32_t* table = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
        int id[kWeightRows];
        float w[kWeightRows];
#pragma unroll
        for (int u = 0; u < kWeightRows; ++u) {
            const int i = min(i0 + 32 * u, end - 1);
            id[u] = __ldg(table + by_block.quotient(i));
            w[u] = 0.f;
        }
        // First column of a token that sees the lane's first row (others add nothing, not 0 times a sum that
        // may be NaN); far before the tokens' rows all see the lane's rows, and no product leaves 32 bits.
        const int first_col = TOKENS ? max(i0 - (n - Q), -kWeightUnit) * grp : 0;
        const float* sc = p.scores + (static_cast<size_t>(s) * p.num_kv_heads + h) * p.score_rows * cols;
        for (int c0 = 0; c0 < cols; c0 += 32) {
            float2 own = make_float2(0.f, 1.f);
            if (c0 + lane < cols) {
                const int c = c0 + lane, j = c / grp;
                const size_t row = row0 + static_cast<size_t>(j) * p.num_heads + (c - j * grp);
                own = nparts > 1 ? p.final_ml[row] : states[row * p.max_parts];
            }
            own.x = own.x == -INFINITY ? 0.f : own.x;
            own.y = 1.f / own.y;
            auto take = [&](const float (&score)[kWeightRows], int c) {
                const float m = __shfl_sync(0xffffffffu, own.x, c - c0), r = __shfl_sync(0xffffffffu, own.y, c - c0);
#pragma unroll
                for (int u = 0; u < kWeightRows; ++u)
                    if (!TOKENS || c >= first_col + 32 * u * grp) w[u] = fmaf(fast_exp2(score[u] - m), r, w[u]);
            };
            const int ce = min(cols, c0 + 32);
            if (cols % 4 == 0) {
                for (int c = c0; c < ce; c += 4) {
                    float v[4][kWeightRows];
#pragma unroll
                    for (int u = 0; u < kWeightRows; ++u) {
                        const float4 x = *reinterpret_cast<const float4*>(sc + static_cast<size_t>(min(i0 + 32 * u, end - 1)) * cols + c);
                        v[0][u] = x.x;
                        v[1][u] = x.y;
                        v[2][u] = x.z;
                        v[3][u] = x.w;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) take(v[e], c + e);
                }
            } else {
                for (int c = c0; c < ce; ++c) {
                    float v[kWeightRows];
#pragma unroll
                    for (int u = 0; u < kWeightRows; ++u) v[u] = sc[static_cast<size_t>(min(i0 + 32 * u, end - 1)) * cols + c];
                    take(v, c);
                }
            }
        }
        if (__any_sync(0xffffffffu, no_sum)) continue;
#pragma unroll
        for (int u = 0; u < kWeightRows; ++u) {
            const int i = i0 + 32 * u;
            // (An id outside the pool: its sequence is flagged, or the ring gave up before its partition.)
            if (i >= end || id[u] < 0 || id[u] >= p.num_blocks) continue;
            float* at = p.row_weights + (static_cast<size_t>(id[u]) * p.num_kv_heads + h) * bs + by_block.rest(i, by_block.quotient(i));
            if (i >= n - Q)
                *at = w[u];
            else
                atomicAdd(at, w[u]);
        }
    }
}

}  // namespace

cudaError_t launch_decode_rows(const DecodeParams& p, pa_dtype dtype, cudaStream_t stream) {
    const size_t smem = 4 * (static_cast<size_t>(kCols) * (p.head_dim + p.partition_size + 2)) + 8 * static_cast<size_t>(p.partition_size);
    const long long grid = static_cast<long long>(p.max_parts) * p.num_seqs * p.num_kv_heads;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // At most 8 x (256 + 752 + 2) floats and 752 row numbers: within the default limit.
    if (dtype == PA_DTYPE_BF16)
        decode_rows_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(p);
    else
        decode_rows_kernel<float><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_row_weights(const DecodeParams& p, const int32_t* item_count, cudaStream_t stream) {
    const long long most = static_cast<long long>(p.max_parts) * p.num_seqs * p.num_kv_heads;
    if (most == 0 || p.context_cap == 0) return cudaSuccess;
    if (most > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int sms = device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (p.partition_size != kDefaultPartition) return cudaErrorInvalidValue;
    const long long ctas = (most + kWeightItems - 1) / kWeightItems;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < 8LL * sms ? ctas : 8LL * sms));
    cfg.blockDim = dim3(kWeightThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = item_count != nullptr ? (p.num_queries > 1 ? row_weights_kernel<true, true> : row_weights_kernel<true, false>)
                                         : (p.num_queries > 1 ? row_weights_kernel<false, true> : row_weights_kernel<false, false>);
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, p, item_count, static_cast<int>(most), Divisor(static_cast<uint32_t>(p.block_size)));
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace pa

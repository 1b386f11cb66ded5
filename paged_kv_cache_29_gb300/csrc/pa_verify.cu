// pa_verify.cu -- verification of drafted tokens (pa_verify_draft).
//
// Token i is accepted while u_i q_i(x_i) < p_i(x_i): products of two fp32 values
// are exact in 64 bits. After the last accepted one a token is drawn from
// r = max(p - q, 0) (or p) by its running sum: the smallest v with
// r(0) + .. + r(v) > u S, S the sum of all. Only that one row of p (and of q) is read.
//
// A cluster of CTAs shares a sequence's row, a CTA a run of its segments of 512
// values. A warp sums a segment: each lane its 16 values as an fp32 value and the
// running error of it (the difference p - q and every addition leave an exact error
// term; fp64 adds and conversions are slow here), the lanes in 64 bits. Running sums over
// the CTA's segments, then over the cluster's CTAs through their shared memory, find
// the one segment that u S falls into; the CTA scans that in 64 bits, a value a thread.
// Every order of addition is fixed by the row's length and the cluster's size.
#include <climits>

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {

namespace {

constexpr int kVerifyThreads = 512;
constexpr int kSegment = 512;                 // a value a thread, in the last step
constexpr int kWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSegments = 4096;            // of a CTA: their running sums fit the default shared memory

// value and error term of a sum of fp32 values
struct Sum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x, float err) {
        const float s = hi + x;
        const float b = s - hi;
        lo += ((hi - (s - b)) + (x - b)) + err;
        hi = s;
    }
};

__device__ __forceinline__ double warp_scan(double v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
    }
    return v;
}

// A lane's part of the segment's sum that begins at v0 - lane: r = max(p - q, 0) or, without q, p
// but for value `out`. All loads go out before their use.
template <bool HAS_Q>
__device__ __forceinline__ double sum_part(const float* pr, const float* qr, int v0, int V, int out) {
    constexpr int N = kSegment / 32;
    float x[N], y[HAS_Q ? N : 1];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int v = v0 + 32 * k;
        x[k] = v < V && (HAS_Q || v != out) ? __ldg(pr + v) : 0.f;
        if constexpr (HAS_Q) y[k] = v < V ? __ldg(qr + v) : 0.f;
    }
    Sum sum;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (HAS_Q) {
            const float diff = x[k] - y[k];
            const float b = x[k] - diff;     // x - y is diff + (x - (diff + b)) + (b - y) exactly
            if (diff > 0.f) sum.add(diff, (x[k] - (diff + b)) + (b - y[k]));
        } else if (x[k] > 0.f) {
            sum.add(x[k], 0.f);
        }
    }
    return static_cast<double>(sum.hi) + static_cast<double>(sum.lo);
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p, int segs_per_cta) {
    extern __shared__ double seg_sum[];       // [segs_per_cta], then their running sums
    __shared__ double cta_total, warp_total[kWarps];
    __shared__ int first_rejected, bad, chosen;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int s = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Q = p.max_drafts, V = p.vocab;
    const int d = p.num_drafts != nullptr ? __ldg(p.num_drafts + s) : Q;
    const bool bad_count = d < 0 || d > Q;
    const float* target = p.target + s * p.target_seq;
    const float* draft = p.draft == nullptr ? nullptr : p.draft + s * p.draft_seq;
    const int32_t* tokens = p.tokens + static_cast<size_t>(s) * Q;
    const float* uniforms = p.uniforms + static_cast<size_t>(s) * (Q + 1);
    // Read by every CTA before the cluster's barrier; lens_out (it may be the
    // same array) is written behind it.
    const int rows = p.context_lens != nullptr ? p.context_lens[s] : 0;
    if (tid == 0) {
        first_rejected = bad_count ? 0 : d;
        bad = bad_count ? PA_DEVERR_TOKEN : 0;
    }
    __syncthreads();
    if (!bad_count && tid < d) {
        const int x = __ldg(tokens + tid);
        if (x < 0 || x >= V) {
            atomicOr(&bad, PA_DEVERR_TOKEN);
        } else {
            const double px = __ldg(target + tid * p.target_row + x);
            const double qx = draft != nullptr ? __ldg(draft + tid * p.draft_row + x) : 1.0f;
            if (!(static_cast<double>(__ldg(uniforms + tid)) * qx < px)) atomicMin(&first_rejected, tid);
        }
    }
    __syncthreads();
    const int a = first_rejected;
    int error = bad;
    if (error == 0 && p.context_lens != nullptr && rows < d - a) error = PA_DEVERR_CONTEXT;
    if (error != 0) {                         // the same in every CTA of the cluster
        if (rank == 0 && tid == 0) raise_error(p.error_word, error);
        return;
    }
    const bool rejected = a < d;
    const float* pr = target + a * p.target_row;
    const float* qr = rejected && draft != nullptr ? draft + a * p.draft_row : nullptr;
    const int looked_up = rejected && draft == nullptr ? __ldg(tokens + a) : -1;
    bool plain = false;                       // from p itself, where the difference leaves nothing
    // r(v) in 64 bits
    auto value = [&](int v) -> double {
        const double x = __ldg(pr + v);
        const double r = plain ? x : qr != nullptr ? x - static_cast<double>(__ldg(qr + v)) : v == looked_up ? 0.0 : x;
        return r > 0.0 ? r : 0.0;
    };

    const int seg0 = rank * segs_per_cta;
    const int segs = max(0, min((V + kSegment - 1) / kSegment - seg0, segs_per_cta));
    double base = 0.0, total = 0.0, own_end = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        plain = pass == 1;
        for (int g = warp; g < segs; g += kWarps) {
            const int v0 = (seg0 + g) * kSegment + lane;
            double v = !plain && qr != nullptr ? sum_part<true>(pr, qr, v0, V, -1)
                                               : sum_part<false>(pr, nullptr, v0, V, plain ? -1 : looked_up);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (lane == 0) seg_sum[g] = v;
        }
        __syncthreads();
        if (warp == 0) {
            double carry = 0.0;
            for (int g0 = 0; g0 < segs; g0 += 32) {
                const double v = warp_scan(g0 + lane < segs ? seg_sum[g0 + lane] : 0.0, lane) + carry;
                if (g0 + lane < segs) seg_sum[g0 + lane] = v;
                carry = __shfl_sync(0xffffffffu, v, min(31, segs - g0 - 1));
            }
            if (lane == 0) cta_total = carry;        // the last running sum itself
        }
        cluster.sync();
        total = 0.0;
        for (int r = 0; r < ranks; ++r) {
            if (r == rank) base = total;
            total += *cluster.map_shared_rank(&cta_total, r);
            if (r == rank) own_end = total;
        }
        // Every CTA has read the totals: another pass may write them, or a CTA end.
        cluster.sync();
        if (total > 0.0) break;
    }
    if (!(total > 0.0)) {
        if (rank == 0 && tid == 0) raise_error(p.error_word, PA_DEVERR_TOKEN);
        return;
    }
    const float u = fminf(fmaxf(__ldg(uniforms + Q), 0.f), 0.99999994f);   // [0, 1)
    const double border = static_cast<double>(u) * total;
    if (!(base <= border && border < own_end)) return;   // one CTA of the cluster goes on
    // The segment: the first whose running sum passes the border. (Where the two ways to
    // sum part by a rounding the walk may go on to the next, or end behind the last.)
    if (tid == 0) chosen = INT_MAX;
    __syncthreads();
    for (int g = tid; g < segs; g += kVerifyThreads)
        if (base + seg_sum[g] > border) atomicMin(&chosen, g);
    __syncthreads();
    const int seg = chosen;                   // there is one: the last running sum is the CTA's end
    double upto = base + (seg > 0 ? seg_sum[seg - 1] : 0.0);
    __syncthreads();
    if (tid == 0) chosen = INT_MAX;
    int token = INT_MAX, last_positive = -1;
    for (int g = seg; g < segs && token == INT_MAX; ++g) {
        const int v = (seg0 + g) * kSegment + tid;
        const double r = v < V ? value(v) : 0.0;
        double run = warp_scan(r, lane);
        if (lane == 31) warp_total[warp] = run;
        __syncthreads();
        run += upto;
        double end = upto;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) run += warp_total[w];
            end += warp_total[w];
        }
        if (r > 0.0 && run > border) atomicMin(&chosen, v);
        if (r > 0.0) last_positive = v;
        __syncthreads();
        token = chosen;
        upto = end;
    }
    if (token == INT_MAX) {
        // The last value that can be drawn: of the segments walked, else before them.
        __syncthreads();                      // every thread has read `chosen`
        if (tid == 0) chosen = -1;
        __syncthreads();
        for (int v = seg0 * kSegment + tid; last_positive < 0 && v < min(V, (seg0 + seg) * kSegment); v += kVerifyThreads)
            if (value(v) > 0.0) atomicMax(&chosen, v);
        if (last_positive >= 0) atomicMax(&chosen, last_positive);
        __syncthreads();
        token = chosen;
    }
    if (warp != 0) return;
    for (int i = lane; i <= Q; i += 32)
        p.out_tokens[static_cast<size_t>(s) * (Q + 1) + i] = i < a ? __ldg(tokens + i) : i == a ? token : -1;
    if (lane == 0) {
        p.num_accepted[s] = a;
        if (p.lens_out != nullptr) p.lens_out[s] = rows - (d - a);
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
    if (p.num_seqs == 0) return cudaSuccess;
    const int sms = device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int segs = (p.vocab + kSegment - 1) / kSegment;
    int ranks = 1;
    while (ranks < kMaxCluster && ranks < segs &&
           (static_cast<long long>(p.num_seqs) * ranks < sms || segs > kMaxSegments * ranks))
        ranks *= 2;
    const int per_cta = (segs + ranks - 1) / ranks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * ranks);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = 8 * static_cast<size_t>(per_cta);   // 32 KB at most
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, verify_kernel, p, per_cta);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace pa

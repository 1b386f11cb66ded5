// pa_verify.cu -- verification of drafted tokens (pa_verify_draft).
//
// Token i is accepted while u_i q_i(x_i) < p_i(x_i): products of two fp32 values
// are exact in 64 bits. After the last accepted one a token is drawn from
// r = max(p - q, 0) (or p) by its running sum: the smallest v with
// r(0) + .. + r(v) > u S, S the sum of all. Only that one row of p (and of q) is read.
//
// Sums are pairs of fp32 values, a sum and its error: the difference p - q and each
// addition leave an exact error term (Knuth's two-sum), and what is lost is below 2^-44 of a sum. (An fp64
// instruction holds the SM's fp64 pipe for 16 cycles a warp: with fp64 lanes the
// additions took as long as the loads.)
//
// A cluster of CTAs shares a sequence's row, a CTA a run of its segments of 512
// values, a warp a segment at a time. Running sums over the CTA's segments, then over
// the cluster's CTAs through their shared memory, find the one segment that u S falls
// into; its CTA scans that, a value a thread. Every order of addition is fixed by the
// row's length and the cluster's size.
//
// 128 sequences, 4 drafts, 131,072 values: 28.6 us for 118 MB, of which 20 stream (5.9 TB/s),
// 2 go before (tokens, then their probabilities) and 6 behind (running sums, cluster, last segment).
// One sequence of 32,000 values: 7.5 us of latencies.
#include <climits>
#include <utility>

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = kThreads;            // a value a thread, in the last step
constexpr int kMaxCluster = 8;
// Segments of a CTA: their running sums fit the default shared memory.
constexpr int kMaxSegments = 4096;
constexpr float kUp = 0x1p100f;
constexpr int kNothing = -2, kNoSums = -3;    // in place of a segment

// A sum of fp32 values as hi + lo, |lo| at most half a step of hi.
struct Sum {
    float hi, lo;
    // + x + err; lo is left to grow (order() or plus() bring the pair to order)
    __device__ __forceinline__ void add(float x, float err) {
        const float s = hi + x;
        const float b = s - hi;
        lo += ((hi - (s - b)) + (x - b)) + err;
        hi = s;
    }
    __device__ __forceinline__ Sum plus(const Sum& o) const {
        const float s = hi + o.hi;
        const float b = s - hi;
        const float e = ((hi - (s - b)) + (o.hi - b)) + (lo + o.lo);
        Sum r;
        r.hi = s + e;
        r.lo = e - (r.hi - s);
        return r;
    }
    __device__ __forceinline__ Sum order() const {
        Sum r;
        r.hi = hi + lo;
        r.lo = lo - (r.hi - hi);
        return r;
    }
    __device__ __forceinline__ Sum minus(const Sum& o) const { return plus(Sum{-o.hi, -o.lo}); }
    __device__ __forceinline__ Sum times(float u) const {
        const float p = hi * u;
        return Sum{p, fmaf(hi, u, -p) + lo * u}.order();
    }
    __device__ __forceinline__ Sum scaled(float by) const { return Sum{hi * by, lo * by}; }   // by a power of two
    __device__ __forceinline__ bool above(const Sum& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
};

// x - y for x > y, else nothing; NaN counts as nothing.
__device__ __forceinline__ void add_excess(Sum& sum, float x, float y) {
    const float diff = x - y;
    const float b = x - diff;                 // x - y is diff + (x - (diff + b)) + (b - y) exactly
    if (diff > 0.f) sum.add(diff, (x - (diff + b)) + (b - y));
}

__device__ __forceinline__ Sum shuffle(const Sum& v, int from) {
    return Sum{__shfl_sync(0xffffffffu, v.hi, from), __shfl_sync(0xffffffffu, v.lo, from)};
}

__device__ __forceinline__ Sum warp_scan(Sum v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        Sum u;
        u.hi = __shfl_up_sync(0xffffffffu, v.hi, off);
        u.lo = __shfl_up_sync(0xffffffffu, v.lo, off);
        if (lane >= off) v = u.plus(v);
    }
    return v;
}

// Two values of a lane side by side.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t plus2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t minus2(uint64_t a, uint64_t b) {   // b * -1 + a, one rounding
    constexpr uint64_t kMinusOnes = 0xbf800000bf800000ull;
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(kMinusOnes), "l"(a));
    return r;
}

// add_excess of two values into two sums, two values an instruction.
template <bool HAS_Q>
__device__ __forceinline__ void add_excess2(uint64_t& hi, uint64_t& lo, float x0, float x1, float y0, float y1) {
    float d0 = x0, d1 = x1;
    uint64_t err = 0;
    if constexpr (HAS_Q) {
        const uint64_t x = two(x0, x1), y = two(y0, y1);
        const uint64_t diff = minus2(x, y);
        const uint64_t b = minus2(x, diff);
        err = plus2(minus2(x, plus2(diff, b)), minus2(b, y));
        float e0, e1;
        apart(diff, d0, d1);
        apart(err, e0, e1);
        err = two(d0 > 0.f ? e0 : 0.f, d1 > 0.f ? e1 : 0.f);
    }
    const uint64_t d = two(fmaxf(d0, 0.f), fmaxf(d1, 0.f));   // NaN: 0
    const uint64_t s = plus2(hi, d);
    const uint64_t b = minus2(s, hi);
    const uint64_t lost = plus2(minus2(hi, minus2(s, b)), minus2(d, b));
    lo = plus2(lo, HAS_Q ? plus2(lost, err) : lost);
    hi = s;
}

// A lane's part of the sum of the segment of 32 N values at v0: r = max(p - q, 0) or,
// without q, max(p, 0). Whole segments: VEC with 16-byte loads, or by single values. All
// loads go out before their use.
template <int N, bool HAS_Q, bool VEC>
__device__ __forceinline__ Sum sum_part(const float* pr, const float* qr, int v0, int lane) {
    float x[N], y[N];
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            *reinterpret_cast<float4*>(x + 4 * k) = __ldg(reinterpret_cast<const float4*>(pr + v0) + lane + 32 * k);
            if constexpr (HAS_Q)
                *reinterpret_cast<float4*>(y + 4 * k) = __ldg(reinterpret_cast<const float4*>(qr + v0) + lane + 32 * k);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            x[k] = __ldg(pr + v0 + lane + 32 * k);
            if constexpr (HAS_Q) y[k] = __ldg(qr + v0 + lane + 32 * k);
        }
    }
    uint64_t hi = 0, lo = 0;
#pragma unroll
    for (int k = 0; k < N; k += 2) add_excess2<HAS_Q>(hi, lo, x[k], x[k + 1], HAS_Q ? y[k] : 0.f, HAS_Q ? y[k + 1] : 0.f);
    Sum a, b;
    apart(hi, a.hi, b.hi);
    apart(lo, a.lo, b.lo);
    return a.plus(b);
}

// The same for a segment that ends behind the row, or holds the value `out` that is left out.
template <int N>
__device__ __forceinline__ Sum sum_some(const float* pr, const float* qr, int v0, int lane, int V, int out) {
    float x[N], y[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int v = v0 + lane + 32 * k;
        x[k] = v < V && v != out ? __ldg(pr + v) : 0.f;
        y[k] = v < V && qr != nullptr ? __ldg(qr + v) : 0.f;
    }
    Sum sum{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N; ++k) add_excess(sum, x[k], y[k]);
    return sum.order();
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p, int segs_per_cta) {
    extern __shared__ Sum seg_sum[];          // [segs_per_cta]: of each segment, then up to its end
    __shared__ Sum cta_total, warp_total[kWarps], border_left;
    __shared__ bool in_units;
    __shared__ int first_rejected, bad, chosen, owner;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Q = p.max_drafts, V = p.vocab;
    const float* target = p.target + s * p.target_seq;
    const float* draft = p.draft == nullptr ? nullptr : p.draft + s * p.draft_seq;
    const int32_t* tokens = p.tokens + static_cast<size_t>(s) * Q;
    const float* uniforms = p.uniforms + static_cast<size_t>(s) * (Q + 1);
    // Independent loads first. (lens_out may be context_lens: it is written behind the
    // cluster's barrier, which every CTA reaches after this read. What may be another call's
    // output is read with ordinary loads, as in the plan of the decode kernels.)
    const int d = p.num_drafts != nullptr ? p.num_drafts[s] : Q;
    const int rows = p.context_lens != nullptr ? p.context_lens[s] : 0;
    const int x = tid < Q ? tokens[tid] : 0;
    const float ux = tid < Q ? __ldg(uniforms + tid) : 0.f;
    const float u_last = __ldg(uniforms + Q);
    const bool bad_count = d < 0 || d > Q;
    if (tid == 0) {
        first_rejected = bad_count ? 0 : d;
        bad = bad_count ? PA_DEVERR_TOKEN : 0;
    }
    __syncthreads();
    if (!bad_count && tid < d) {
        if (x < 0 || x >= V) {
            atomicOr(&bad, PA_DEVERR_TOKEN);
        } else {
            const double px = __ldg(target + tid * p.target_row + x);
            const double qx = draft != nullptr ? __ldg(draft + tid * p.draft_row + x) : 1.0f;
            if (!(static_cast<double>(ux) * qx < px)) atomicMin(&first_rejected, tid);
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
    int left_out = rejected && draft == nullptr ? tokens[a] : -1;   // looked up: q is 1 there

    const int seg0 = rank * segs_per_cta;
    const int segs = max(0, min((V + kSegment - 1) / kSegment - seg0, segs_per_cta));
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1) {                      // the difference leaves nothing: from p itself
            qr = nullptr;
            left_out = -1;
        }
        constexpr int N = kSegment / 32;
        const bool vec = ((reinterpret_cast<uintptr_t>(pr) | reinterpret_cast<uintptr_t>(qr)) & 15u) == 0;
        for (int g = warp; g < segs; g += kWarps) {
            const int v0 = (seg0 + g) * kSegment;
            Sum v;
            if (v0 + kSegment > V || (left_out >= v0 && left_out < v0 + kSegment))
                v = sum_some<N>(pr, qr, v0, lane, V, left_out);
            else if (qr != nullptr)
                v = vec ? sum_part<N, true, true>(pr, qr, v0, lane) : sum_part<N, true, false>(pr, qr, v0, lane);
            else
                v = vec ? sum_part<N, false, true>(pr, nullptr, v0, lane) : sum_part<N, false, false>(pr, nullptr, v0, lane);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                Sum o;
                o.hi = __shfl_xor_sync(0xffffffffu, v.hi, off);
                o.lo = __shfl_xor_sync(0xffffffffu, v.lo, off);
                v = v.plus(o);
            }
            if (lane == 0) seg_sum[g] = v;
        }
        __syncthreads();
        if (warp == 0) {
            // Running sums: each lane's run of segments, then the lanes'.
            const int run = (segs + 31) / 32, g0 = min(segs, lane * run), g1 = min(segs, g0 + run);
            Sum own{0.f, 0.f};
            for (int g = g0; g < g1; ++g) own = own.plus(seg_sum[g]);
            const Sum incl = warp_scan(own, lane);
            Sum upto = shuffle(incl, lane > 0 ? lane - 1 : 0);
            if (lane == 0) upto = Sum{0.f, 0.f};
            for (int g = g0; g < g1; ++g) {
                upto = upto.plus(seg_sum[g]);
                seg_sum[g] = upto;
            }
            __syncwarp();
            if (lane == 0) cta_total = segs > 0 ? seg_sum[segs - 1] : Sum{0.f, 0.f};
        }
        cluster.sync();
        if (warp == 0) {
            // Where u S falls: in this CTA's part, and in which of its segments?
            const Sum mine = lane < ranks ? *cluster.map_shared_rank(&cta_total, lane) : Sum{0.f, 0.f};
            Sum total{0.f, 0.f}, base{0.f, 0.f}, end{0.f, 0.f};
            for (int r = 0; r < ranks; ++r) {
                if (r == rank) base = total;
                total = total.plus(shuffle(mine, r));
                if (r == rank) end = total;
            }
            // Sums of fp32 values lose nothing at the low end of fp32's range, but u S has bits
            // below them: there all are compared in units of 2^-100.
            const bool tiny = total.hi < 0x1p-60f;
            if (tiny) {
                total = total.scaled(kUp);
                base = base.scaled(kUp);
                end = end.scaled(kUp);
                for (int g = lane; g < segs; g += 32) seg_sum[g] = seg_sum[g].scaled(kUp);
                __syncwarp();
            }
            // Sums that values are added to never shrink, and u S is below S: it falls into one part.
            const Sum border = total.times(fminf(fmaxf(u_last, 0.f), 0.99999994f));   // u in [0, 1)
            const bool here = !base.above(border) && end.above(border);
            int seg = segs - 1;
            if (here) {
                for (int g0 = 0; g0 < segs; g0 += 32) {
                    const unsigned hit = __ballot_sync(0xffffffffu, g0 + lane < segs && base.plus(seg_sum[g0 + lane]).above(border));
                    if (hit != 0u) {
                        seg = g0 + __ffs(hit) - 1;
                        break;
                    }
                }
            }
            if (lane == 0) {
                border_left = border.minus(here && seg > 0 ? base.plus(seg_sum[seg - 1]) : base);
                in_units = tiny;
                // A value that is infinite has left a sum that is NaN: nothing to draw from.
                owner = total.hi > 0.f ? (here ? seg : -1) : total.hi == 0.f ? kNothing : kNoSums;
                chosen = INT_MAX;
            }
        }
        __syncthreads();
        if (owner != kNothing) break;
        cluster.sync();                       // every CTA has read the totals: the second pass writes them
    }
    // The totals are read; no CTA ends before all have said so.
    auto arrived = cluster.barrier_arrive();
    const int seg = owner;
    if (seg <= kNothing && rank == 0 && tid == 0) raise_error(p.error_word, PA_DEVERR_TOKEN);
    if (seg >= 0) {
        // The first value whose running sum passes the border. (Where the two ways to sum part
        // by a rounding the walk may go on to the next segment, or end behind the last.)
        Sum upto{0.f, 0.f};
        const Sum border = border_left;
        int token = INT_MAX, last_positive = -1;
        for (int g = seg; g < segs && token == INT_MAX; ++g) {
            const int v = (seg0 + g) * kSegment + tid;
            Sum r{0.f, 0.f};
            if (v < V && v != left_out) add_excess(r, __ldg(pr + v), qr != nullptr ? __ldg(qr + v) : 0.f);
            if (in_units) r = r.scaled(kUp);
            Sum run = warp_scan(r, lane);
            if (lane == 31) warp_total[warp] = run;
            __syncthreads();
            Sum before = upto;
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) run = before.plus(run);
                before = before.plus(warp_total[w]);
            }
            upto = before;
            if (r.hi > 0.f) {
                last_positive = v;
                if (run.above(border)) atomicMin(&chosen, v);
            }
            __syncthreads();
            token = chosen;
        }
        if (token == INT_MAX) {
            // The last value that can be drawn: of the segments walked, else before them.
            __syncthreads();                  // every thread has read `chosen`
            if (tid == 0) chosen = -1;
            __syncthreads();
            for (int v = seg0 * kSegment + tid; last_positive < 0 && v < min(V, (seg0 + seg) * kSegment); v += kThreads)
                if (v != left_out && __ldg(pr + v) > (qr != nullptr ? __ldg(qr + v) : 0.f)) atomicMax(&chosen, v);
            if (last_positive >= 0) atomicMax(&chosen, last_positive);
            __syncthreads();
            token = chosen;
        }
        for (int i = tid; i <= Q; i += kThreads)
            p.out_tokens[static_cast<size_t>(s) * (Q + 1) + i] = i < a ? tokens[i] : i == a ? token : -1;
        if (tid == 0) {
            p.num_accepted[s] = a;
            if (p.lens_out != nullptr) p.lens_out[s] = rows - (d - a);
        }
    }
    cluster.barrier_wait(std::move(arrived));
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
    if (p.num_seqs == 0) return cudaSuccess;
    const long long sms = device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int segs = (p.vocab + kSegment - 1) / kSegment;
    // CTAs of a sequence: until they are one for each SM, two fit one. The last doubling only
    // where its clusters of eight all find room at once (37 sequences of 50,021 values: 12.7 us
    // with clusters of eight, 9 with four).
    int ranks = 1;
    while (ranks < kMaxCluster && ranks < segs) {
        const bool room = ranks < 4 || 5LL * p.num_seqs * 2 * ranks <= 8 * sms;
        if ((p.num_seqs * static_cast<long long>(ranks) >= sms || !room) && segs <= kMaxSegments * ranks) break;
        ranks *= 2;
    }
    const int per_cta = (segs + ranks - 1) / ranks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Sum) * static_cast<size_t>(per_cta);   // 32 KB at most
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, verify_kernel, p, per_cta);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace pa

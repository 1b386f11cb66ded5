// pa_decode_int4.cu -- decode attention over a 4-bit cache (row format:
// pa_int4.cuh), one CTA per (sequence, KV head, partition).
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) decode_int4_kernel(const DecodeParams p) {
    extern __shared__ float sm[];
    const int D = p.head_dim, Hkv = p.num_kv_heads, G = p.num_heads / Hkv, Q = p.num_queries;
    const int ncols = G * Q, P = p.partition_size;
    float* q = sm;                      // [ncols][D]
    float* sc = q + ncols * D;          // [ncols][P]
    float* ml = sc + ncols * P;         // [ncols][2]
    const int part = blockIdx.x, h = blockIdx.y % Hkv, s = blockIdx.y / Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = p.context_lens[s];
    if (n < 0 || n > p.context_cap || (n > 0 && n < Q)) {
        if (part == 0 && h == 0 && tid == 0) raise_error(p.error_word, PA_DEVERR_CONTEXT);
        return;
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
    auto qrow = [&](int c) {
        return (static_cast<size_t>(s) * Q + c / G) * p.num_heads + h * G + c % G;
    };
    if (n == 0) {
        if (part == 0)
            for (int i = tid; i < ncols * D; i += kThreads)
                out[qrow(i / D) * D + i % D] = __float2bfloat16_rn(0.f);
        return;
    }
    const int base = seq_row_base(n, p.window);
    const int lo = base + part * P, hi = min(n, lo + P);
    if (lo >= hi) return;
    const int nparts = (n - base + P - 1) / P;
    const int window = p.window > 0 ? p.window - (Q - 1) : 0;
    for (int i = tid; i < ncols * D; i += kThreads)
        q[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[qrow(i / D) * D + i % D]) * p.scale_log2;
    __syncthreads();
    auto row_of = [&](int i) -> long long {
        const int id = p.block_tables[static_cast<size_t>(s) * p.max_blocks_per_seq + i / p.block_size];
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) raise_error(p.error_word, PA_DEVERR_BLOCK_ID);
            return (static_cast<long long>(h)) * p.block_size;
        }
        return (static_cast<long long>(id) * Hkv + h) * p.block_size + i % p.block_size;
    };
    const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
    const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
    const uint32_t* kp = p.k_pairs;
    const uint32_t* vp = p.v_pairs;
    for (int i = lo + warp; i < hi; i += kThreads / 32) {
        const long long r = row_of(i);
        const float rl = int4_lo(kp[r]), rs = int4_step(kp[r]);
        for (int c = 0; c < ncols; ++c) {
            float acc = 0.f;
            for (int d = lane; d < D; d += 32) {
                const int b = kc[r * (D / 2) + d / 2];
                acc = fmaf(q[c * D + d], fmaf(rs, static_cast<float>((d & 1) ? b >> 4 : b & 15), rl), acc);
            }
            for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            const int last = n - Q + c / G;
            if (lane == 0)
                sc[c * P + i - lo] = (i > last || (window > 0 && i <= last - window)) ? -INFINITY : acc;
        }
    }
    __syncthreads();
    for (int c = warp; c < ncols; c += kThreads / 32) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < hi - lo; i += 32) m = fmaxf(m, sc[c * P + i]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -INFINITY ? 0.f : m;
        for (int i = lane; i < hi - lo; i += 32) {
            const float e = fast_exp2(sc[c * P + i] - ref);
            sc[c * P + i] = e;
            l += e;
        }
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            ml[2 * c] = m;
            ml[2 * c + 1] = l;
        }
    }
    __syncthreads();
    for (int c = 0; c < ncols; ++c)
        for (int d = tid; d < D; d += kThreads) {
            float o = 0.f;
            for (int i = lo; i < hi; ++i) {
                // A masked row's pair may be anything.
                if (sc[c * P + i - lo] == 0.f) continue;
                const long long r = row_of(i);
                const int b = vc[r * (D / 2) + d / 2];
                o = fmaf(sc[c * P + i - lo],
                         fmaf(int4_step(vp[r]), static_cast<float>((d & 1) ? b >> 4 : b & 15), int4_lo(vp[r])), o);
            }
            if (nparts == 1) {
                out[qrow(c) * D + d] = __float2bfloat16_rn(o / ml[2 * c + 1]);
            } else {
                const size_t slot = qrow(c) * p.max_parts + part;
                p.part_o[slot * D + d] = o;
                if (d == 0) {
                    p.part_ml[2 * slot] = ml[2 * c];
                    p.part_ml[2 * slot + 1] = ml[2 * c + 1];
                }
            }
        }
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams& p, cudaStream_t stream) {
    const int ncols = p.num_heads / p.num_kv_heads * p.num_queries;
    const size_t smem = sizeof(float) * (static_cast<size_t>(ncols) * (p.head_dim + p.partition_size + 2));
    decode_int4_kernel<<<dim3(p.max_parts, p.num_seqs * p.num_kv_heads), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa

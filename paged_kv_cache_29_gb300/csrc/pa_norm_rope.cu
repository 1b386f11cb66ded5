// pa_norm_rope.cu -- per-head norms of q and k and the rotation by position in
// one pass over the rows of a step or a prompt; the K rows go to a buffer, into
// their slots of a paged pool (V beside them), or quantised into a 4-bit cache.
//
//   y = x * (mean x^2 + eps)^(-1/2) * (w + offset),
//   (a, b) -> (a cos - b sin, b cos + a sin) for each pair of y,
//
// fp32 throughout, one rounding at the store.
//
// TPR lanes hold a row, 8 dims each; a pair's other half is 8 lanes' worth
// away (halves) or in the same lane (interleaved). A warp works on one token:
// its cosines and sines are loaded once and stay in registers for all the rows
// that the warp takes of it (rows part, part + splits, ... of the token's q, K
// and V heads).
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;

enum Dest { kOut, kPool, kPool4 };

__device__ __forceinline__ float round_to(float x, const float*) { return x; }
__device__ __forceinline__ float round_to(float x, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(x));
}

template <typename T, int TPR, Dest DEST>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsPerWarp = 32 / TPR;
    const int lane = threadIdx.x & 31;
    const int sub = lane / TPR, c = lane % TPR;
    const long long warp = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const long long t = warp / p.splits;
    const int part = static_cast<int>(warp - t * p.splits);
    if (t >= p.num_tokens) return;                       // whole warps

    const int D = p.head_dim;
    const bool live = 8 * c < D;
    const int half = p.rot_dim / 2;
    const bool turned = 8 * c < p.rot_dim;
    const bool second = !p.interleaved && 8 * c >= half;  // holds b's
    // This lane's cosines, and sines with the sign that its element takes.
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (p.rot_dim > 0) {
        bool ok = true;
        for (int a = 0; a < p.num_axes; ++a) {
            const int pos = __ldg(p.positions + static_cast<long long>(a) * p.num_tokens + t);
            ok = ok && pos >= 0 && pos < p.max_position;
        }
        if (!ok) {
            if (part == 0 && lane == 0) raise_error(p.error_word, PA_DEVERR_POSITION);
            return;
        }
        if (turned) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = p.interleaved ? 4 * c + e / 2 : 8 * c - (second ? half : 0) + e;
                const long long axis = p.pair_axis[i];
                const int pos = __ldg(p.positions + axis * p.num_tokens + t);
                const float* row = p.cos_sin + static_cast<long long>(pos) * p.rot_dim;
                const bool b = p.interleaved ? (e & 1) : second;
                cs[e] = __ldg(row + i);
                const float s = __ldg(row + half + i);
                sn[e] = b ? s : -s;
            }
        }
    }
    long long slot = -1;
    if constexpr (DEST != kOut) {
        slot = __ldg(p.slot_mapping + t);
        if (slot >= p.num_slots) {
            if (part == 0 && lane == 0) raise_error(p.error_word, PA_DEVERR_SLOT);
            slot = -1;
        }
    }
    const long long blk = slot >= 0 ? slot / p.block_size : 0;
    const int off = slot >= 0 ? static_cast<int>(slot - blk * p.block_size) : 0;
    const int Hq = p.num_heads, Hkv = p.num_kv_heads;
    const int rows = DEST == kOut ? Hq + Hkv : slot >= 0 ? Hq + 2 * Hkv : Hq;
    const int partner = p.interleaved ? 0 : (lane - c) + (second ? c - half / 8 : c + half / 8);

    for (int r0 = part * kRowsPerWarp; r0 < rows; r0 += p.splits * kRowsPerWarp) {
        const int r = r0 + sub;
        const bool on = r < rows && live;
        const bool is_q = r < Hq, is_v = r >= Hq + Hkv;
        const int h = is_q ? r : is_v ? r - Hq - Hkv : r - Hq;
        // The row's 8 elements as they are (V is copied bit for bit), and as fp32.
        constexpr int kVecs = sizeof(T) / 2;
        uint4 raw[kVecs];
        float x[8];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (on) {
            const T* src = is_q   ? static_cast<const T*>(p.q) + t * p.q_stride
                           : is_v ? static_cast<const T*>(p.v) + t * p.v_stride
                                  : static_cast<const T*>(p.k) + t * p.k_stride;
            const uint4* at = reinterpret_cast<const uint4*>(src + static_cast<long long>(h) * D + 8 * c);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) raw[i] = at[i];
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) ElemTraits<T>::unpack(raw[i], x + i * ElemTraits<T>::kPerChunk);
        const void* weight = is_q ? p.q_weight : is_v ? nullptr : p.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
        if (weight != nullptr && live) {
            const float inv = 1.0f / sqrtf(ss / static_cast<float>(D) + p.eps);
            float w[8];
            if (p.weight_bf16)
                load8(static_cast<const __nv_bfloat16*>(weight) + 8 * c, w);
            else
                load8(static_cast<const float*>(weight) + 8 * c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e] * inv * (w[e] + p.weight_offset);
        }
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float far = __shfl_sync(0xffffffffu, y[e], partner & 31);
            const float other = p.interleaved ? y[e ^ 1] : far;
            z[e] = turned ? fmaf(y[e], cs[e], other * sn[e]) : y[e];
        }
        if (is_q) {
            if (on)
                store8(static_cast<T*>(p.q_out) + t * p.q_out_stride + static_cast<long long>(h) * D + 8 * c, z);
        } else if (DEST == kOut) {
            if (on)
                store8(static_cast<T*>(p.k_out) + t * p.k_out_stride + static_cast<long long>(h) * D + 8 * c, z);
        }
        if constexpr (DEST != kOut) {
            const long long row = (blk * Hkv + h) * p.block_size + off;
            if constexpr (DEST == kPool) {
                if (on && is_v) {
                    uint4* at = reinterpret_cast<uint4*>(static_cast<T*>(p.v_cache) + row * D + 8 * c);
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) at[i] = raw[i];
                } else if (on && !is_q) {
                    store8(static_cast<T*>(p.k_cache) + row * D + 8 * c, z);
                }
            } else {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = is_v ? x[e] : round_to(z[e], static_cast<const T*>(nullptr));
                const uint32_t pair = int4_row_pair<TPR>(u, live);
                if (on && !is_q) {
                    reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                                                row * (D / 2))[c] = int4_codes(u, pair);
                    if (c == 0) static_cast<uint32_t*>(is_v ? p.v_params : p.k_params)[row] = pair;
                }
            }
        }
    }
}

template <typename T, Dest DEST>
cudaError_t run(NormRopeParams p, cudaStream_t stream) {
    const int tpr = p.head_dim <= 64 ? 8 : p.head_dim <= 128 ? 16 : 32;
    const int rows = p.num_heads + p.num_kv_heads * (DEST == kOut ? 1 : 2);
    const int passes = (rows * tpr + 31) / 32;
    p.splits = passes < 4 ? passes : 4;
    const long long warps = static_cast<long long>(p.num_tokens) * p.splits;
    const long long blocks = (warps * 32 + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    };
    return tpr == 8    ? go(norm_rope_kernel<T, 8, DEST>)
           : tpr == 16 ? go(norm_rope_kernel<T, 16, DEST>)
                       : go(norm_rope_kernel<T, 32, DEST>);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, pa_dtype dtype, cudaStream_t stream) {
    const bool bf = dtype == PA_DTYPE_BF16;
    if (p.k_params != nullptr)
        return bf ? run<__nv_bfloat16, kPool4>(p, stream) : run<float, kPool4>(p, stream);
    if (p.k_cache != nullptr)
        return bf ? run<__nv_bfloat16, kPool>(p, stream) : run<float, kPool>(p, stream);
    return bf ? run<__nv_bfloat16, kOut>(p, stream) : run<float, kOut>(p, stream);
}

}  // namespace pa

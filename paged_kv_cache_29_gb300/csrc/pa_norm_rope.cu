// pa_norm_rope.cu -- per-head norms of q and k and the rotation by position in
// one pass over the rows of a step or a prompt; the K rows go to a buffer, into
// their slots of a paged pool (V beside them), or quantised into a 4-bit cache.
//
//   y = x * (mean x^2 + eps)^(-1/2) * (w + offset),
//   (a, b) -> (a cos - b sin, b cos + a sin) for each pair of y,
//
// fp32 throughout, one rounding at the store.
//
// TPR lanes hold a row, 8 dims each, dealt so that both halves of a pair are in
// one lane: with pairs (i, i + rot / 2) lane c < rot / 8 holds dims 4 c .. + 3
// and rot / 2 + 4 c .. + 3, every other lane dims 8 c .. + 7. Either way a lane
// turns pairs 4 c .. 4 c + 3, so four cosines and four sines, loaded once per
// token, serve every row that the warp takes of it; nothing but the sum of
// squares crosses lanes. A warp works on one token: passes part, part + splits,
// ... of its q, K and V rows, numbered through, U passes' loads in flight.
//
// Bound by memory once there are a few thousand tokens: 16,384 tokens of 32 q, K and
// V heads of 128 dims (bf16, K and V into a pool) 128.3 us, 6,345 GB/s beside a
// plain copy's 6,797; 4,099 tokens with 8 KV heads and three axes 18.0 us, 4,780
// GB/s: all 4,099 warps are resident at once, so that the chain of each (positions,
// table rows, first store) and the last warps' end are not hidden behind others.
// 128 tokens 3.8 us, that chain alone.
#include <atomic>

#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;

enum Dest { kOut, kPool, kPool4 };

// Four consecutive elements.
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    using Raw = uint2;
    __device__ static __forceinline__ void unpack(const Raw& r, float* x) {
        x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
    }
    __device__ static __forceinline__ Raw pack(const float* x) {
        return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
};
template <>
struct Quad<float> {
    using Raw = uint4;
    __device__ static __forceinline__ void unpack(const Raw& r, float* x) {
        x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
    }
    __device__ static __forceinline__ Raw pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

template <typename T, int TPR, Dest DEST>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    // A programmatic dependent itself: resident before the kernel ahead of it on
    // the stream is done (2.8 us against 3.1 for a call among its like), it waits
    // for that one before it touches memory, and so does a decode call after it.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    using Q = Quad<T>;
    using Raw = typename Q::Raw;
    constexpr int kRowsPerPass = 32 / TPR;
    constexpr int U = 2;                                 // passes of a batch
    const int lane = threadIdx.x & 31;
    const int sub = lane / TPR, c = lane % TPR;
    // Unsigned: the last CTA's warps may pass 2^31.
    const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t token = p.splits == 1 ? warp : warp / static_cast<uint32_t>(p.splits);
    const int part = static_cast<int>(warp - token * p.splits);
    if (token >= static_cast<uint32_t>(p.num_tokens)) return;   // whole warps
    const long long t = token;

    const int D = p.head_dim, half = p.rot_dim / 2;
    const bool live = 8 * c < D, turned = 8 * c < p.rot_dim;
    const bool split = turned && !p.interleaved;         // the lane holds two halves' quads
    const int d0 = split ? 4 * c : 8 * c, d1 = split ? half + 4 * c : 8 * c + 4;

    // Rows of q and K are loaded a batch of U passes ahead of their use, the
    // first batch of q before the positions are known.
    Raw raw[U][2];
    auto load_batch = [&](const T* from, int rows, int pass) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (pass + u * p.splits) * kRowsPerPass + sub;
            raw[u][0] = raw[u][1] = Raw{};
            if (h < rows && live) {
                const T* row = from + static_cast<long long>(h) * D;
                raw[u][0] = *reinterpret_cast<const Raw*>(row + d0);
                raw[u][1] = *reinterpret_cast<const Raw*>(row + d1);
            }
        }
    };
    const T* const q = static_cast<const T*>(p.q) + t * p.q_stride;
    const T* const k = static_cast<const T*>(p.k) + t * p.k_stride;
    int k_part = part + p.k_shift, v_part = part + p.v_shift;
    if (k_part >= p.splits) k_part -= p.splits;
    if (v_part >= p.splits) v_part -= p.splits;
    if (part * kRowsPerPass < p.num_heads)
        load_batch(q, p.num_heads, part);
    else
        load_batch(k, p.num_kv_heads, k_part);

    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
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
            const uint32_t axes = *reinterpret_cast<const uint32_t*>(p.pair_axis + 4 * c);
            if (axes == (axes & 0xffu) * 0x01010101u) {  // one axis: whole quads of the table
                const int pos = __ldg(p.positions + static_cast<long long>(axes & 0xffu) * p.num_tokens + t);
                const float* row = p.cos_sin + static_cast<long long>(pos) * p.rot_dim + 4 * c;
                const float4 a = __ldg(reinterpret_cast<const float4*>(row));
                const float4 b = __ldg(reinterpret_cast<const float4*>(row + half));
                cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
                sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long axis = (axes >> (8 * i)) & 0xffu;
                    const int pos = __ldg(p.positions + axis * p.num_tokens + t);
                    const float* row = p.cos_sin + static_cast<long long>(pos) * p.rot_dim + 4 * c + i;
                    cs[i] = __ldg(row);
                    sn[i] = __ldg(row + half);
                }
            }
        }
    }
    long long row0 = 0;                                  // the slot's row of KV head 0 in the pool
    bool append = false;
    if constexpr (DEST != kOut) {
        const long long slot = __ldg(p.slot_mapping + t);
        append = slot >= 0 && slot < p.num_slots;
        if (slot >= p.num_slots && part == 0 && lane == 0) raise_error(p.error_word, PA_DEVERR_SLOT);
        if (append) row0 = slot_row(slot, p.num_slots, p.num_kv_heads, p.block_size);
    }

    // Normed and turned rows of q or K, passes start, start + splits, ...; raw holds
    // the first batch, and that of K (then_k) at q's end.
    auto turn_rows = [&](const T* from, int rows, int start, const void* weight, bool then_k, auto&& put) {
        float w[8];
        if (weight != nullptr && live) {
            if (p.weight_bf16) {
                const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(weight);
                Quad<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint2*>(s + d0)), w);
                Quad<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint2*>(s + d1)), w + 4);
            } else {
                const float* s = static_cast<const float*>(weight);
                Quad<float>::unpack(__ldg(reinterpret_cast<const uint4*>(s + d0)), w);
                Quad<float>::unpack(__ldg(reinterpret_cast<const uint4*>(s + d1)), w + 4);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] += p.weight_offset;
        }
        for (int pass = start; pass * kRowsPerPass < rows; pass += U * p.splits) {
            float in[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Q::unpack(raw[u][0], in[u]);
                Q::unpack(raw[u][1], in[u] + 4);
            }
            if ((pass + U * p.splits) * kRowsPerPass < rows)
                load_batch(from, rows, pass + U * p.splits);
            else if (then_k)
                load_batch(k, p.num_kv_heads, k_part);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int first = (pass + u * p.splits) * kRowsPerPass;
                if (first >= rows) break;                // whole warps
                float* const x = in[u];
                if (weight != nullptr) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int o = TPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = 1.0f / sqrtf(ss / static_cast<float>(D) + p.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= inv * w[e];
                }
                if (split) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[i], b = x[i + 4];
                        x[i] = fmaf(a, cs[i], -(b * sn[i]));
                        x[i + 4] = fmaf(b, cs[i], a * sn[i]);
                    }
                } else if (turned) {                     // other dims pass through, infinities and zeros' signs too
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = fmaf(a, cs[i], -(b * sn[i]));
                        x[2 * i + 1] = fmaf(b, cs[i], a * sn[i]);
                    }
                }
                put(first + sub, first + sub < rows && live, x);
            }
        }
    };
    auto store_row = [&](void* to, bool on, const float* x) {
        if (on) {
            *reinterpret_cast<Raw*>(static_cast<T*>(to) + d0) = Q::pack(x);
            *reinterpret_cast<Raw*>(static_cast<T*>(to) + d1) = Q::pack(x + 4);
        }
    };
    // A row's 8 values of this lane as codes (dims a .. + 3 and b .. + 3).
    auto store_row4 = [&](bool v, long long row, bool on, const float* x, int a, int b) {
        const uint32_t pair = int4_row_pair<TPR, sizeof(T) == 2>(x, on);
        if (on) {
            uint32_t codes;
            int4_codes<8>(x, pair, &codes);
            uint8_t* to = static_cast<uint8_t*>(v ? p.v_cache : p.k_cache) + row * (D / 2);
            *reinterpret_cast<uint16_t*>(to + a / 2) = static_cast<uint16_t>(codes);
            *reinterpret_cast<uint16_t*>(to + b / 2) = static_cast<uint16_t>(codes >> 16);
            if (c == 0) static_cast<uint32_t*>(v ? p.v_params : p.k_params)[row] = pair;
        }
    };

    T* const q_out = static_cast<T*>(p.q_out) + t * p.q_out_stride;
    turn_rows(q, p.num_heads, part, p.q_weight, DEST == kOut || append,
              [&](int h, bool on, const float* x) { store_row(q_out + static_cast<long long>(h) * D, on, x); });
    if constexpr (DEST == kOut) {
        T* const k_out = static_cast<T*>(p.k_out) + t * p.k_out_stride;
        turn_rows(k, p.num_kv_heads, k_part, p.k_weight, false,
                  [&](int h, bool on, const float* x) { store_row(k_out + static_cast<long long>(h) * D, on, x); });
    } else {
        if (!append) return;
        const T* const v = static_cast<const T*>(p.v) + t * p.v_stride;
        if constexpr (DEST == kPool) {
            turn_rows(k, p.num_kv_heads, k_part, p.k_weight, false, [&](int h, bool on, const float* x) {
                store_row(static_cast<T*>(p.k_cache) + (row0 + static_cast<long long>(h) * p.block_size) * D, on, x);
            });
            // V as it is, 16 bytes a lane.
            constexpr int kVecs = sizeof(T) / 2, UV = 4;
            for (int pass = v_part; pass * kRowsPerPass < p.num_kv_heads; pass += UV * p.splits) {
                uint4 vec[UV][kVecs];
#pragma unroll
                for (int u = 0; u < UV; ++u) {
                    const int h = (pass + u * p.splits) * kRowsPerPass + sub;
                    if (h < p.num_kv_heads && live) {
                        const uint4* at = reinterpret_cast<const uint4*>(v + static_cast<long long>(h) * D + 8 * c);
#pragma unroll
                        for (int i = 0; i < kVecs; ++i) vec[u][i] = at[i];
                    }
                }
#pragma unroll
                for (int u = 0; u < UV; ++u) {
                    const int h = (pass + u * p.splits) * kRowsPerPass + sub;
                    if (h < p.num_kv_heads && live) {
                        uint4* at = reinterpret_cast<uint4*>(
                            static_cast<T*>(p.v_cache) + (row0 + static_cast<long long>(h) * p.block_size) * D + 8 * c);
#pragma unroll
                        for (int i = 0; i < kVecs; ++i) at[i] = vec[u][i];
                    }
                }
            }
        } else {
            turn_rows(k, p.num_kv_heads, k_part, p.k_weight, false, [&](int h, bool on, float* x) {
                // The codes are those of the row as pa_norm_rope would store it.
                float y[8];
                Q::unpack(Q::pack(x), y);
                Q::unpack(Q::pack(x + 4), y + 4);
                store_row4(false, row0 + static_cast<long long>(h) * p.block_size, on, y, d0, d1);
            });
            for (int first = v_part * kRowsPerPass; first < p.num_kv_heads; first += p.splits * kRowsPerPass) {
                const int h = first + sub;
                const bool on = h < p.num_kv_heads && live;
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
                if (on) load8(v + static_cast<long long>(h) * D + 8 * c, x);
                store_row4(true, row0 + static_cast<long long>(h) * p.block_size, on, x, 8 * c, 8 * c + 4);
            }
        }
    }
}

template <typename T, int TPR, Dest DEST>
cudaError_t run(NormRopeParams p, cudaStream_t stream) {
    auto kernel = norm_rope_kernel<T, TPR, DEST>;
    static std::atomic<int> cached_ctas[kMaxDevices];
    int resident = 0;
    cudaError_t err = resident_ctas(kernel, kThreads, cached_ctas, &resident);
    if (err != cudaSuccess) return err;
    resident *= kThreads / 32;
    // Warps per token: as many as are resident at once, with equal shares of the
    // passes. 32 q heads and 8 KV heads of 128 dims (24 passes), bf16, into a pool,
    // 4,256 warps: 300 tokens 4.5 us with 12 warps each (10.0 with one, 6.2 with
    // 24), 1,000 tokens 7.6 with four (12.3; six 8.9), 2,000 tokens 12.5 with two
    // (17.2; three 15.4). More tokens take one warp each, whose table rows and
    // weights serve every row: 4,099 tokens 20.5 us (two 22.4), 16,384 tokens 70.9 (77.9).
    const int q_passes = (p.num_heads * TPR + 31) / 32, kv_passes = (p.num_kv_heads * TPR + 31) / 32;
    const int passes = q_passes + (DEST == kOut ? 1 : 2) * kv_passes;
    const int most = max(1, min(passes, resident / p.num_tokens));
    const int share = (passes + most - 1) / most;
    p.splits = (passes + share - 1) / share;
    p.k_shift = (p.splits - q_passes % p.splits) % p.splits;
    p.v_shift = (p.splits - (q_passes + kv_passes) % p.splits) % p.splits;
    const long long warps = static_cast<long long>(p.num_tokens) * p.splits;
    const long long blocks = (warps * 32 + kThreads - 1) / kThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, p);
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <typename T, Dest DEST>
cudaError_t pick(const NormRopeParams& p, cudaStream_t stream) {
    return p.head_dim <= 64    ? run<T, 8, DEST>(p, stream)
           : p.head_dim <= 128 ? run<T, 16, DEST>(p, stream)
                               : run<T, 32, DEST>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, pa_dtype dtype, cudaStream_t stream) {
    const bool bf = dtype == PA_DTYPE_BF16;
    if (p.k_params != nullptr)
        return bf ? pick<__nv_bfloat16, kPool4>(p, stream) : pick<float, kPool4>(p, stream);
    if (p.k_cache != nullptr)
        return bf ? pick<__nv_bfloat16, kPool>(p, stream) : pick<float, kPool>(p, stream);
    return bf ? pick<__nv_bfloat16, kOut>(p, stream) : pick<float, kOut>(p, stream);
}

}  // namespace pa

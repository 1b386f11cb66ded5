// pa_append_int4.cu -- the quantising append into a 4-bit cache and the gather
// of its rows as plain values (row format: pa_int4.cuh). Both are one pass over
// memory. A warp works on one token (or one row of one sequence) and goes over
// its KV heads, TPR lanes per head: the token's slot (the row's block) is looked
// up once, reads of new rows and writes of values run over
// consecutive heads, contiguous.
//
// Measured at 65,536 tokens, 8 KV heads of 128 dims, blocks of 16 in no order:
//            bf16 rows             fp32 rows
//   append   62.2 us, 5,461 GB/s   89.3 us, 6,809 GB/s
//   gather   54.2 us, 6,271 GB/s   92.4 us, 6,579 GB/s
// beside a plain copy's 6,797 GB/s: memory bounds all but the append of bf16 rows, where
// it is the arithmetic per element (ALU pipe 60 % busy, issue 68 %): unpacking, the
// minimum and maximum, five fp32 operations for the quotient, packing.
#include <algorithm>
#include <atomic>

#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarpsPerCta = kThreads / 32;
// CTAs of the gather, in times what is resident (nine per SM of the bf16 kernel), so
// that sequences of 16 to 8,192 rows spread: append and gather of 128 of them 365.1
// us, 365.5 with eleven, 366.2 with ten, 385 with three and a half, 363.4 with sixteen.
// The gather of 32 equal sequences: 54.3 us, 54.8, 54.7, 55.9 and 54.5.
constexpr int kGatherWaves = 12;

// Sixteen elements as they are loaded, their fp32 values, and the row's pair.
template <typename T, int TPR>
struct Sixteen;
template <int TPR>
struct Sixteen<float, TPR> {
    float4 v[4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void values(float* x) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * i] = v[i].x; x[4 * i + 1] = v[i].y; x[4 * i + 2] = v[i].z; x[4 * i + 3] = v[i].w;
        }
    }
    __device__ __forceinline__ uint32_t pair(bool on) const {
        float mn = INFINITY, mx = -INFINITY;
        if (on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mn = fminf(fminf(fminf(mn, v[i].x), fminf(v[i].y, v[i].z)), v[i].w);
                mx = fmaxf(fmaxf(fmaxf(mx, v[i].x), fmaxf(v[i].y, v[i].z)), v[i].w);
            }
        }
#pragma unroll
        for (int off = TPR / 2; off > 0; off >>= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        return int4_pair<false>(mn, mx);
    }
};
template <int TPR>
struct Sixteen<__nv_bfloat16, TPR> {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v[0] = __ldg(reinterpret_cast<const uint4*>(p));
        v[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void clear() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void values(float* x) const {
        ElemTraits<__nv_bfloat16>::unpack(v[0], x);
        ElemTraits<__nv_bfloat16>::unpack(v[1], x + 8);
    }
    // The minimum and minus the maximum side by side as bf16: one shuffle and
    // one packed minimum per level.
    __device__ __forceinline__ uint32_t pair(bool on) const {
        auto h2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        auto u = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); };
        auto lo4 = [&](const uint4& a) { return __hmin2(__hmin2(h2(a.x), h2(a.y)), __hmin2(h2(a.z), h2(a.w))); };
        auto hi4 = [&](const uint4& a) { return __hmax2(__hmax2(h2(a.x), h2(a.y)), __hmax2(h2(a.z), h2(a.w))); };
        const uint32_t mn = u(__hmin2(lo4(v[0]), lo4(v[1])));
        const uint32_t mx = u(__hmax2(hi4(v[0]), hi4(v[1]))) ^ 0x80008000u;
        uint32_t m = u(__hmin2(h2(__byte_perm(mn, mx, 0x5410)), h2(__byte_perm(mn, mx, 0x7632))));
        if (!on) m = 0x7f807f80u;                        // +inf twice
#pragma unroll
        for (int off = TPR / 2; off > 0; off >>= 1)
            m = u(__hmin2(h2(m), h2(__shfl_xor_sync(0xffffffffu, m, off))));
        return int4_pair<true>(bf16_lo(m), -bf16_hi(m));
    }
};

// 16 dims a lane: the pair and its reciprocal, which every lane of a row works
// out, cost four rows of a pass once. A pass takes K and V of the same heads, whose
// offsets are the same: 62.1 us at the size above (five CTAs of twice the threads 63.7;
// with K's and V's passes apart 69.1, and 79.1 with one fp32 value per instruction instead
// of two). Ten CTAs on an SM (fp32 nine): with eight 66.1. Codes of four dims joined by
// an exact fp32 FMA instead of shifted sums: 3 us more.
template <typename TIn, int TPR>
__global__ void __launch_bounds__(kThreads, sizeof(TIn) == 2 ? 10 : 9)
append_int4_kernel(const TIn* __restrict__ k_new, const TIn* __restrict__ v_new,
                   const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
                   uint8_t* __restrict__ v_cache, uint32_t* __restrict__ k_params,
                   uint32_t* __restrict__ v_params, int num_tokens, int splits, int head_dim,
                   int num_kv_heads, int block_size, long long num_slots, int32_t* error_word) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsPerPass = 32 / TPR;
    const int lane = threadIdx.x & 31;
    const int sub = lane / TPR, c = lane % TPR;
    const bool live = 16 * c < head_dim;
    // Unsigned: the last CTA's warps may pass 2^31.
    const uint32_t warp = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
    const uint32_t t = splits == 1 ? warp : warp / static_cast<uint32_t>(splits);
    const int part = static_cast<int>(warp - t * splits);
    if (t >= static_cast<uint32_t>(num_tokens)) return;
    const long long slot = __ldg(slot_mapping + t);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (part == 0 && lane == 0) raise_error(error_word, PA_DEVERR_SLOT);
        return;
    }
    const long long row0 = slot_row(slot, num_slots, num_kv_heads, block_size);
    const size_t from = static_cast<size_t>(t) * num_kv_heads * head_dim + 16 * c;
    const size_t codes0 = static_cast<size_t>(row0) * (head_dim / 2) + 8 * c;
    const size_t code_stride = static_cast<size_t>(block_size) * (head_dim / 2);   // between heads
    // A pass takes K and V of kRowsPerPass heads.
    for (int h0 = part * kRowsPerPass; h0 < num_kv_heads; h0 += splits * kRowsPerPass) {
        const size_t h = h0 + sub;
        const bool on = h < num_kv_heads && live;
        Sixteen<TIn, TPR> in[2];
        in[0].clear();
        in[1].clear();
        if (on) {
            in[0].load(k_new + from + h * head_dim);
            in[1].load(v_new + from + h * head_dim);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint32_t pair = in[v].pair(on);
            if (on) {
                float x[16];
                in[v].values(x);
                uint32_t codes[2];
                int4_codes<16>(x, pair, codes);
                *reinterpret_cast<uint2*>((v ? v_cache : k_cache) + codes0 + h * code_stride) =
                    make_uint2(codes[0], codes[1]);
                if (c == 0) (v ? v_params : k_params)[row0 + h * block_size] = pair;
            }
        }
    }
}

// The values of a row of L words, one in each of the first L of its lanes; every
// lane of the warp takes part (on: this one stores). bf16: lane c stores its own
// word's eight dims, 16 bytes; the FMA c s + lo of two dims at a time rounds the exact
// sum once (c, s and lo are bf16 values; 128 + c is the bf16 bits 0x4300 | c).
// fp32: eight dims are 32 bytes, and two 16-byte stores of them would each touch
// every other half sector, so lane c stores quads c and c + L of the row instead,
// taken from the lanes that hold their words (the 65,536 rows above: 94.3 us against
// 139.6).
template <int TPR>
__device__ __forceinline__ void put_values(__nv_bfloat16* row, uint32_t w, uint32_t pair, int c, int, bool on) {
    if (!on) return;
    auto h2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    auto u = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); };
    const __nv_bfloat162 s = h2(__byte_perm(pair, 0u, 0x3232)), lo = h2(__byte_perm(pair, 0u, 0x1010));
    uint32_t r[4];                                       // dims (e, e + 4)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t bits = ((w >> (4 * e)) & 0x000f000fu) | 0x43004300u;
        r[e] = u(__hfma2(__hsub2(h2(bits), h2(0x43004300u)), s, lo));
    }
    *reinterpret_cast<uint4*>(row + 8 * c) = make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                                                        __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
}
template <int TPR>
__device__ __forceinline__ void put_values(float* row, uint32_t w, uint32_t pair, int c, int L, bool on) {
    const float lo = int4_lo(pair), step = int4_step(pair);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int quad = c + k * L;
        const uint32_t word = __shfl_sync(0xffffffffu, w, quad / 2, TPR) >> (16 * (quad & 1));
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)           // 2^23 + c is the fp32 bits 0x4b000000 | c
            x[e] = fmaf(step, __uint_as_float(((word >> (4 * e)) & 15u) | 0x4b000000u) - 8388608.f, lo);
        if (on) *reinterpret_cast<float4*>(row + 4 * quad) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

template <typename TOut, int TPR>
__global__ void __launch_bounds__(kThreads, 9)
gather_int4_kernel(const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                   const uint32_t* __restrict__ k_params, const uint32_t* __restrict__ v_params,
                   const int32_t* __restrict__ block_tables,
                   const int32_t* __restrict__ context_lens,
                   const int64_t* __restrict__ row_starts, TOut* __restrict__ k_out,
                   TOut* __restrict__ v_out, long long num_rows, int num_kv_heads, int head_dim,
                   int block_size, int num_blocks, int max_blocks_per_seq, int context_cap,
                   int32_t* error_word) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsPerPass = 32 / TPR;
    constexpr int U = 4;                           // passes in flight
    const int s = blockIdx.y;
    const int n = __ldg(context_lens + s);
    const long long start = __ldg(row_starts + s);
    if (n < 0 || n > context_cap || start < 0 || start > num_rows - n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(error_word, PA_DEVERR_CONTEXT);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int sub = lane / TPR, c = lane % TPR;
    const int words = head_dim / 8;
    const bool live = c < words;
    const int32_t* table = block_tables + static_cast<size_t>(s) * max_blocks_per_seq;
    const uint32_t stride = gridDim.x * kWarpsPerCta;
    // Unsigned: the row after the last may pass 2^31. Block ids a row ahead.
    const uint32_t un = static_cast<uint32_t>(n), ubs = static_cast<uint32_t>(block_size);
    uint32_t row = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
    int id_next = row < un ? __ldg(table + row / ubs) : 0;
    for (; row < un; row += stride) {
        const int id = id_next;
        if (row + stride < un) id_next = __ldg(table + (row + stride) / ubs);
        if (id < 0 || id >= num_blocks) {
            if (lane == 0) raise_error(error_word, PA_DEVERR_BLOCK_ID);
            continue;
        }
        const size_t in0 = static_cast<size_t>(id) * num_kv_heads * block_size + row % ubs;
        const size_t out0 = (static_cast<size_t>(start) + row) * num_kv_heads * head_dim;
        for (int pass = 0; pass * kRowsPerPass < num_kv_heads; pass += U) {
            uint32_t w[U][2], pair[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (pass + u) * kRowsPerPass + sub;
                w[u][0] = w[u][1] = pair[u][0] = pair[u][1] = 0u;
                if (h < num_kv_heads && live) {
                    const size_t r = in0 + static_cast<size_t>(h) * block_size;
                    w[u][0] = __ldg(reinterpret_cast<const uint32_t*>(k_cache + r * (head_dim / 2)) + c);
                    w[u][1] = __ldg(reinterpret_cast<const uint32_t*>(v_cache + r * (head_dim / 2)) + c);
                    pair[u][0] = __ldg(k_params + r);
                    pair[u][1] = __ldg(v_params + r);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (pass + u) * kRowsPerPass + sub;
                const bool on = h < num_kv_heads && live;
                const size_t to = out0 + static_cast<size_t>(h) * head_dim;
                put_values<TPR>(k_out + to, w[u][0], pair[u][0], c, words, on);
                put_values<TPR>(v_out + to, w[u][1], pair[u][1], c, words, on);
            }
        }
    }
}

}  // namespace

namespace {

template <typename TIn, int TPR>
cudaError_t run_append(const TIn* k_new, const TIn* v_new, const int64_t* slot_mapping, uint8_t* k_cache,
                       uint8_t* v_cache, uint32_t* k_params, uint32_t* v_params, int num_tokens,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks, int32_t* error_word,
                       cudaStream_t stream) {
    auto kernel = append_int4_kernel<TIn, TPR>;
    static std::atomic<int> cached_ctas[kMaxDevices];
    int resident = 0;
    const cudaError_t err = resident_ctas(kernel, kThreads, cached_ctas, &resident);
    if (err != cudaSuccess) return err;
    // With few tokens, as many warps as the device holds at once share a token's heads in
    // equal parts. 32 KV heads of bf16 (8 passes), 40 warps on an SM: 1,000 tokens 5.9 us
    // with four warps each (two 6.9, six 6.5), 1,500 tokens 7.7 with four (two 8.9, one
    // 12.7), 3,000 tokens 14.0 with two (one 16.6). fp32, 36 warps on an SM: 2,000 tokens
    // 15.1 us with two; three, the count for 40 warps on an SM, 17.6.
    const int passes = static_cast<int>((static_cast<long long>(num_kv_heads) * TPR + 31) / 32);
    const int most = max(1, min(passes, resident * kWarpsPerCta / num_tokens));
    const int share = (passes + most - 1) / most;
    const int splits = (passes + share - 1) / share;
    const long long blocks = (static_cast<long long>(num_tokens) * splits + kWarpsPerCta - 1) / kWarpsPerCta;
    kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        k_new, v_new, slot_mapping, k_cache, v_cache, k_params, v_params, num_tokens, splits, head_dim,
        num_kv_heads, block_size, static_cast<long long>(num_blocks) * block_size, error_word);
    return cudaGetLastError();
}

template <typename TOut, int TPR>
cudaError_t run_gather(const uint8_t* k_cache, const uint8_t* v_cache, const uint32_t* k_params,
                       const uint32_t* v_params, const int32_t* block_tables, const int32_t* context_lens,
                       const int64_t* row_starts, TOut* k_out, TOut* v_out, long long num_rows, int num_seqs,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks, int max_blocks_per_seq,
                       int max_context_len, int32_t* error_word, cudaStream_t stream) {
    auto kernel = gather_int4_kernel<TOut, TPR>;
    static std::atomic<int> cached_ctas[kMaxDevices];
    int resident = 0;
    cudaError_t err = resident_ctas(kernel, kThreads, cached_ctas, &resident);
    if (err != cudaSuccess) return err;
    // Rows beyond a sequence's length cost nothing but a CTA's look at it, so the
    // sequences share a bounded number of CTAs, at most one warp per row.
    const long long rows = (static_cast<long long>(max_context_len) + kWarpsPerCta - 1) / kWarpsPerCta;
    const long long share = (static_cast<long long>(kGatherWaves) * resident + num_seqs - 1) / num_seqs;
    const long long bx = std::max(1LL, std::min(rows, share));
    for (int s0 = 0; s0 < num_seqs; s0 += 65535) {   // grid.y holds 65,535 sequences
        const int m = num_seqs - s0 < 65535 ? num_seqs - s0 : 65535;
        kernel<<<dim3(static_cast<unsigned>(bx), static_cast<unsigned>(m)), kThreads, 0, stream>>>(
            k_cache, v_cache, k_params, v_params, block_tables + static_cast<size_t>(s0) * max_blocks_per_seq,
            context_lens + s0, row_starts + s0, k_out, v_out, num_rows, num_kv_heads, head_dim, block_size,
            num_blocks, max_blocks_per_seq, max_context_len, error_word);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_append_int4(const void* k_new, const void* v_new, pa_dtype new_dtype,
                               const int64_t* slot_mapping, void* k_cache, void* v_cache,
                               void* k_params, void* v_params, int num_tokens, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, int32_t* error_word,
                               cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    auto pick = [&](auto tag) {
        using TIn = decltype(tag);
        auto run = head_dim <= 64 ? run_append<TIn, 4> : head_dim <= 128 ? run_append<TIn, 8> : run_append<TIn, 16>;
        return run(static_cast<const TIn*>(k_new), static_cast<const TIn*>(v_new), slot_mapping,
                   static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), static_cast<uint32_t*>(k_params),
                   static_cast<uint32_t*>(v_params), num_tokens, num_kv_heads, head_dim, block_size, num_blocks,
                   error_word, stream);
    };
    return new_dtype == PA_DTYPE_BF16 ? pick(__nv_bfloat16{}) : pick(float{});
}

cudaError_t launch_gather_int4(const void* k_cache, const void* v_cache, const void* k_params,
                               const void* v_params, const int32_t* block_tables,
                               const int32_t* context_lens, const int64_t* row_starts,
                               void* k_out, void* v_out, pa_dtype out_dtype, long long num_rows,
                               int num_seqs, int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, int max_blocks_per_seq, int max_context_len,
                               int32_t* error_word, cudaStream_t stream) {
    if (num_seqs == 0) return cudaSuccess;
    auto pick = [&](auto tag) {
        using TOut = decltype(tag);
        auto run = head_dim <= 64 ? run_gather<TOut, 8> : head_dim <= 128 ? run_gather<TOut, 16> : run_gather<TOut, 32>;
        return run(static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                   static_cast<const uint32_t*>(k_params), static_cast<const uint32_t*>(v_params), block_tables,
                   context_lens, row_starts, static_cast<TOut*>(k_out), static_cast<TOut*>(v_out), num_rows, num_seqs,
                   num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq, max_context_len, error_word,
                   stream);
    };
    return out_dtype == PA_DTYPE_BF16 ? pick(__nv_bfloat16{}) : pick(float{});
}

}  // namespace pa

// pa_append_int4.cu -- the quantising append into a 4-bit cache and the gather
// of its rows as plain values (row format: pa_int4.cuh). Both are one pass over
// memory. A warp works on one token (or one row of one sequence) and goes over
// its KV heads, TPR lanes per head with 8 dims each: the token's slot (the row's
// block) is looked up once, reads of new rows and writes of values run over
// consecutive heads, contiguous.
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpsPerCta = kThreads / 32;
// Warps that fill the device (16 per SM); with fewer tokens than that, several
// warps share a token's heads.
constexpr long long kFillWarps = 2432;
#ifndef PA_GX
#define PA_GX 4864
#endif

// Eight elements as they are loaded, their fp32 values, and the row's pair.
template <typename T, int TPR>
struct Eight;
template <int TPR>
struct Eight<float, TPR> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void values(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ uint32_t pair(bool on) const {
        float x[8];
        values(x);
        return int4_row_pair<TPR>(x, on);
    }
};
template <int TPR>
struct Eight<__nv_bfloat16, TPR> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void values(float* x) const { ElemTraits<__nv_bfloat16>::unpack(v, x); }
    // The minimum and minus the maximum side by side as bf16: one shuffle and
    // one packed minimum per level.
    __device__ __forceinline__ uint32_t pair(bool on) const {
        auto h2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        auto u = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); };
        const uint32_t mn = u(__hmin2(__hmin2(h2(v.x), h2(v.y)), __hmin2(h2(v.z), h2(v.w))));
        const uint32_t mx = u(__hmax2(__hmax2(h2(v.x), h2(v.y)), __hmax2(h2(v.z), h2(v.w)))) ^ 0x80008000u;
        uint32_t m = u(__hmin2(h2(__byte_perm(mn, mx, 0x5410)), h2(__byte_perm(mn, mx, 0x7632))));
        if (!on) m = 0x7f807f80u;                        // +inf twice
#pragma unroll
        for (int off = TPR / 2; off > 0; off >>= 1)
            m = u(__hmin2(h2(m), h2(__shfl_xor_sync(0xffffffffu, m, off))));
        return int4_pair(bf16_lo(m), -bf16_hi(m));
    }
};

template <typename TIn, int TPR>
__global__ void __launch_bounds__(kThreads)
append_int4_kernel(const TIn* __restrict__ k_new, const TIn* __restrict__ v_new,
                   const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
                   uint8_t* __restrict__ v_cache, uint32_t* __restrict__ k_params,
                   uint32_t* __restrict__ v_params, int num_tokens, int splits, int head_dim,
                   int num_kv_heads, int block_size, long long num_slots, int32_t* error_word) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsPerPass = 32 / TPR;
    constexpr int U = sizeof(TIn) == 2 ? 4 : 2;          // passes in flight
    const int lane = threadIdx.x & 31;
    const int sub = lane / TPR, c = lane % TPR;
    const bool live = 8 * c < head_dim;
    const long long warp = static_cast<long long>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
    const long long t = warp / splits;
    const int part = static_cast<int>(warp - t * splits);
    if (t >= num_tokens) return;
    const long long slot = __ldg(slot_mapping + t);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (part == 0 && lane == 0) raise_error(error_word, PA_DEVERR_SLOT);
        return;
    }
    const long long blk = slot / block_size;
    const long long row0 = blk * num_kv_heads * block_size + (slot - blk * block_size);
    const long long from = t * num_kv_heads * head_dim + 8 * c;
    // The K heads, then the V heads.
    const int rows = 2 * num_kv_heads;
    for (int pass = part; pass * kRowsPerPass < rows; pass += U * splits) {
        Eight<TIn, TPR> in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = (pass + u * splits) * kRowsPerPass + sub;
            const bool v = r >= num_kv_heads;
            in[u].clear();
            if (r < rows && live)
                in[u].load((v ? v_new : k_new) + from + static_cast<long long>(v ? r - num_kv_heads : r) * head_dim);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int first = (pass + u * splits) * kRowsPerPass;
            if (first >= rows) break;                    // whole warps
            const int r = first + sub;
            const bool v = r >= num_kv_heads, on = r < rows && live;
            const uint32_t pair = in[u].pair(on);
            if (on) {
                float x[8];
                in[u].values(x);
                const long long row = row0 + static_cast<long long>(v ? r - num_kv_heads : r) * block_size;
                reinterpret_cast<uint32_t*>((v ? v_cache : k_cache) + row * (head_dim / 2))[c] = int4_codes(x, pair);
                if (c == 0) (v ? v_params : k_params)[row] = pair;
            }
        }
    }
}

// Eight dims' values. bf16: the FMA c s + lo of two dims at a time rounds the
// exact sum once (c, s and lo are bf16 values; 128 + c is the bf16 bits 0x4300 | c).
__device__ __forceinline__ void put_values(__nv_bfloat16* p, uint32_t w, uint32_t pair) {
    auto h2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    auto u = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); };
    const __nv_bfloat162 s = h2(__byte_perm(pair, 0u, 0x3232)), lo = h2(__byte_perm(pair, 0u, 0x1010));
    uint32_t r[4];                                       // dims (e, e + 4)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t bits = ((w >> (4 * e)) & 0x000f000fu) | 0x43004300u;
        r[e] = u(__hfma2(__hsub2(h2(bits), h2(0x43004300u)), s, lo));
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                                              __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
}
__device__ __forceinline__ void put_values(float* p, uint32_t w, uint32_t pair) {
    const float lo = int4_lo(pair), step = int4_step(pair);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(step, static_cast<float>((w >> (4 * e)) & 15u), lo);
    store8(p, x);
}

template <typename TOut, int TPR>
__global__ void __launch_bounds__(kThreads)
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
    constexpr int U = 4;                                 // passes in flight
    const int s = blockIdx.y;
    const int n = __ldg(context_lens + s);
    const long long start = __ldg(row_starts + s);
    if (n < 0 || n > context_cap || start < 0 || start > num_rows - n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(error_word, PA_DEVERR_CONTEXT);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int sub = lane / TPR, c = lane % TPR;
    const bool live = 8 * c < head_dim;
    const int32_t* table = block_tables + static_cast<size_t>(s) * max_blocks_per_seq;
    const int stride = gridDim.x * kWarpsPerCta;
    for (int row = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5); row < n; row += stride) {
        const int col = row / block_size;
        const int id = __ldg(table + col);
        if (id < 0 || id >= num_blocks) {
            if (lane == 0) raise_error(error_word, PA_DEVERR_BLOCK_ID);
            continue;
        }
        const size_t in0 = static_cast<size_t>(id) * num_kv_heads * block_size + (row - col * block_size);
        const size_t out0 = (static_cast<size_t>(start) + row) * num_kv_heads * head_dim + 8 * c;
        for (int pass = 0; pass * kRowsPerPass < num_kv_heads; pass += U) {
            uint32_t w[U][2], pair[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (pass + u) * kRowsPerPass + sub;
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
                if (h < num_kv_heads && live) {
                    const size_t to = out0 + static_cast<size_t>(h) * head_dim;
                    put_values(k_out + to, w[u][0], pair[u][0]);
                    put_values(v_out + to, w[u][1], pair[u][1]);
                }
            }
        }
    }
}

int lanes_per_row(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

}  // namespace

cudaError_t launch_append_int4(const void* k_new, const void* v_new, pa_dtype new_dtype,
                               const int64_t* slot_mapping, void* k_cache, void* v_cache,
                               void* k_params, void* v_params, int num_tokens, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, int32_t* error_word,
                               cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    const int tpr = lanes_per_row(head_dim);
    const long long passes = (2LL * num_kv_heads * tpr + 31) / 32;
    const long long want = (kFillWarps + num_tokens - 1) / num_tokens;
    const int splits = static_cast<int>(want < passes ? want : passes);
    const long long blocks =
        (static_cast<long long>(num_tokens) * splits + kWarpsPerCta - 1) / kWarpsPerCta;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto run = [&](auto kernel, auto tag) {
        using TIn = decltype(tag);
        kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
            static_cast<const TIn*>(k_new), static_cast<const TIn*>(v_new), slot_mapping,
            static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
            static_cast<uint32_t*>(k_params), static_cast<uint32_t*>(v_params), num_tokens, splits,
            head_dim, num_kv_heads, block_size, static_cast<long long>(num_blocks) * block_size,
            error_word);
        return cudaGetLastError();
    };
    auto pick = [&](auto tag) {
        using TIn = decltype(tag);
        return tpr == 8    ? run(append_int4_kernel<TIn, 8>, tag)
               : tpr == 16 ? run(append_int4_kernel<TIn, 16>, tag)
                           : run(append_int4_kernel<TIn, 32>, tag);
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
    const int tpr = lanes_per_row(head_dim);
    // Rows beyond a sequence's length cost nothing but a CTA's look at it, so the
    // sequences share a bounded number of CTAs, at most one warp per row.
    long long bx = (max_context_len + kWarpsPerCta - 1) / kWarpsPerCta;
    const long long share = (PA_GX + num_seqs - 1) / num_seqs;
    if (bx > share) bx = share;
    if (bx < 1) bx = 1;
    auto run = [&](auto kernel, auto tag) {
        using TOut = decltype(tag);
        for (int s0 = 0; s0 < num_seqs; s0 += 65535) {   // grid.y holds 65,535 sequences
            const int m = num_seqs - s0 < 65535 ? num_seqs - s0 : 65535;
            kernel<<<dim3(static_cast<unsigned>(bx), static_cast<unsigned>(m)), kThreads, 0, stream>>>(
                static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                static_cast<const uint32_t*>(k_params), static_cast<const uint32_t*>(v_params),
                block_tables + static_cast<size_t>(s0) * max_blocks_per_seq, context_lens + s0,
                row_starts + s0, static_cast<TOut*>(k_out), static_cast<TOut*>(v_out), num_rows,
                num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq,
                max_context_len, error_word);
            const cudaError_t err = cudaGetLastError();
            if (err != cudaSuccess) return err;
        }
        return cudaSuccess;
    };
    auto pick = [&](auto tag) {
        using TOut = decltype(tag);
        return tpr == 8    ? run(gather_int4_kernel<TOut, 8>, tag)
               : tpr == 16 ? run(gather_int4_kernel<TOut, 16>, tag)
                           : run(gather_int4_kernel<TOut, 32>, tag);
    };
    return out_dtype == PA_DTYPE_BF16 ? pick(__nv_bfloat16{}) : pick(float{});
}

}  // namespace pa

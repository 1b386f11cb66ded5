// pa_append_int4.cu -- the quantising append into a 4-bit cache and the gather
// of its rows as plain values (row format: pa_int4.cuh). Both are one pass
// over memory.
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

// TPR lanes per (token, KV head, K or V) row, 8 dims each: butterfly minimum
// and maximum, then 8 codes (4 bytes) per lane. Consecutive rows go to
// consecutive lane groups, so a warp reads whole 16-byte chunks in order.
template <typename TIn, int TPR>
__global__ void __launch_bounds__(kThreads)
append_int4_kernel(const TIn* __restrict__ k_new, const TIn* __restrict__ v_new,
                   const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
                   uint8_t* __restrict__ v_cache, uint32_t* __restrict__ k_params,
                   uint32_t* __restrict__ v_params, long long rows, int head_dim,
                   int num_kv_heads, int block_size, long long num_slots, int32_t* error_word) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsPerWarp = 32 / TPR;
    const int lane = threadIdx.x & 31;
    const int c = lane % TPR;
    const bool live = 8 * c < head_dim;
    const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    const long long warp = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    for (long long r0 = warp * kRowsPerWarp; r0 < 2 * rows; r0 += warps * kRowsPerWarp) {
        const long long w = r0 + lane / TPR;
        const bool is_v = w >= rows;
        const long long rowi = is_v ? w - rows : w;          // (token, kv head)
        const long long t = rowi / num_kv_heads;
        const int h = static_cast<int>(rowi - t * num_kv_heads);
        long long slot = -1;
        if (w < 2 * rows) {
            slot = __ldg(slot_mapping + t);
            if (slot >= num_slots) {
                if (c == 0 && h == 0 && !is_v) raise_error(error_word, PA_DEVERR_SLOT);
                slot = -1;
            }
        }
        const bool on = slot >= 0 && live;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        if (on) load8((is_v ? v_new : k_new) + rowi * head_dim + 8 * c, x);
        const uint32_t pair = int4_row_pair<TPR>(x, on);
        if (on) {
            const long long blk = slot / block_size;
            const long long r = (blk * num_kv_heads + h) * block_size + (slot - blk * block_size);
            reinterpret_cast<uint32_t*>((is_v ? v_cache : k_cache) + r * (head_dim / 2))[c] =
                int4_codes(x, pair);
            if (c == 0) (is_v ? v_params : k_params)[r] = pair;
        }
    }
}

// One thread per 8 dims of one (row, KV head): 4 bytes of codes and the row's
// pair in, 8 values out, K and V both.
template <typename TOut>
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
    const int s = blockIdx.y;
    const int n = __ldg(context_lens + s);
    const long long start = __ldg(row_starts + s);
    if (n < 0 || n > context_cap || start < 0 || start > num_rows - n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(error_word, PA_DEVERR_CONTEXT);
        return;
    }
    const int cpr = head_dim / 8;                      // chunks per row
    const long long per_row = static_cast<long long>(num_kv_heads) * cpr;
    const long long stride = static_cast<long long>(gridDim.x) * kThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n * per_row;
         i += stride) {
        const int row = static_cast<int>(i / per_row);
        const int rem = static_cast<int>(i - row * per_row);
        const int h = rem / cpr, c = rem - h * cpr;
        const int col = row / block_size;
        const int id = __ldg(block_tables + static_cast<size_t>(s) * max_blocks_per_seq + col);
        if (id < 0 || id >= num_blocks) {
            if (rem == 0) raise_error(error_word, PA_DEVERR_BLOCK_ID);
            continue;
        }
        const size_t r = (static_cast<size_t>(id) * num_kv_heads + h) * block_size + (row - col * block_size);
        const size_t dst = ((static_cast<size_t>(start) + row) * num_kv_heads + h) * head_dim + 8 * c;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint32_t pair = __ldg((which ? v_params : k_params) + r);
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>((which ? v_cache : k_cache) +
                                                                       r * (head_dim / 2)) + c);
            const float lo = int4_lo(pair), step = int4_step(pair);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(step, static_cast<float>((w >> (4 * e)) & 15u), lo);
            store8((which ? v_out : k_out) + dst, x);
        }
    }
}

}  // namespace

cudaError_t launch_append_int4(const void* k_new, const void* v_new, pa_dtype new_dtype,
                               const int64_t* slot_mapping, void* k_cache, void* v_cache,
                               void* k_params, void* v_params, int num_tokens, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, int32_t* error_word,
                               cudaStream_t stream) {
    const long long rows = static_cast<long long>(num_tokens) * num_kv_heads;
    if (rows == 0) return cudaSuccess;
    const int tpr = head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32;
    long long blocks = (2 * rows * tpr + kThreads - 1) / kThreads;
    if (blocks > 1 << 16) blocks = 1 << 16;
    auto run = [&](auto kernel, auto tag) {
        using TIn = decltype(tag);
        kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
            static_cast<const TIn*>(k_new), static_cast<const TIn*>(v_new), slot_mapping,
            static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
            static_cast<uint32_t*>(k_params), static_cast<uint32_t*>(v_params), rows, head_dim,
            num_kv_heads, block_size, static_cast<long long>(num_blocks) * block_size, error_word);
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
    const long long chunks = static_cast<long long>(max_context_len) * num_kv_heads * (head_dim / 8);
    long long bx = (chunks + kThreads - 1) / kThreads;
    if (bx < 1) bx = 1;
    if (bx > 1024) bx = 1024;
    auto run = [&](auto tag) {
        using TOut = decltype(tag);
        for (int s0 = 0; s0 < num_seqs; s0 += 65535) {   // grid.y holds 65,535 sequences
            const int m = num_seqs - s0 < 65535 ? num_seqs - s0 : 65535;
            gather_int4_kernel<TOut><<<dim3(static_cast<unsigned>(bx), static_cast<unsigned>(m)),
                                       kThreads, 0, stream>>>(
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
    return out_dtype == PA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // namespace pa

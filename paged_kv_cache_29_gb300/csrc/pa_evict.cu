// pa_evict.cu -- eviction by accumulated attention weight (pa_evict).
//
// Of the m rows between the first num_sinks and the last num_recent of a sequence,
// the `more` with the largest weights stay under each KV head. Weights become 32-bit
// keys in their order; a radix selection, eight bits a pass from the top, finds the
// more-th largest key and how many of the rows that hold just that key stay: the
// first ones. A walk over the rows in order then numbers the rows that stay, and
// lists each that changes its place as a pair of pool rows (from, to).
//
// The list is in the rows' order, to <= from within a sequence: a stretch of the list
// that was read whole may be written whatever of it stands in its way, and no
// later stretch reads a row that an earlier one wrote. So rows can move in place, a
// stretch at a time, as long as all of a stretch's reads come before its writes. Bytes of a
// row at different offsets never meet: each warp moves one slice of the row under one
// KV head through the whole list on its own, with no barrier beyond its own.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kSelectThreads = 256;

// 32 bits in the order of the weights: NaN as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, KV head): the list of its rows' moves.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t warp_sums[kSelectThreads / 32];
    __shared__ uint32_t found[2];             // digit, rows of larger digits
    __shared__ int bad;
    const int s = blockIdx.x / p.num_kv_heads;
    const int h = blockIdx.x - s * p.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = p.block_size;
    const int n = __ldg(p.context_lens + s);
    int keep = __ldg(p.keep_lens + s);
    const bool odd = n < 0 || n > p.context_cap || keep < 0;
    keep = min(keep, n);
    const int first = odd ? 0 : min(n, p.num_sinks);             // rows [first, last) may leave
    const int last = odd ? 0 : max(first, n - min(n, p.num_recent));
    const int more = keep - first - (n - last);                  // rows of them that stay
    const int32_t* from = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    const int32_t* to = p.out_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    if (tid == 0) bad = 0;
    __syncthreads();
    if (!odd && more >= 0) {
        bool outside = false;
        for (int b = tid; b < (n + bs - 1) / bs; b += kSelectThreads) {
            const int id = __ldg(from + b);
            outside |= id < 0 || id >= p.num_blocks;
        }
        for (int b = tid; b < (keep + bs - 1) / bs; b += kSelectThreads) {
            const int id = __ldg(to + b);
            outside |= id < 0 || id >= p.num_blocks;
        }
        if (outside) bad = 1;
    }
    __syncthreads();
    if (odd || more < 0 || bad) {
        if (tid == 0) {
            if (h == 0) {
                raise_error(p.error_word, odd || more < 0 ? PA_DEVERR_CONTEXT : PA_DEVERR_BLOCK_ID);
                p.new_lens[s] = n;
            }
            p.counts[blockIdx.x] = 0;
        }
        return;
    }
    if (tid == 0 && h == 0) p.new_lens[s] = keep;
    auto from_row = [&](int i) {
        return (static_cast<uint32_t>(__ldg(from + i / bs)) * p.num_kv_heads + h) * bs + i % bs;
    };
    auto to_row = [&](int i) {
        return (static_cast<uint32_t>(__ldg(to + i / bs)) * p.num_kv_heads + h) * bs + i % bs;
    };

    // The more-th largest key, and how many rows that hold it stay.
    uint32_t border = 0, level = 0;
    const int m = last - first;
    if (more == 0) {
        border = 0xffffffffu;                // no key is that large
    } else if (more < m) {
        uint32_t want = more;
        for (int shift = 24; shift >= 0; shift -= 8) {
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            hist[tid] = 0;
            __syncthreads();
            for (int i = first + tid; i < last; i += kSelectThreads) {
                const uint32_t key = weight_key(p.row_weights[from_row(i)]);
                if ((key & mask) == border) atomicAdd(&hist[(key >> shift) & 255u], 1u);
            }
            __syncthreads();
            // Rows of larger digits: an inclusive scan from the top; thread t has digit 255 - t.
            const uint32_t own = hist[255 - tid];
            uint32_t incl = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += u;
            }
            if (lane == 31) warp_sums[warp] = incl;
            __syncthreads();
            for (int w = 0; w < warp; ++w) incl += warp_sums[w];
            if (incl >= want && incl - own < want) {
                found[0] = 255 - tid;
                found[1] = incl - own;
            }
            __syncthreads();
            border |= found[0] << shift;
            want -= found[1];
        }
        level = want;
    }                                        // else all stay: every key is above 0

    // Number the rows that stay, in order, and list those that change their place.
    uint2* list = p.moves + static_cast<size_t>(blockIdx.x) * p.context_cap;
    uint32_t above0 = 0, equal0 = 0, listed0 = 0;   // rows before this stretch: larger, equal, listed
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + tid;
        bool above = false, equal = false;
        if (i < n) {
            if (i < first || i >= last) {
                above = true;
            } else {
                const uint32_t key = weight_key(p.row_weights[from_row(i)]);
                above = key > border;
                equal = key == border;
            }
        }
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t va = __ballot_sync(0xffffffffu, above), ve = __ballot_sync(0xffffffffu, equal);
        __syncthreads();
        if (lane == 0) warp_sums[warp] = __popc(va) | (__popc(ve) << 16);
        __syncthreads();
        uint32_t a = above0 + __popc(va & below), e = equal0 + __popc(ve & below);
        uint32_t ta = 0, te = 0;
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            const uint32_t v = warp_sums[w];
            if (w < warp) {
                a += v & 0xffffu;
                e += v >> 16;
            }
            ta += v & 0xffffu;
            te += v >> 16;
        }
        const bool stays = above || (equal && e < level);
        uint32_t src = 0, dst = 0;
        if (stays) {
            src = from_row(i);
            dst = to_row(a + min(e, level));
        }
        const bool moves = stays && src != dst;
        const uint32_t vm = __ballot_sync(0xffffffffu, moves);
        __syncthreads();
        if (lane == 0) warp_sums[warp] = __popc(vm);
        __syncthreads();
        uint32_t at = listed0 + __popc(vm & below), tm = 0;
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            if (w < warp) at += warp_sums[w];
            tm += warp_sums[w];
        }
        if (moves) list[at] = make_uint2(src, dst);
        above0 += ta;
        equal0 += te;
        listed0 += tm;
    }
    if (tid == 0) p.counts[blockIdx.x] = listed0;
}

// Moves. A warp per (sequence, KV head, slice): slices 0 .. 2 kSlices - 1 are parts of
// the K and V rows, the ones after them the 4-byte values beside the rows.
constexpr int kMoveThreads = 128;
constexpr int kBatch = 8;                     // loads of a lane before their stores

template <typename T>
__device__ __forceinline__ void move_values(T* base, const uint2* list, int count, int lanes, int lane, size_t pitch) {
    // `lanes` lanes share a row, 32 / lanes rows at a time; pitch: elements of T per row.
    const int sub = lane % lanes, per = 32 / lanes;
    for (int j0 = 0; j0 < count; j0 += per * kBatch) {
        T v[kBatch];
        uint32_t dst[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = j0 + u * per + lane / lanes;
            if (j < count) {
                const uint2 mv = list[j];
                dst[u] = mv.y;
                v[u] = base[mv.x * pitch + sub];
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (j0 + u * per + lane / lanes < count) base[dst[u] * pitch + sub] = v[u];
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int slices, int units) {
    const long long unit = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long sh = unit / units;
    const int part = static_cast<int>(unit - sh * units);
    if (sh >= static_cast<long long>(p.num_seqs) * p.num_kv_heads) return;
    if (part == 0 && sh % p.num_kv_heads == 0 && lane == 0)
        p.lens_out[sh / p.num_kv_heads] = p.new_lens[sh / p.num_kv_heads];
    const int count = p.counts[sh];
    const uint2* list = p.moves + sh * p.context_cap;
    if (part < 2 * slices) {
        const int which = part / slices, slice = part - which * slices;
        const int lanes = p.row_bytes / 16 / slices;
        uint4* base = static_cast<uint4*>(which ? p.v_cache : p.k_cache) + slice * lanes;
        if (lanes <= 32) move_values(base, list, count, lanes, lane, p.row_bytes / 16);
    } else {
        const int which = part - 2 * slices;
        uint32_t* base = which == 0 ? reinterpret_cast<uint32_t*>(p.row_weights) : which == 1 ? p.k_params : p.v_params;
        move_values(base, list, count, 1, lane, 1);
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    const long long heads = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
    if (heads == 0) return cudaSuccess;
    evict_select_kernel<<<static_cast<unsigned>(heads), kSelectThreads, 0, stream>>>(p);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int slices = p.row_bytes / 16;     // 16 bytes each
    const int units = 2 * slices + (p.k_params ? 3 : 1);
    const long long ctas = (heads * units + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    evict_move_kernel<<<static_cast<unsigned>(ctas), kMoveThreads, 0, stream>>>(p, slices, units);
    return cudaGetLastError();
}

}  // namespace pa

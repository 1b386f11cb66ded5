// pa_evict.cu -- eviction by accumulated attention weight (pa_evict).
//
// Of the m rows between the first num_sinks and the last num_recent of a sequence,
// the `more` with the largest weights stay under each KV head. Weights become 32-bit
// keys in their order; passes that count the keys in 256 equal parts of a range, from that
// of all keys on, find the part with the more-th largest, until few enough are left to be
// ranked against one another (mostly after one pass): that key, and how many of the
// rows that hold just that key stay, the first ones. A walk over the rows in order then numbers the rows that stay: the
// j-th of them moves to row j, and is listed as a pair of pool rows (from, to).
//
// A cluster of CTAs shares the rows under one KV head of a sequence. A CTA holds the
// keys of a run of rows in shared memory, so that the weights are read once; counts by
// part, and of rows that stay, are added up through the cluster's shared memory.
//
// The list is in the rows' order, to <= from within a sequence: a stretch of the list
// that was read whole may be written whatever of it stands in its way, and no
// later stretch reads a row that an earlier one wrote. So rows can move in place, a
// stretch at a time, as long as all of a stretch's reads come before its writes; the reads
// of later stretches may come before them too. Bytes of a row at different offsets
// never meet: CTAs move slices of the rows under one KV head through the whole list, with
// no barrier between them.
//
// 128 sequences of 1,640 rows to half, in place, 8 KV heads of 128, bf16: selection 24 us, bound by
// latencies (six trips to memory and some 20 barriers a CTA, in 1.7 rounds of CTAs); moves 141 us for 854 MB,
// 6.1 TB/s, bound by memory.
#include <atomic>
#include <climits>

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {

namespace {

constexpr int kMaxCluster = 8;
constexpr int kFew = 256;                     // candidates that are ranked against one another
constexpr int kCopies = 2;                    // of the counts: 16 lanes at most meet in one
constexpr int kApart = -1;                    // in place of a first move: no block is moved from and to
constexpr uint32_t kStays = 0xffffffffu;      // key of a row that stays in any case; no weight has it
// Keys that a CTA holds at most. Where the bound on the lengths allows more than a cluster
// holds, it holds those of sequences with up to kShortKeys rows a CTA; longer ones read their
// weights again in every pass.
constexpr int kMaxKeys = 48 * 1024;
constexpr int kShortKeys = 8 * 1024;
constexpr int kMaxOrdered = 256;              // sequences that are taken in the order of their lengths

// 32 bits in the order of the weights: NaN as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One cluster per (sequence, KV head): the list of its rows' moves, and from where on rows
// change their place.
// HELD: every CTA's keys fit its shared memory, by the bound on the lengths.
template <int kSelectThreads, bool HELD>
__global__ void __launch_bounds__(kSelectThreads, kSelectThreads == 256 ? 4 : 2) evict_select_kernel(const EvictParams p) {
    constexpr int kSelectWarps = kSelectThreads / 32;
    static_assert(kSelectThreads >= 256, "a thread per part, a warp per CTA of the cluster");
    extern __shared__ uint32_t keys[];        // of the CTA's rows (HELD)
    __shared__ uint32_t hist[256 * kCopies];
    __shared__ uint32_t parts[2][256];       // this CTA's counts by part, of two passes
    __shared__ uint32_t few[2][kFew];         // candidates: this CTA's, the cluster's
    __shared__ uint32_t few_count[2];
    __shared__ uint32_t range[2], all_range[2];   // least and largest key of a weight
    __shared__ uint32_t scan_sums[8];
    __shared__ uint32_t found[3];             // part, rows of larger parts, rows of this part
    __shared__ uint2 warp_counts[kSelectWarps];
    __shared__ uint2 cta_counts;              // rows of the CTA above the border, at it
    __shared__ uint2 cluster_counts;          // of the CTAs before it
    __shared__ int flags, all_flags, first_move;
    constexpr int kBad = 1, kSame = 2;        // a block outside the pool; one that rows stay in
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    auto meet = [&] {                         // (a barrier of one CTA is the cheaper one)
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    grid_dependency_wait();
    grid_launch_dependents();
    const int sh = blockIdx.x / ranks;        // (what the list and the lengths are kept by)
    const int unit = sh / p.num_kv_heads;
    const int h = sh - unit * p.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = p.block_size;
    int s = unit, n, keep;
    if (p.order != nullptr) {
        // The unit-th sequence when the longest come first, by eight classes of lengths, each half
        // the one before it; a warp counts 32 sequences' classes, all warps add up the counts.
        __shared__ uint2 counts[32];          // [class][warp]
        __shared__ int own[3];
        int cls = 8;
        n = keep = 0;
        if (tid < p.num_seqs) {
            n = p.context_lens[tid];          // (ordinary loads, as the plan of the decode kernels)
            keep = p.keep_lens[tid];
            cls = n <= 0 ? 7 : min(7, max(0, __clz(n) - __clz(p.context_cap)));
        }
        uint32_t peers = 0, count = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t in = __ballot_sync(0xffffffffu, cls == k);
            if (cls == k) peers = in;
            if (lane == k) count = __popc(in);
        }
        if (warp < 8 && lane < 8) reinterpret_cast<uint32_t*>(counts)[lane * 8 + warp] = count;
        __syncthreads();
        if (warp < 8) {
            const uint2 c = counts[lane];
            uint32_t before = c.x + c.y;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += u;
            }
            const int at = (cls * 8 + warp) & 63;
            const uint32_t upto = __shfl_sync(0xffffffffu, before - c.x - c.y, at / 2);
            const uint32_t even = __shfl_sync(0xffffffffu, c.x, at / 2);
            const uint32_t place = upto + (at & 1 ? even : 0u) + __popc(peers & ((1u << lane) - 1u));
            if (cls < 8 && place == static_cast<uint32_t>(unit)) {
                own[0] = tid;
                own[1] = n;
                own[2] = keep;
            }
        }
        __syncthreads();
        s = own[0];
        n = own[1];
        keep = own[2];
        if (tid == 0 && rank == 0 && h == 0) p.order[unit] = s;
    } else {
        n = p.context_lens[s];
        keep = p.keep_lens[s];
    }
    const bool odd = n < 0 || n > p.context_cap || keep < 0;
    keep = min(keep, n);
    const int first = odd ? 0 : min(n, p.num_sinks);             // rows [first, last) may leave
    const int last = odd ? 0 : max(first, n - min(n, p.num_recent));
    const int more = keep - first - (n - last);                  // rows of them that stay
    if (odd || more < 0) {                    // the same in every CTA of the cluster
        if (tid == 0 && rank == 0) {
            if (h == 0) {
                raise_error(p.error_word, PA_DEVERR_CONTEXT);
                p.new_lens[unit] = n;
            }
            p.starts[sh] = INT_MAX;
        }
        return;
    }
    const int32_t* from = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    const int32_t* to = p.out_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    // This CTA's rows, and this warp's: runs of whole 32s.
    const int share = ((n + ranks - 1) / ranks + 31) / 32 * 32;
    const int row0 = min(n, rank * share), row1 = min(n, row0 + share);
    const int warp_share = ((row1 - row0 + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int w0 = min(row1, row0 + warp * warp_share), w1 = min(row1, w0 + warp_share);
    const bool held = HELD || share <= kShortKeys;
    if (tid == 0) {
        flags = 0;
        first_move = INT_MAX;
        few_count[0] = few_count[1] = 0;
        range[0] = kStays;
        range[1] = 0;
    }
    for (int i = tid; i < 256 * kCopies; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    auto block_index = [&](int i) { return p.by_block.quotient(i); };
    auto pool_row = [&](int id, int i) {
        return (static_cast<uint32_t>(id) * p.num_kv_heads + h) * bs + p.by_block.rest(i, block_index(i));
    };
    auto key_of = [&](int i, int id) {
        const uint32_t key = weight_key(p.row_weights[pool_row(id, i)]);
        return i < first || i >= last ? kStays : key;
    };
    bool outside = false, same = false;
    uint32_t least = kStays, most = 0;        // of the weights' keys
    for (int b = rank * kSelectThreads + tid; b < (keep + bs - 1) / bs; b += ranks * kSelectThreads) {
        const int id = __ldg(to + b);
        outside |= id < 0 || id >= p.num_blocks;
        same |= id == __ldg(from + b);
    }
    constexpr int kRows = kSelectThreads == 256 ? 4 : 8;   // rows of a thread whose loads are on the way together
    for (int i0 = row0 + tid; i0 < row1; i0 += kRows * kSelectThreads) {
        int id[kRows];
        uint32_t k[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) id[u] = __ldg(from + block_index(min(i0 + u * kSelectThreads, row1 - 1)));
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const bool in = id[u] >= 0 && id[u] < p.num_blocks;
            outside |= !in;
            if (!in) id[u] = 0;               // (its key is not used)
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) k[u] = key_of(min(i0 + u * kSelectThreads, row1 - 1), id[u]);
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (i0 + u * kSelectThreads < row1) {
                if (held) keys[i0 + u * kSelectThreads - row0] = k[u];
                if (k[u] != kStays) {
                    least = min(least, k[u]);
                    most = max(most, k[u]);
                }
            }
    }
    if (outside) atomicOr(&flags, kBad);
    if (same) atomicOr(&flags, kSame);
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        atomicMin(&range[0], least);
        atomicMax(&range[1], most);
    }
    meet();
    if (warp == 0) {
        const int theirs = lane >= ranks ? 0 : ranks > 1 ? *cluster.map_shared_rank(&flags, lane) : flags;
        const uint32_t all = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(theirs));
        least = lane >= ranks ? kStays : ranks > 1 ? cluster.map_shared_rank(&range[0], lane)[0] : range[0];
        most = lane >= ranks ? 0u : ranks > 1 ? cluster.map_shared_rank(&range[0], lane)[1] : range[1];
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            all_flags = static_cast<int>(all);
            all_range[0] = least;
            all_range[1] = most;
        }
    }
    __syncthreads();
    if (all_flags & kBad) {
        if (tid == 0 && rank == 0) {
            if (h == 0) {
                raise_error(p.error_word, PA_DEVERR_BLOCK_ID);
                p.new_lens[unit] = n;
            }
            p.starts[sh] = INT_MAX;
        }
        meet();                               // every CTA has read the others' flags
        return;
    }
    auto key_at = [&](int i) { return held ? keys[i - row0] : key_of(i, __ldg(from + block_index(i))); };

    // The more-th largest key of [first, last), and how many rows that hold it stay.
    uint32_t border = 0, level = 0;
    if (more == 0) {
        border = kStays - 1;                  // no weight's key is that large
    } else if (more < last - first) {
        uint32_t want = more;
        border = all_range[0];                // least key of the range, 256 parts of 2^shift
        int shift = max(0, 24 - __clz(all_range[1] - border));
        uint32_t in_range = 256;              // parts that the range has
        auto part_of = [&](uint32_t key) { return (key - border) >> shift; };
        for (int pass = 0;; ++pass) {
            for (int i = row0 + tid; i < row1; i += kSelectThreads) {
                const uint32_t key = key_at(i);
                if (key != kStays && part_of(key) < in_range)   // (below the range: it wraps beyond)
                    atomicAdd(&hist[part_of(key) * kCopies + (lane & (kCopies - 1))], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t sum = 0;
#pragma unroll
                for (int c = 0; c < kCopies; ++c) {
                    sum += hist[tid * kCopies + c];
                    hist[tid * kCopies + c] = 0;
                }
                parts[pass & 1][tid] = sum;
            }
            // (The other CTAs read parts[pass & 1]; it is written again two passes on,
            // behind the next pass's barrier.)
            meet();
            uint32_t own = 0, incl = 0;
            if (tid < 256) {
                // Rows of larger parts: an inclusive scan from the top; thread t has part 255 - t.
                for (int r = 0; r < ranks; ++r)
                    own += ranks > 1 ? cluster.map_shared_rank(&parts[pass & 1][0], r)[255 - tid] : parts[pass & 1][255 - tid];
                incl = own;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += u;
                }
                if (lane == 31) scan_sums[warp] = incl;
            }
            __syncthreads();
            if (tid < 256) {
                for (int w = 0; w < warp; ++w) incl += scan_sums[w];
                if (incl >= want && incl - own < want) {
                    found[0] = 255 - tid;
                    found[1] = incl - own;
                    found[2] = own;
                }
            }
            __syncthreads();
            border += found[0] << shift;
            want -= found[1];
            if (shift == 0) break;
            if (found[2] <= kFew) {
                // Few rows are in that part: the border is the key of the one that fewer than
                // `want` are above, and with its equals at least `want`.
                for (int i = row0 + tid; i < row1; i += kSelectThreads) {
                    const uint32_t key = key_at(i);
                    if (key != kStays && part_of(key) == 0u) few[0][atomicAdd(&few_count[0], 1u)] = key;
                }
                meet();
                if (warp < ranks) {           // a warp takes another CTA's
                    const uint32_t c = *cluster.map_shared_rank(&few_count[0], warp);
                    const uint32_t* theirs = cluster.map_shared_rank(&few[0][0], warp);
                    for (uint32_t i = lane; i < c; i += 32) few[1][atomicAdd(&few_count[1], 1u)] = theirs[i];
                }
                __syncthreads();
                const uint32_t count = few_count[1];
                for (uint32_t i = tid; i < count; i += kSelectThreads) {
                    const uint32_t key = few[1][i];
                    uint32_t larger = 0, same = 0;
                    for (uint32_t k = 0; k < count; ++k) {
                        larger += few[1][k] > key;
                        same += few[1][k] == key;
                    }
                    if (larger < want && larger + same >= want) {   // (each of its equals writes the same)
                        found[0] = key;
                        found[1] = larger;
                    }
                }
                __syncthreads();
                border = found[0];
                want -= found[1];
                break;                        // (the cluster meets again before a CTA can end)
            }
            in_range = shift >= 8 ? 256u : 1u << shift;
            shift = max(0, shift - 8);
        }
        level = want;
    }                                         // else all stay: every key is above 0

    // Rows above the border and at it, by warp, CTA and cluster.
    uint32_t above = 0, equal = 0;
    for (int i = w0 + lane; i - lane < w1; i += 32) {
        const uint32_t key = i < w1 ? key_at(i) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, i < w1 && key > border));
        equal += __popc(__ballot_sync(0xffffffffu, i < w1 && key == border));
    }
    if (lane == 0) warp_counts[warp] = make_uint2(above, equal);
    __syncthreads();
    above = equal = 0;                        // now: before this warp's rows
    uint2 all = make_uint2(0, 0);
    for (int w = 0; w < kSelectWarps; ++w) {
        const uint2 c = warp_counts[w];
        if (w < warp) {
            above += c.x;
            equal += c.y;
        }
        all.x += c.x;
        all.y += c.y;
    }
    if (ranks > 1) {
        if (tid == 0) cta_counts = all;
        cluster.sync();
        if (warp == 0) {
            const uint2 c = lane < rank ? *cluster.map_shared_rank(&cta_counts, lane) : make_uint2(0, 0);
            const uint32_t x = __reduce_add_sync(0xffffffffu, c.x), y = __reduce_add_sync(0xffffffffu, c.y);
            if (lane == 0) cluster_counts = make_uint2(x, y);
        }
        __syncthreads();
        above += cluster_counts.x;
        equal += cluster_counts.y;
    }
    uint2* list = p.moves + static_cast<size_t>(sh) * p.context_cap;
    int moved = INT_MAX;
    constexpr int kAhead = 4;                 // rows of a lane whose table entries are on the way together
    for (int i0 = w0 + lane; i0 - lane < w1; i0 += 32 * kAhead) {
        int to_row[kAhead], from_id[kAhead], to_id[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + 32 * u;
            const uint32_t key = i < w1 ? key_at(i) : 0u;
            const uint32_t va = __ballot_sync(0xffffffffu, i < w1 && key > border);
            const uint32_t ve = __ballot_sync(0xffffffffu, i < w1 && key == border);
            const uint32_t before = (1u << lane) - 1u;
            const uint32_t e = equal + __popc(ve & before);
            const bool stays = i < w1 && (key > border || (key == border && e < level));
            to_row[u] = stays ? static_cast<int>(above + __popc(va & before) + min(e, level)) : -1;
            if (stays) {
                from_id[u] = __ldg(from + block_index(i));
                to_id[u] = __ldg(to + block_index(to_row[u]));
            }
            above += __popc(va);
            equal += __popc(ve);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (to_row[u] < 0) continue;
            const uint32_t src = pool_row(from_id[u], i0 + 32 * u), dst = pool_row(to_id[u], to_row[u]);
            list[to_row[u]] = make_uint2(src, dst);
            if (src != dst) moved = min(moved, to_row[u]);
        }
    }
    moved = __reduce_min_sync(0xffffffffu, moved);
    if (lane == 0 && moved != INT_MAX) atomicMin(&first_move, moved);
    meet();
    if (rank == 0 && tid == 0) {
        int start = INT_MAX;
        for (int r = 0; r < ranks; ++r) start = min(start, *cluster.map_shared_rank(&first_move, r));
        p.starts[sh] = all_flags & kSame ? start : kApart;
        if (h == 0) p.new_lens[unit] = keep;
    }
    meet();                           // no CTA ends before rank 0 has read it
}

// Moves: `ctas` CTAs of WARPS warps per (sequence, KV head). The 16-byte pieces of a K and a V
// row side by side, and the 4-byte values beside them, are a row. Where no block is moved from
// and to, each CTA takes a run of whole rows; else each takes slices (of `lanes` pieces) of
// every row, and the last one the values.

// List entries [start, count): a lane moves the element at `at` of its rows (none if null),
// `lanes` lanes (a power of two) share a row, pitch: elements from row to row.
// kBatch: rows of a lane per stretch.
template <typename T, int WARPS, int kBatch>
__device__ __forceinline__ void move_rows(T* at, const uint2* list, int start, int count, int lanes, size_t pitch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = 32 / lanes;               // rows of a warp at a time
    const int own = warp * per + lane / lanes;
    const int step = WARPS * per;
    uint2 mv[kBatch], mv_next[kBatch];
    T v[kBatch], v_next[kBatch];
    auto look = [&](uint2 (&m)[kBatch], int j0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = j0 + u * step + own;
            if (j < count) m[u] = list[j];
        }
    };
    auto read = [&](T (&x)[kBatch], const uint2 (&m)[kBatch], int j0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (at != nullptr && j0 + u * step + own < count) x[u] = at[m[u].x * pitch];
    };
    look(mv, start);
    read(v, mv, start);
    look(mv_next, start + kBatch * step);
    for (int j0 = start; j0 < count; j0 += kBatch * step) {
        // The next stretch is read before this one is written; every thread's reads of this
        // one are before the barrier, the writes behind it.
        read(v_next, mv_next, j0 + kBatch * step);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (at != nullptr && j0 + u * step + own < count) at[mv[u].y * pitch] = v[u];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            mv[u] = mv_next[u];
            v[u] = v_next[u];
        }
        look(mv_next, j0 + 2 * kBatch * step);
    }
}

template <int WARPS, int kBatch>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 3 : 4) evict_move_kernel(const EvictParams p, int lanes, int ctas) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int sh = blockIdx.x / ctas;
    const int part = blockIdx.x - sh * ctas;
    const int unit = sh / p.num_kv_heads;
    int count = p.new_lens[unit];
    int start = p.starts[sh];
    // Nothing reads the lengths any more: lens_out may be the array they are in.
    if (part == 0 && sh == unit * p.num_kv_heads && threadIdx.x == 0)
        p.lens_out[p.order != nullptr ? p.order[unit] : unit] = count;
    const int pieces = 2 * (p.row_bytes / 16);
    int slice = part, step = ctas - 1;
    bool values = part == ctas - 1;
    if (start == kApart) {
        lanes = min(32, pieces & -pieces);
        const int run = max((count + ctas - 1) / ctas, WARPS * kBatch * 32 / lanes);   // a stretch at least
        start = min(count, part * run);
        count = min(count, start + run);
        slice = 0;
        step = 1;
        values = true;
    }
    if (start >= count) return;
    const uint2* list = p.moves + static_cast<size_t>(sh) * p.context_cap;
    const int lane = threadIdx.x & 31;
    if (slice < step)
        for (; slice < pieces / lanes; slice += step) {
            const int piece = slice * lanes + lane % lanes;
            uint4* at = piece < pieces / 2 ? static_cast<uint4*>(p.k_cache) + piece
                                           : static_cast<uint4*>(p.v_cache) + (piece - pieces / 2);
            move_rows<uint4, WARPS, kBatch>(at, list, start, count, lanes, p.row_bytes / 16);
        }
    if (values) {
        if (p.k_params == nullptr) {
            move_rows<uint32_t, WARPS, kBatch>(reinterpret_cast<uint32_t*>(p.row_weights), list, start, count, 1, 1);
        } else {                              // three values in a group of four lanes
            uint32_t* at = lane % 4 == 0   ? reinterpret_cast<uint32_t*>(p.row_weights)
                           : lane % 4 == 1 ? p.k_params
                           : lane % 4 == 2 ? p.v_params
                                           : nullptr;
            move_rows<uint32_t, WARPS, kBatch>(at, list, start, count, 4, 1);
        }
    }
}

}  // namespace

cudaError_t launch_evict(EvictParams p, cudaStream_t stream) {
    const int heads = p.num_seqs * p.num_kv_heads;
    if (heads == 0) return cudaSuccess;
    const int sms = device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    int ranks = 1;
    while (ranks < kMaxCluster && static_cast<long long>(heads) * ranks < 2 * sms && p.context_cap / ranks > 2048) ranks *= 2;
    const int share = ((p.context_cap + ranks - 1) / ranks + 31) / 32 * 32;
    // Many CTAs hold few keys each, so that several fit an SM: 1,024 of them with a bound of
    // 32,768 rows and lengths of 1,640 take 189 us so, 202 with room for the bound.
    // Longest sequences first, where CTAs wait for room and lengths may differ much (128 sequences of
    // 1,640 rows take 171 us so, 177 as they come, 256 of them 340 and 365; but 256 of 300
    // rows and a bound of 600 124 and 121; with a copy of 5 us that restores the weights).
    if (p.num_seqs > kMaxOrdered || static_cast<long long>(heads) * ranks <= 4LL * sms || share <= 2048) p.order = nullptr;
    const int most_keys = static_cast<long long>(heads) * ranks <= 4LL * sms ? kMaxKeys : kShortKeys;
    const bool all_held = share <= most_keys;
    const int max_keys = all_held ? share : kShortKeys;
    // More threads where a CTA has many rows; else smaller CTAs, more of them to an SM.
    auto* select = !all_held      ? evict_select_kernel<512, false>
                   : share > 8192 ? evict_select_kernel<512, true>
                                  : evict_select_kernel<256, true>;
    cudaError_t err = cudaSuccess;
    if (max_keys > 8192) {                    // beyond the shared memory that needs no asking: once per device
        static std::atomic<bool> asked[kMaxDevices];   // (of evict_select_kernel<512, true>)
        int dev = 0;
        err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        if (dev >= kMaxDevices || !asked[dev].load(std::memory_order_relaxed)) {
            err = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMaxKeys);
            if (err != cudaSuccess) return err;
            if (dev < kMaxDevices) asked[dev].store(true, std::memory_order_relaxed);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(heads) * ranks);
    cfg.blockDim = dim3(share > 8192 ? 512 : 256);
    cfg.dynamicSmemBytes = 4 * static_cast<size_t>(max_keys);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // Programmatic dependents where the keys take little shared memory. Where they take
    // much, moving CTAs beside selecting ones have little of the SM's memory left for loads
    // on their way: those of 128 sequences of 1,640 rows then take 325 us, and 143 without.
    const bool early = share <= 2048;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    err = cudaLaunchKernelEx(&cfg, select, p);
    if (err != cudaSuccess) return err;
    // Slices of 128 bytes, or what divides the rows. Few sequences: of 32 bytes (a sector), larger
    // CTAs and more of them.
    const int pieces = 2 * (p.row_bytes / 16);
    const bool wide = heads < sms;
    const int most_ctas = wide ? 32 : 64;
    int lanes = 1;
    while (lanes < (wide ? 2 : 8) && pieces % (2 * lanes) == 0) lanes *= 2;
    while (lanes < 32 && pieces / lanes >= most_ctas && pieces % (2 * lanes) == 0) lanes *= 2;
    const int slices = pieces / lanes;
    const int ctas = wide || slices >= most_ctas ? most_ctas : slices + 1;
    if (static_cast<long long>(heads) * ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(static_cast<unsigned>(heads) * ctas);
    cfg.blockDim = dim3(wide ? 256 : 128);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attr + 1;
    cfg.numAttrs = early ? 1 : 0;
    err = cudaLaunchKernelEx(&cfg, wide ? evict_move_kernel<8, 4> : evict_move_kernel<4, 8>, p, lanes, ctas);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace pa

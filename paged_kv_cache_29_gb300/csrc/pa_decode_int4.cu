// pa_decode_int4.cu -- decode attention over a 4-bit cache (row format:
// pa_int4.cuh), bf16 q and output.
//
// Mathematics. K row i is lo_i + s_i c_i, so with q' = q * scale * log2(e)
//   S_i = s_i (q' . c_i) + lo_i (sum_d q'_d)
//   O   = sum_i p_i s_i c_i(V) + sum_i p_i lo_i(V),  p_i = 2^(S_i - M)
// and only the codes go through matrix products: 16 K codes x 8 query columns
// and 16 dims x 16 rows of V codes x 8 columns per m16n8k16 f16 MMA.
//
// Codes as f16 without a conversion: the bits 0x000c are the f16 subnormal
// c * 2^-24, the bits 0x00c0 are 16 c * 2^-24 and a byte 0x00dc is their sum,
// exact MMA operands all three. 2^24 is taken out of the score's and the
// output's scale.
//   K: nibbles (0, 4), (1, 5), (2, 6), (3, 7) of a word are pairs of dims of one
//   row, and q is dealt the same way, divided by 16 for the second and fourth
//   pair: 4 ANDs and a shift for 8 codes.
//   V: a transposing 8-bit ldmatrix gives a lane the bytes of four rows of one
//   byte column (two dims); w & 0x000f000f (and the other two rows') is the
//   even dim's operand, w & 0x00ff00ff the odd dim's, whose output is even + 16
//   odd and is taken apart at the end: 4 instructions for 8 codes.
// (ANDs and permutes run at half rate, and their pipe is the busiest. A byte
// 0..15 is also the e4m3 value c * 2^-9, one AND for four codes; but the e4m3 MMA
// converts its operands to f16 itself: the batch below took 66 us with it.)
//
// q is scaled by a power of two per head to [2^12, 2^13) before it becomes f16
// (exact: bf16 has fewer bits), up to |scale| max |q| of 2^115; sum q' is the product with a
// row of ones.
// A probability times its row's step is the V operand in f16. Its range, 2^-14 to
// 2^16, is spent on the rows that count: a column's reference M is taken over S +
// log2 a, a = |s| + 2^-12 |lo| the size of the row's part in the output, so that
// with E = 2^(S - M) the largest E a of the rows so far is 2^7 to 2^15 and a row of
// large step but little weight pushes nobody below. (The part of lo keeps sum E lo
// in range where s is 0, in rows of one value; a finite row's s is some 2^-12 |lo|
// at least otherwise. Relative to the largest step alone, a row of no weight with a
// step of 2^20 times the others' cost these all but 5 bits.) M is raised, and the sums
// rescaled, only when a row goes past 2^15: most units need no cross-lane maximum
// and no rescale. M is rounded to fp32, S - M once from the exact product: scores
// below 2^27 (2^28 in base 2, where M is off by at most 8) keep E a below 2^15.2 and
// the largest above 2^-1. E is fp32 and not below 2^-126 for rows that count as long as
// steps stay below 2^100; under 2^-102 a step loses bits. Sums, z = sum E lo, scores
// and outputs are fp32.
//
// Work: items (sequence, KV head, partition) of kItemRows rows, a sequence's last
// one of up to kTailRows more, dealt to persistent CTAs in the order of
// pa_plan.cuh (plan4 below); warp w of a CTA takes units w, w + 4, ... of
// 32 rows (two 16-row tiles, each inside one block) of each item. Every warp
// streams its own units through its own shared-memory ring with 16-byte
// cp.async, STAGES - 1 units ahead and across item boundaries: a tile is 1 KB of
// K codes, 1 KB of V codes and 128 bytes of pairs, too small for one producer
// warp to keep four consumers fed. At an item's end the warps' states are
// merged through shared memory.
//
// Measured: 128 sequences, 32 heads over 8 KV heads of 128 dims, 209,835 rows: 48.9
// us, 4,830 GB/s of 6,797 (a plain copy); 32 sequences of 32 KV heads 38.3 us, 4,320
// GB/s. The kernel is bound on two sides at once: three warps per scheduler issue 52 %
// of the cycles (the ALU pipe's ANDs and permutes 50 %, tensor pipe 28 %); when it took
// 48.2 us, it took 46.6 without its loads and 45.7 without its arithmetic, of which about
// 6 pass before the first tile is there and 3 are the merge launch (48.2: with references
// over the scores alone and one step exponent for all rows, which lost bits, see above).
// Measured on that build and earlier ones, no change: four interleaved chains of q . c
// MMAs, both tiles' weights before either's products, two fp32 values per instruction.
// Slower: the next unit's q . c ahead of this unit's softmax or among its products (49.8 to
// 51.2), four CTAs on an SM with 128 registers and two stages (51.6; 35.8 instead of 37.7
// for the second batch, whose items spread better over 608 CTAs, but less in flight
// everywhere else, so one rule for all), exponentials before the vote (50.7).
#include <atomic>

#include "pa_int4.cuh"
#include "pa_plan.cuh"
#include "pa_tile_math_quant.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads4 = kWarps * 32;
constexpr int kItemRows = kDefaultPartition4;
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kTailRows = kPartitionTail4;
constexpr int kWarpUnits = (kItemRows + kTailRows + kUnitRows * kWarps - 1) / (kUnitRows * kWarps);   // of an item, at most
constexpr float kRaise = 15.f, kPut = 7.f;                   // E a stays below 2^kRaise; a raise puts it at 2^kPut
constexpr float kSizeBias = 65536.f + 127.f;                 // of row_size
static_assert(2 * kWarpUnits <= 32, "a lane per tile holds its place in the pool");

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16_if(bool on, uint32_t dst, const void* src) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src), "r"(static_cast<int>(on))
        : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
// The size a = |s| + 2^-12 |lo| + 2^-102 of a V row's pair (above; the append's s are
// not negative, others' may be): the upper 16 bits of a as the low bits of 2^23.
__device__ __forceinline__ float row_size(uint32_t pair) {
    const float a = fmaf(fabsf(int4_lo(pair)), 0x1p-12f, 0x1p-102f) + fabsf(int4_step(pair));
    return __uint_as_float(__byte_perm(__float_as_uint(a), 0x4b000000u, 0x7432));
}
// An 8 x 8 matrix of 16-bit elements, two per lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void grid_dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// The work list of one CTA, in the order of pa_plan.cuh: every partition but each
// sequence's last by sequence, partition and KV head, then the last ones in 16 size
// buckets, largest first, by sequence within a bucket; dealt in a snake. Warp w
// takes the w-th quarter of the sequences, 32 at a time, so that one barrier
// joins the warps' counts: the list is there 2.0 us into the launch at 128
// sequences (the context lengths' own latency is most of it), where the general
// plan (two partition sizes, barriers per 128 sequences) took 6.3. Tried and
// slower: one CTA of three such groups per SM that take its items in turn from a
// counter (the GQA batch 53.8 us against 50.6: the CTAs' ends then agree, at the
// time at which the last of them ended before).
constexpr int kListItems = 32;                 // of the CTA's items in shared memory
constexpr int kItemShift = 10;
static_assert(kItemRows == 1 << kItemShift && kPlanBuckets == 16 && kWarps == 4, "");
// Partitions of a sequence that spans so many rows (> 0); the last one's bucket.
__device__ __forceinline__ int parts4(int span) { return max(1, (span - kTailRows + kItemRows - 1) >> kItemShift); }
__device__ __forceinline__ int bucket4(int rows) { return max(0, (kItemRows - rows) * kPlanBuckets >> kItemShift); }
struct Plan4 {
    int4 list[kListItems];                     // the CTA's items; the rest in p.items
    int full[kWarps];                          // a warp's sequences' partitions but the last
    int hist[kWarps][kPlanBuckets];            // and the last ones, by bucket
    alignas(8) float col_f[2][8];              // q columns' factors, two items' in turn; read in pairs
    int col_row[8];                            // column c's row beside column 0's
};

// All threads of the CTA; returns the launch's item count. The lists may be
// read after the next __syncthreads.
__device__ int plan4(const DecodeParams& p, int c, int C, Plan4* sm) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.num_seqs, Hkv = p.num_kv_heads;
    const int per_warp = (B + kThreads4 - 1) / kThreads4 * 32;
    const int begin = warp * per_warp, end = min(B, begin + per_warp);
    const float inv_c = 1.0f / static_cast<float>(C);
    if (lane < kPlanBuckets) sm->hist[warp][lane] = 0;
    __syncwarp();

    int full = 0, n_kept = -1;
    for (int s0 = begin; s0 < end; s0 += 32) {
        const int s = s0 + lane;
        const bool mine = s < end && (s < C ? s : s % C) == c;
        const int n = s < end ? plan_len(p, s, mine) : -1;
        n_kept = n;
        const int span = n > 0 ? n - seq_row_base(n, p.window) : 0;
        const int nf = n > 0 ? parts4(span) - 1 : 0;
        full += __reduce_add_sync(0xffffffffu, nf);
        if (n > 0) atomicAdd(&sm->hist[warp][bucket4(span - nf * kItemRows)], 1);
        // The output rows of empty sequences are zeros.
        unsigned empty = __ballot_sync(0xffffffffu, mine && n == 0);
        while (empty != 0u) {
            const int e = s0 + __ffs(empty) - 1;
            empty &= empty - 1u;
            const int chunks = p.num_queries * p.num_heads * p.head_dim / 8;   // of 16 bytes
            uint4* rows = static_cast<uint4*>(p.out) + static_cast<size_t>(e) * chunks;
            for (int i = lane; i < chunks; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (lane == 0) sm->full[warp] = full;
    __syncthreads();

    int full_at = 0, full_all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) full_at += sm->full[w];
        full_all += sm->full[w];
    }
    // Lane b < 16: where this warp's last partitions of bucket b start.
    int part_at = 0, part_all = 0;
    {
        int before = 0, count = 0;
        if (lane < kPlanBuckets) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int h = sm->hist[w][lane];
                if (w < warp) before += h;
                count += h;
            }
        }
        int incl = count;
#pragma unroll
        for (int off = 1; off < kPlanBuckets; off <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += u;
        }
        part_at = incl - count + before;
        part_all = __shfl_sync(0xffffffffu, incl, kPlanBuckets - 1);
    }
    // Puts those of items a .. e - 1 that are this CTA's. The first round is
    // found in fp32 and may come out one early, never late.
    auto put = [&](int a, int e, auto&& item) {
        if (a >= e) return;
        for (int j = max(0, static_cast<int>(static_cast<float>(a) * inv_c * 0.999999f) - 1); j * C < e; ++j) {
            const int k = snake_item(c, j, C);
            if (k < a || k >= e) continue;
            if (j < kListItems)
                sm->list[j] = item(k - a);
            else
                p.items[k] = item(k - a);
        }
    };
    const unsigned below = (1u << lane) - 1u;
    for (int s0 = begin; s0 < end; s0 += 32) {
        const int s = s0 + lane;
        const int n = per_warp == 32 ? n_kept : s < end ? plan_len(p, s, false) : -1;
        const int span = n > 0 ? n - seq_row_base(n, p.window) : 0;
        const int nf = n > 0 ? parts4(span) - 1 : 0;
        int incl = nf;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += u;
        }
        const int a = (full_at + incl - nf) * Hkv;
        put(a, a + nf * Hkv, [&](int i) { return make_int4(s, i % Hkv, i / Hkv, n); });
        full_at += __shfl_sync(0xffffffffu, incl, 31);

        const int b = n > 0 ? bucket4(span - nf * kItemRows) : kPlanBuckets;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        const int start = __shfl_sync(0xffffffffu, part_at, b & (kPlanBuckets - 1));
        if (n > 0) {
            const int f = (full_all + start + __popc(same & below)) * Hkv;
            put(f, f + Hkv, [&](int i) { return make_int4(s, i, nf, n); });
        }
        if (per_warp > 32) {
#pragma unroll
            for (int k = 0; k < kPlanBuckets; ++k) {
                const unsigned m = __ballot_sync(0xffffffffu, b == k);
                if (lane == k) part_at += __popc(m);
            }
        }
    }
    return (full_all + part_all) * Hkv;
}

template <int D, int STAGES>
struct Smem4 {
    static constexpr int kCodes = kTileRows * D / 2;                 // K or V codes of a tile
    static constexpr int kTile = 2 * kCodes + 2 * kTileRows * 4;
    static constexpr int kStage = 2 * kTile;
    static constexpr int kRing = kWarps * STAGES * kStage;
    // A warp's outputs of one column; four floats of padding spread the float2
    // stores of a half-warp (4 dim pairs x 4 column pairs) over all banks.
    static constexpr int kCol = D + 4;
    static constexpr int kState = 8 * (kCol + 2);                    // o, then m, l
    static constexpr int kMerge = kWarps * kState * 4;
    static constexpr int kQFrag = (D / 32) * 32 * 16;                // q fragments [D / 32][lane]
    static constexpr int kQ = kRing + kMerge;                        // two items' in turn
    static constexpr int kPlan = kQ + 2 * kQFrag;
    static constexpr int kBytes = kPlan + static_cast<int>(sizeof(Plan4));
    static_assert((kRing + kMerge) % 16 == 0, "16-byte fragments follow");
};

// D: head dim. kShared: at most four query columns, and the two tiles of a unit
// share the eight columns of the products: columns 0-3 are the first tile's, 4-7 the
// second's, each with a state of its own, joined where the warps' are. A lane then has
// four scores of a unit to work on instead of eight (128 sequences of 209,835 rows,
// four columns: 48.8 -> 48.0 us; 32 sequences, one column: 38.3 -> 37.7, both as built then).
template <int D, bool kShared, int STAGES, int MIN_CTAS>
__global__ void __launch_bounds__(kThreads4, MIN_CTAS) decode_int4_kernel(const DecodeParams p) {
    using Smem = Smem4<D, STAGES>;
    constexpr int kKWords = D / 32;       // words of K codes per lane and row
    constexpr int kMt = D / 16;           // m-tiles of the output
    constexpr int kSets = kShared ? 1 : 2;   // of 16 rows x 8 columns of scores in a unit

    extern __shared__ __align__(128) uint8_t smem_raw[];
    float* merge = reinterpret_cast<float*>(smem_raw + Smem::kRing);
    uint4* q_frags = reinterpret_cast<uint4*>(smem_raw + Smem::kQ);
    Plan4* const plan = reinterpret_cast<Plan4*>(smem_raw + Smem::kPlan);
    int* const col_row = plan->col_row;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, t4 = lane & 3;
    const int own = t4 >> 1;              // kShared: the tile whose scores this lane has
    const int c0 = kShared ? 2 * (t4 & 1) : 2 * t4, c1 = c0 + 1;   // its query columns
    const uint32_t ring = smem_addr(smem_raw) + warp * STAGES * Smem::kStage;
    const uint32_t ring_end = ring + STAGES * Smem::kStage;

    grid_dependency_wait();
    grid_launch_dependents();

    const int C = gridDim.x, c = blockIdx.x;
    const int Hkv = p.num_kv_heads, bs = p.block_size, Q = p.num_queries;
    const int grp = p.num_heads / Hkv, ncols = grp * Q;
    const int window = p.window > 0 ? p.window - (Q - 1) : 0;   // of one query token
    // Query column c = G j + g is head g of the group, query token j.
    if (threadIdx.x < 8) col_row[threadIdx.x] = threadIdx.x / grp * p.num_heads + threadIdx.x % grp;

    const int bs_log2 = (bs & (bs - 1)) == 0 ? __ffs(bs) - 1 : -1;

    // ---- the warp's stream of units: this lane's tile in the pool (tile units of
    // 16 rows; lane i: the warp's i-th tile of the item), the next unit, units.
    uint32_t place = 0;
    int next_unit = 0, num_units = 0;
    // The item after it: descriptor and this lane's block id; then one more.
    int4 d_next = make_int4(-1, 0, 0, 0), d_after = make_int4(-1, 0, 0, 0);
    int id_next = 0, off_next = 0;
    uint32_t issue_at = ring;

    // The warp's units of item d, its first row, and the warp's tiles (the last
    // unit may have one).
    auto units_of = [&](const int4& d, int& lo, int& tiles) {
        const int base = seq_row_base(d.w, p.window);
        lo = base + d.z * kItemRows;
        const int rows = d.z == parts4(d.w - base) - 1 ? d.w - lo : kItemRows;
        const int nt = (rows + kTileRows - 1) / kTileRows;
        const int nu = (nt + 1) / 2;
        const int cnt = (nu - warp + kWarps - 1) / kWarps;
        // Only the item's very last unit can be half a one.
        tiles = 2 * cnt - ((nt & 1) && cnt > 0 && warp + kWarps * (cnt - 1) == nu - 1 ? 1 : 0);
        return cnt;
    };
    // Requests the block id of this lane's tile of item d.
    auto fetch = [&](const int4& d) {
        id_next = 0;
        if (d.x < 0) return;
        int lo, tiles;
        units_of(d, lo, tiles);
        if (lane < tiles) {
            const int tok = lo + kUnitRows * (warp + kWarps * (lane >> 1)) + kTileRows * (lane & 1);
            const int col = bs_log2 >= 0 ? tok >> bs_log2 : tok / bs;
            off_next = (tok - col * bs) / kTileRows;
            id_next = __ldg(p.block_tables + static_cast<size_t>(d.x) * p.max_blocks_per_seq + col);
        }
    };
    // Makes the fetched item d the stream's current one. A block id outside
    // the pool is flagged and replaced: the output is unspecified, every read
    // stays inside the pool.
    auto enter = [&](const int4& d) {
        int lo, num_tiles;
        num_units = units_of(d, lo, num_tiles);
        next_unit = 0;
        int id = id_next;
        if (id < 0 || id >= p.num_blocks) {
            raise_error(p.error_word, PA_DEVERR_BLOCK_ID);
            id = 0;
        }
        // A unit's missing second tile is the pool's first one: in bounds, and
        // every row of it is masked.
        place = lane < num_tiles ? (static_cast<uint32_t>(id) * Hkv + d.y) * (bs / kTileRows) + off_next : 0u;
    };
    // Copies one tile. A lane takes 16-byte chunk `lane` (and lane + 32) of the K
    // and of the V codes, rows in order; chunks are permuted within each 128
    // bytes so that the reads below hit every bank once: K rows 2 gid + const by
    // lanes (gid, t4), V chunks of 8 rows in order.
    const int line = lane >> 3;            // of 128 bytes: 2 rows (D = 128) or 4
    const uint32_t k_to = line * 128 + (((lane & 7) ^ ((line & 1) << (D == 128 ? 2 : 1))) << 4);
    const uint32_t v_to = Smem::kCodes + line * 128 + (((lane & 7) ^ (D == 128 ? line : line & 1)) << 4);
    const uint8_t* const k_from = static_cast<const uint8_t*>(p.k_cache) + lane * 16;
    const uint8_t* const v_from = static_cast<const uint8_t*>(p.v_cache) + lane * 16;
    // Pairs of both tiles in one instruction: lanes 0-7 the first tile's, 8-15
    // the second's (4 chunks of K, 4 of V each).
    const uint32_t* const pairs_from = ((lane & 4) ? p.v_pairs : p.k_pairs) + (lane & 3) * 4;
    const uint32_t pairs_to = ((lane >> 3) & 1) * Smem::kTile + 2 * Smem::kCodes + (lane & 7) * 16;
    auto copy_codes = [&](uint32_t tile, uint32_t to) {
        const uint8_t* ks = k_from + static_cast<size_t>(tile) * Smem::kCodes;
        const uint8_t* vs = v_from + static_cast<size_t>(tile) * Smem::kCodes;
        cp_async_16(to + k_to, ks);
        cp_async_16(to + v_to, vs);
        if constexpr (D == 128) {          // 4 lines on: both permutations repeat
            cp_async_16(to + k_to + 512, ks + 512);
            cp_async_16(to + v_to + 512, vs + 512);
        }
    };
    int total = 0, j_next = 1;
    auto own_item = [&](int j) -> int4 {
        const int k = snake_item(c, j, C);
        if (k >= total) return make_int4(-1, 0, 0, 0);
        return j < kListItems ? plan->list[j] : p.items[k];
    };
    // The next unit of the stream, if any; a commit group in any case.
    auto issue = [&]() {
        while (next_unit == num_units && d_next.x >= 0) {
            enter(d_next);
            d_next = d_after;
            fetch(d_next);
            ++j_next;
            d_after = own_item(j_next + 1);
        }
        if (next_unit < num_units) {
            const uint32_t a = __shfl_sync(0xffffffffu, place, 2 * next_unit);
            const uint32_t b = __shfl_sync(0xffffffffu, place, 2 * next_unit + 1);
            copy_codes(a, issue_at);
            copy_codes(b, issue_at + Smem::kTile);
            cp_async_16_if(lane < 16, issue_at + pairs_to,
                           pairs_from + static_cast<size_t>((lane & 8) ? b : a) * kTileRows);
            ++next_unit;
        }
        cp_async_commit();
        issue_at += Smem::kStage;
        if (issue_at == ring_end) issue_at = ring;
    };

    // ---- q of an item. Warp w deals columns 2 w and 2 w + 1: 16 lanes each (8
    // with D = 64), 8 dims a lane, as f16 into the B fragments of the MMAs' lanes
    // (gid = column, t4 = the lane's quarter of the dims).
    constexpr int kQLanes = D / 8;
    const int q_col = 2 * warp + lane / 16, q_part = lane % 16;
    const bool q_mine = q_col < ncols && q_part < kQLanes;
    const int q_row = q_mine ? q_col / grp * p.num_heads + q_col % grp : 0;
    uint4 q_raw = make_uint4(0u, 0u, 0u, 0u);   // of the next item to deal
    auto load_q = [&](const int4& d) {
        if (d.x >= 0 && q_mine)
            q_raw = __ldg(reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(p.q) +
                (static_cast<size_t>(d.x) * Q * p.num_heads + d.y * grp + q_row) * D) + q_part);
    };
    auto deal_q = [&](int buf) {
        uint4* q_frag = q_frags + buf * (Smem::kQFrag / 16);
        const uint32_t w[4] = {q_raw.x, q_raw.y, q_raw.z, q_raw.w};
        float x[8], mx = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo(w[e]);
            x[2 * e + 1] = bf16_hi(w[e]);
            mx = fmaxf(mx, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        // f = 2^(139 - ex) with mx * f in [2^12, 2^13). A negative scale turns q, so
        // that the factor F below is positive.
        const int ex = max(13, min(253, static_cast<int>(__float_as_uint(mx) >> 23)));
        const float f = copysignf(__uint_as_float(static_cast<uint32_t>(266 - ex) << 23), p.scale_log2);
        const float g = f * 0.0625f;
        if (q_col < 8 && q_part < kQLanes)
            q_frag[q_part % kKWords * 32 + q_col * 4 + q_part / kKWords] =
                make_uint4(pack_f16x2(x[0] * f, x[4] * f), pack_f16x2(x[1] * g, x[5] * g),
                           pack_f16x2(x[2] * f, x[6] * f), pack_f16x2(x[3] * g, x[7] * g));
        // S = F S', S' = s acc + lo qsum, acc = f 2^-24 q . c, qsum = f 2^-24 q . 1,
        // F = |scale| 2^24 / f, kept above 0 (scale 0 gives equal weights). 2^24 / f is
        // multiplied on in two halves: its range is wider than F's, and F below 2^128 is
        // |scale| mx below 2^115.
        if (q_part == 0) {
            const int k = ex - 115, k0 = k >> 1;
            const float F = fabsf(p.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + k0) << 23) *
                            __uint_as_float(static_cast<uint32_t>(127 + k - k0) << 23);
            plan->col_f[buf][q_col] = fmaxf(F, __uint_as_float(1u));
        }
    };
    uint32_t qb[kKWords][4];
    float qf[2], qsum[2];                  // of columns c0 and c1
    auto take_q = [&](int buf) {
        const uint4* q_frag = q_frags + buf * (Smem::kQFrag / 16);
        float ones[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kKWords; ++i) {
            const uint4 v = q_frag[i * 32 + (kShared ? lane & 15 : lane)];
            qb[i][0] = v.x; qb[i][1] = v.y; qb[i][2] = v.z; qb[i][3] = v.w;
            mma_16816_f16(ones, 0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u, v.x, v.y);
            mma_16816_f16(ones, 0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u, v.z, v.w);
        }
        const float2 F = *reinterpret_cast<const float2*>(&plan->col_f[buf][c0]);
        qf[0] = F.x; qf[1] = F.y;
        qsum[0] = ones[0]; qsum[1] = ones[1];
    };

    // Takes a pair with an infinity or NaN out of a row's products and puts NaN
    // into the scores that are not masked.
    auto confine = [](uint32_t& pair, float& a, float& b) {
        if ((pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u) {
            pair = 0u;
            if (a != -INFINITY) a = NAN;
            if (b != -INFINITY) b = NAN;
        }
    };

    total = plan4(p, c, C, plan);
    __syncthreads();
    int4 it = own_item(0);
    if (it.x < 0) return;
    fetch(it);
    enter(it);
    load_q(it);
    d_next = own_item(1);
    fetch(d_next);
    d_after = own_item(2);
#pragma unroll 1
    for (int i = 0; i < STAGES - 1; ++i) issue();
    deal_q(0);
    __syncthreads();

    uint32_t at = ring;                    // the stage of the next unit
    const int j0 = c0 / grp, j1 = c1 / grp;   // the columns' query tokens
    // This lane's offsets into a tile: K rows 2 gid and 2 gid + 1, the V row that
    // it points ldmatrix at (lanes 16-31: the next 16 bytes of the same rows).
    const int k_unit = D == 128 ? t4 ^ ((gid & 1) << 2) : (((gid & 1) << 2) | (t4 >> 1)) ^ (gid & 2);
    const uint32_t k_at = D == 128 ? gid * 128 : (gid >> 1) * 128 + (t4 & 1) * 8;
    const int vr = lane & 15;
    const uint32_t v_row = D == 128 ? (vr >> 1) * 128 : (vr >> 2) * 128;
    const int v_unit = D == 128 ? (((vr & 1) << 2) | (lane >> 4)) ^ ((vr >> 1) & 3)
                                : (((vr & 3) << 1) | (lane >> 4)) ^ ((vr >> 2) & 1);
    int4 it_next = own_item(1);
    for (int j = 0; it.x >= 0; ++j) {
        const int n = it.w;
        int lo, tiles;
        const int cnt = units_of(it, lo, tiles);
        const int4 it_after = own_item(j + 2);
        take_q(j & 1);
        load_q(it_next);                   // dealt at this item's end
        float o[kMt][4];
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][e] = 0.f;
        // References M; r = -M (0 while a column has seen no row).
        float m0 = -INFINITY, m1 = -INFINITY, r0 = 0.f, r1 = 0.f;
        float l0 = 0.f, l1 = 0.f, z0 = 0.f, z1 = 0.f;
        float raise_at = -INFINITY;        // until every column has seen a row

        for (int i = 0; i < cnt; ++i) {
            issue();
            cp_async_wait_group<STAGES - 1>();
            __syncwarp();
            const int row0 = lo + kUnitRows * (warp + kWarps * i);

            // ---- S' of rows 2 gid, 2 gid + 1 of a tile (both tiles), columns c0, c1
            float S[kSets][4];
            uint2 vp[kSets];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t kb = at + h * Smem::kTile + k_at;
                uint32_t kw[2][kKWords];
                if constexpr (D == 128) {
                    const uint4 a = lds128(kb + k_unit * 16), b = lds128(kb + (k_unit ^ 4) * 16);
                    kw[0][0] = a.x; kw[0][1] = a.y; kw[0][2] = a.z; kw[0][3] = a.w;
                    kw[1][0] = b.x; kw[1][1] = b.y; kw[1][2] = b.z; kw[1][3] = b.w;
                } else {
                    const uint2 a = lds64(kb + k_unit * 16), b = lds64(kb + (k_unit ^ 2) * 16);
                    kw[0][0] = a.x; kw[0][1] = a.y;
                    kw[1][0] = b.x; kw[1][1] = b.y;
                }
                float acc[4] = {0.f, 0.f, 0.f, 0.f}, bcc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < kKWords; ++u) {
                    const uint32_t a = kw[0][u], b = kw[1][u], a8 = a >> 8, b8 = b >> 8;
                    mma_16816_f16(acc, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u,
                                  b & 0x00f000f0u, qb[u][0], qb[u][1]);
                    mma_16816_f16(bcc, a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u,
                                  b8 & 0x00f000f0u, qb[u][2], qb[u][3]);
                }
                const int set = kShared ? 0 : h;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!kShared || h == 0 || own == 1) S[set][e] = acc[e] + bcc[e];
            }
#pragma unroll
            for (int h = 0; h < kSets; ++h) {
                const uint32_t pb = at + (kShared ? own : h) * Smem::kTile + 2 * Smem::kCodes;
                const uint2 kp = lds64(pb + 8 * gid);
                vp[h] = lds64(pb + 64 + 8 * gid);
                S[h][0] = fmaf(int4_step(kp.x), S[h][0], int4_lo(kp.x) * qsum[0]);
                S[h][1] = fmaf(int4_step(kp.x), S[h][1], int4_lo(kp.x) * qsum[1]);
                S[h][2] = fmaf(int4_step(kp.y), S[h][2], int4_lo(kp.y) * qsum[0]);
                S[h][3] = fmaf(int4_step(kp.y), S[h][3], int4_lo(kp.y) * qsum[1]);
            }
            if (row0 + kUnitRows - 1 > n - Q || (window > 0 && row0 <= n - 1 - window)) {
                // Some token does not see some row of the unit (whose second tile
                // may not be there at all).
                const int top0 = n - Q + j0, top1 = n - Q + j1;
                const int w = window > 0 ? window : INT_MAX;
#pragma unroll
                for (int h = 0; h < kSets; ++h) {
                    const int r = row0 + kTileRows * (kShared ? own : h) + 2 * gid;
                    if (!(r <= top0 && top0 - r < w)) S[h][0] = -INFINITY;
                    if (!(r <= top1 && top1 - r < w)) S[h][1] = -INFINITY;
                    if (!(r + 1 <= top0 && top0 - r - 1 < w)) S[h][2] = -INFINITY;
                    if (!(r + 1 <= top1 && top1 - r - 1 < w)) S[h][3] = -INFINITY;
                    // Rows that no token sees may hold any pair.
                    if (r >= n || n - Q - r >= w) vp[h].x = 0u;
                    if (r + 1 >= n || n - Q - r - 1 >= w) vp[h].y = 0u;
                    // A pair that is not finite reaches the tokens that see its row
                    // through their scores: as a factor it would reach the others
                    // too (0 * infinity).
                    confine(vp[h].x, S[h][0], S[h][1]);
                    confine(vp[h].y, S[h][2], S[h][3]);
                }
            }
            // X = F S' - M, and beside it log2 of the row's a (see above): the upper
            // half of a's bits b stands for b / 128 - 127, at most 0.1 too low. As the
            // low bits of 2^23 and in units of 1 / 128 it reads 65536 + b / 128.
            float X[kSets][4], ab[kSets][2];
            float top = -INFINITY;
#pragma unroll
            for (int h = 0; h < kSets; ++h) {
                X[h][0] = fmaf(S[h][0], qf[0], r0); X[h][1] = fmaf(S[h][1], qf[1], r1);
                X[h][2] = fmaf(S[h][2], qf[0], r0); X[h][3] = fmaf(S[h][3], qf[1], r1);
                ab[h][0] = row_size(vp[h].x);
                ab[h][1] = row_size(vp[h].y);
                top = fmaxf(top, fmaxf(fmaf(ab[h][0], 0x1p-7f, fmaxf(X[h][0], X[h][1])),
                                       fmaf(ab[h][1], 0x1p-7f, fmaxf(X[h][2], X[h][3]))));
            }
            if (__any_sync(0xffffffffu, top > raise_at)) {
                float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
                for (int h = 0; h < kSets; ++h) {
                    const float x = fmaf(ab[h][0], 0x1p-7f, -kSizeBias), y = fmaf(ab[h][1], 0x1p-7f, -kSizeBias);
                    n0 = fmaxf(n0, fmaxf(fmaf(S[h][0], qf[0], x), fmaf(S[h][2], qf[0], y)));
                    n1 = fmaxf(n1, fmaxf(fmaf(S[h][1], qf[1], x), fmaf(S[h][3], qf[1], y)));
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
                    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
                }
                n0 = fmaxf(m0, n0 - kPut);
                n1 = fmaxf(m1, n1 - kPut);
                // Square roots of the sums' factors, applied twice: a factor may be
                // below fp32's range where the sum is large.
                const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(0.5f * (m0 - n0));
                const float a1 = m1 == -INFINITY ? 0.f : fast_exp2(0.5f * (m1 - n1));
                m0 = n0; m1 = n1;
                r0 = m0 == -INFINITY ? 0.f : -m0;
                r1 = m1 == -INFINITY ? 0.f : -m1;
                // A column that has seen no row yet takes its first reference
                // from the next unit.
                raise_at = __any_sync(0xffffffffu, m0 == -INFINITY || m1 == -INFINITY) ? -INFINITY
                                                                                       : kSizeBias + kRaise;
#pragma unroll
                for (int h = 0; h < kSets; ++h) {
                    X[h][0] = fmaf(S[h][0], qf[0], r0); X[h][1] = fmaf(S[h][1], qf[1], r1);
                    X[h][2] = fmaf(S[h][2], qf[0], r0); X[h][3] = fmaf(S[h][3], qf[1], r1);
                }
                if (i > 0) {               // else every sum is 0
                    l0 = l0 * a0 * a0; z0 = z0 * a0 * a0;
                    l1 = l1 * a1 * a1; z1 = z1 * a1 * a1;
                    const float b0 = a0 * a0, b1 = a1 * a1;
#pragma unroll
                    for (int mt = 0; mt < kMt; ++mt) {
                        o[mt][0] *= b0; o[mt][1] *= b1; o[mt][2] *= b0; o[mt][3] *= b1;
                    }
                }
            }
            // ---- o += codes(V)^T . P, tile by tile
            uint32_t b0[kSets], b1[kSets];
            auto weights = [&](int h) {
                const float E0 = fast_exp2(X[h][0]), E1 = fast_exp2(X[h][1]);
                const float E2 = fast_exp2(X[h][2]), E3 = fast_exp2(X[h][3]);
                const float u0 = int4_step(vp[h].x), u1 = int4_step(vp[h].y);
                const float y0 = int4_lo(vp[h].x), y1 = int4_lo(vp[h].y);
                l0 += E0 + E2;
                l1 += E1 + E3;
                z0 = fmaf(E2, y1, fmaf(E0, y0, z0));
                z1 = fmaf(E3, y1, fmaf(E1, y0, z1));
                // B operand: lane (gid, t4) takes column gid, the rows of lane groups
                // 2 t4 and 2 t4 + 1: rows 4 t4, 4 t4 + 2 (b0) and 4 t4 + 1, 4 t4 + 3 (b1)
                b0[h] = transpose8x8(pack_f16x2(E0 * u0, E1 * u0));
                b1[h] = transpose8x8(pack_f16x2(E2 * u1, E3 * u1));
            };
            if constexpr (kShared) weights(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (!kShared) weights(h);
                const bool mine = !kShared || (gid >> 2) == h;   // the other tile's columns weigh 0
                const uint32_t p0 = mine ? b0[h % kSets] : 0u, p1 = mine ? b1[h % kSets] : 0u;
                const uint32_t vb = at + h * Smem::kTile + Smem::kCodes + v_row;
#pragma unroll
                for (int u = 0; u < D / 64; ++u) {
                    // Rows 4 t4 .. + 3 (bytes 0..3) of byte columns 32 u + gid, + 8, + 16, + 24.
                    uint32_t w[4];
                    ldsm_x2_trans_b8(vb + ((v_unit ^ (2 * u)) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t x = w[q] & 0x00ff00ffu, y = prmt(w[q], 0u, 0x4341u);
                        mma_16816_f16(o[4 * u + q], x & 0x000f000fu, x, y & 0x000f000fu, y, p0, p1);
                    }
                }
            }
            __syncwarp();                  // the stage may be filled again
            at += Smem::kStage;
            if (at == ring_end) at = ring;
        }

        // ---- the warp's state and its share of the next item's q
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
            z0 += __shfl_xor_sync(0xffffffffu, z0, off);
            z1 += __shfl_xor_sync(0xffffffffu, z1, off);
        }
        float* st = merge + warp * Smem::kState;
        float* ml = st + 8 * Smem::kCol;
        const int s0 = 2 * t4, s1 = s0 + 1;   // of the state's columns
        // With its sum brought to [1, 2) by a power of two, a state's outputs are of the
        // size of V, whatever M: states join by what they weigh.
        const int x0 = min(253, static_cast<int>(__float_as_uint(l0) >> 23 & 255u));
        const int x1 = min(253, static_cast<int>(__float_as_uint(l1) >> 23 & 255u));
        const float f0 = __uint_as_float(static_cast<uint32_t>(254 - x0) << 23);
        const float f1 = __uint_as_float(static_cast<uint32_t>(254 - x1) << 23);
        if (gid == 0) {
            ml[s0] = m0 + static_cast<float>(x0 - 127);
            ml[s1] = m1 + static_cast<float>(x1 - 127);
            ml[8 + s0] = l0 * f0;
            ml[8 + s1] = l1 * f1;
        }
        z0 *= f0;
        z1 *= f1;
        // even dims: o 2^24; odd ones: (o - even's) 2^20
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
            const int d = 16 * mt + 2 * gid;   // dims d and d + 1
            *reinterpret_cast<float2*>(st + s0 * Smem::kCol + d) =
                make_float2(fmaf(o[mt][0] * 16777216.f, f0, z0),
                            fmaf((o[mt][2] - o[mt][0]) * 1048576.f, f0, z0));
            *reinterpret_cast<float2*>(st + s1 * Smem::kCol + d) =
                make_float2(fmaf(o[mt][1] * 16777216.f, f1, z1),
                            fmaf((o[mt][3] - o[mt][1]) * 1048576.f, f1, z1));
        }
        deal_q((j + 1) & 1);
        __syncthreads();                   // the states and the next q are complete
        const int nparts = parts4(n - seq_row_base(n, p.window));
        // Four dims of a column per thread.
        for (int idx = threadIdx.x; idx < ncols * (D / 4); idx += kThreads4) {
            const int g = idx / (D / 4), d = idx % (D / 4) * 4;
            const float* col = merge + g * Smem::kCol + d;
            const float* mlg = merge + 8 * Smem::kCol + g;
            constexpr int kParts = kShared ? 2 * kWarps : kWarps;   // column g, and g + 4, of each warp
            float M = -INFINITY, L = 0.f, O[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kParts; ++w) M = fmaxf(M, mlg[w % kWarps * Smem::kState + w / kWarps * 4]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kParts; ++w) {
                const float* cw4 = col + w % kWarps * Smem::kState + w / kWarps * 4 * Smem::kCol;
                const float* ml4 = mlg + w % kWarps * Smem::kState + w / kWarps * 4;
                const float cw = fast_exp2(ml4[0] - ref);
                const float2 a = *reinterpret_cast<const float2*>(cw4);
                const float2 b = *reinterpret_cast<const float2*>(cw4 + 2);
                L = fmaf(cw, ml4[8], L);
                O[0] = fmaf(cw, a.x, O[0]);
                O[1] = fmaf(cw, a.y, O[1]);
                O[2] = fmaf(cw, b.x, O[2]);
                O[3] = fmaf(cw, b.y, O[3]);
            }
            const size_t row = static_cast<size_t>(it.x) * Q * p.num_heads + it.y * grp + col_row[g];
            if (nparts == 1) {
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D + d) =
                    make_uint2(pack_bf16x2(O[0] / L, O[1] / L), pack_bf16x2(O[2] / L, O[3] / L));
            } else {
                const size_t slot = row * p.max_parts + it.z;
                *reinterpret_cast<float4*>(p.part_o + slot * D + d) = make_float4(O[0], O[1], O[2], O[3]);
                if (d == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * slot) = make_float2(M, L);
            }
        }
        __syncthreads();                   // the next states overwrite these
        it = it_next;
        it_next = it_after;
    }
    cp_async_wait_group<0>();
}

template <int D, bool SHARED, int STAGES, int MIN_CTAS>
cudaError_t run(const DecodeParams& p, int sm_count, cudaStream_t stream) {
    auto kernel = decode_int4_kernel<D, SHARED, STAGES, MIN_CTAS>;
    constexpr int smem = Smem4<D, STAGES>::kBytes;
    // The shared-memory attribute and the resulting CTAs per SM are set up
    // once per device and instance.
    static std::atomic<int> cached_per_sm[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    int per_sm = dev < kMaxDevices ? cached_per_sm[dev].load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads4, smem);
        if (err != cudaSuccess) return err;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        if (dev < kMaxDevices) cached_per_sm[dev].store(per_sm, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sm_count * per_sm));
    cfg.blockDim = dim3(kThreads4);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, p);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams& p, cudaStream_t stream) {
    static std::atomic<int> cached_sms[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    int sms = dev < kMaxDevices ? cached_sms[dev].load(std::memory_order_relaxed) : 0;
    if (sms <= 0) {
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        if (dev < kMaxDevices) cached_sms[dev].store(sms, std::memory_order_relaxed);
    }
    const int ncols = p.num_heads / p.num_kv_heads * p.num_queries;
    if (p.head_dim == 128)
        return ncols <= 4 ? run<128, true, 3, 3>(p, sms, stream) : run<128, false, 3, 3>(p, sms, stream);
    return ncols <= 4 ? run<64, true, 4, 3>(p, sms, stream) : run<64, false, 4, 3>(p, sms, stream);
}

}  // namespace pa

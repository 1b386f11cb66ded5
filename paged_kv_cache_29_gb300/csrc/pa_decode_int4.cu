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
// c * 2^-24 and the bits 0x00c0 are 16 c * 2^-24, exact MMA operands both. So
// one AND gives the codes of two dims (K) or two rows (V), and one shift by 8
// the next two of a word: 5 instructions for 8 codes. The factor 16 of the odd
// dims is taken out of q (K) and out of the output (V), 2^24 out of the
// score's and the output's scale.
//   K words need nothing more: nibbles (0, 4), (1, 5), (2, 6), (3, 7) of a word
//   are pairs of dims of one row, and q is dealt the same way.
//   V pairs two rows of one dim: one byte permute puts the halves of two rows'
//   words side by side (6 instructions for 8 codes).
//
// q is scaled by a power of two per head to [2^12, 2^13) before it becomes f16
// (exact: bf16 has fewer bits), whatever its size. A probability times its
// row's s_i is the V operand: with s_i = 2^e_i u_i (u_i < 2) the running
// reference M bounds T_i = S_i + e_i, so that 2^(T_i - M) u_i stays in f16's
// range for any sizes of the steps. M is raised only when a T exceeds it by
// more than 8 (operands up to 2^9 are as exact): most tiles need no cross-lane
// maximum and no rescale. Sums, z = sum p lo, scores and outputs are fp32.
//
// Work: items of at most 512 rows (sequence, KV head, partition) dealt to
// persistent CTAs (pa_plan.cuh); warp w of a CTA takes the 16-row tiles w,
// w + 4, ... of each item. Every warp streams its own tiles through its own
// shared-memory ring with 16-byte cp.async, STAGES - 1 tiles ahead and across
// item boundaries: a tile is 1 KB of K codes, 1 KB of V codes and 128 bytes of
// pairs, too small for one producer warp to keep four consumers fed. At an
// item's end the warps' states are merged through shared memory.
#include <atomic>

#include "pa_decode_stream.cuh"
#include "pa_int4.cuh"
#include "pa_tile_math_quant.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads4 = kWarps * 32;
constexpr int kItemRows = kDefaultPartition;
constexpr int kWarpTiles = kItemRows / kTileRows / kWarps;   // a warp's tiles of an item
constexpr float kRaise = 8.f;                                // see M above
static_assert(kWarpTiles <= 32, "a lane per tile holds its place in the pool");

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// e + 127 of a V row: its step's exponent, but at least its lo's less 20 (then
// lo 2^-e stays below 2^21, and a step that loses bits as an f16 operand adds
// less than 2^-30 of lo) and at least -100 (2^-e and its sums stay finite).
__device__ __forceinline__ uint32_t value_exponent(uint32_t pair) {
    return max(pair >> 23, max((pair >> 7) & 0xffu, 47u) - 20u);
}
// An 8 x 8 matrix of 16-bit elements, two per lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <int D, int NC, int STAGES>
struct Smem4 {
    static constexpr int kCodes = kTileRows * D / 2;                 // K or V codes of a tile
    static constexpr int kStage = 2 * kCodes + 2 * kTileRows * 4;
    static constexpr int kRing = kWarps * STAGES * kStage;
    // A warp's output of one column: lane group gid holds dims gid * D / 8 ..;
    // two floats of padding per group and four per column spread the float2
    // stores of a half-warp over all banks.
    static constexpr int kLaneDims = D / 8;
    static constexpr int kCol = 8 * (kLaneDims + 2) + 4;
    static constexpr int kState = NC * (kCol + 2);                   // o, then m, l
    static constexpr int kMerge = kWarps * kState * 4;
    static constexpr int kBytes = kRing + kMerge + 2 * 16;
    static_assert(kMerge >= 4 * plan_scratch_ints(kThreads4), "the plan's scratch lives there");
    static_assert((kRing + kMerge) % 16 == 0, "the first items follow");
};

// D: head dim. NC: query columns the state holds (an item uses ncols <= NC).
template <int D, int NC, int STAGES, int MIN_CTAS>
__global__ void __launch_bounds__(kThreads4, MIN_CTAS) decode_int4_kernel(const DecodeParams p) {
    using Smem = Smem4<D, NC, STAGES>;
    constexpr int kKWords = D / 32;       // words of K codes per lane and row
    constexpr int kVWords = D / 64;       // words of V codes per lane and row
    constexpr int kMt = D / 16;           // m-tiles of the output
    constexpr int kLaneDims = Smem::kLaneDims;

    extern __shared__ __align__(128) uint8_t smem_raw[];
    float* merge = reinterpret_cast<float*>(smem_raw + Smem::kRing);
    int4* first_items = reinterpret_cast<int4*>(smem_raw + Smem::kRing + Smem::kMerge);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_addr(smem_raw) + warp * STAGES * Smem::kStage;

    grid_dependency_wait();
    grid_launch_dependents();

    const int C = gridDim.x, c = blockIdx.x;
    const int Hkv = p.num_kv_heads, bs = p.block_size, Q = p.num_queries;
    const int grp = p.num_heads / Hkv, ncols = grp * Q;
    const int window = p.window > 0 ? p.window - (Q - 1) : 0;   // of one query token

    // ---- the warp's stream of tiles: item desc, this lane's tile in the pool
    // (tile units of 16 rows; lane i: the warp's i-th tile), next tile, count.
    uint32_t place = 0;
    int next_tile = 0, num_tiles = 0;
    // The item after it: descriptor and this lane's block id; then one more.
    int4 d_next = make_int4(-1, 0, 0, 0), d_after = make_int4(-1, 0, 0, 0);
    int id_next = 0, off_next = 0;
    int issue_stage = 0;

    auto tiles_of = [&](const int4& d, int& lo) {
        const int base = seq_row_base(d.w, p.window);
        lo = base + d.z * kItemRows;
        const int hi = min(d.w, lo + kItemRows);
        const int nt = (hi - lo + kTileRows - 1) / kTileRows;
        return (nt - warp + kWarps - 1) / kWarps;            // tiles warp, warp + W, ...
    };
    // Requests the block id of this lane's tile of item d.
    auto fetch = [&](const int4& d) {
        id_next = 0;
        if (d.x < 0) return;
        int lo;
        const int cnt = tiles_of(d, lo);
        if (lane < cnt) {
            const int tok = lo + kTileRows * (warp + kWarps * lane);
            const int col = tok / bs;
            off_next = (tok - col * bs) / kTileRows;
            id_next = __ldg(p.block_tables + static_cast<size_t>(d.x) * p.max_blocks_per_seq + col);
        }
    };
    // Makes the fetched item d the stream's current one. A block id outside
    // the pool is flagged and replaced: the output is unspecified, every read
    // stays inside the pool.
    auto enter = [&](const int4& d) {
        int lo;
        num_tiles = tiles_of(d, lo);
        next_tile = 0;
        int id = id_next;
        if (id < 0 || id >= p.num_blocks) {
            raise_error(p.error_word, PA_DEVERR_BLOCK_ID);
            id = 0;
        }
        place = (static_cast<uint32_t>(id) * Hkv + d.y) * (bs / kTileRows) + off_next;
    };
    // Copies one tile into the given stage (one commit group).
    auto copy_tile = [&](uint32_t tile) {
        const uint32_t dst = ring + issue_stage * Smem::kStage;
        const size_t at = static_cast<size_t>(tile) * Smem::kCodes;
        const uint8_t* ks = static_cast<const uint8_t*>(p.k_cache) + at + lane * 16;
        const uint8_t* vs = static_cast<const uint8_t*>(p.v_cache) + at + lane * 16;
        // V chunks are permuted within their 128 bytes so that the reads of
        // rows 2 t4 + const by the lanes (gid, t4) hit every bank once.
        const int line = lane >> 3;
        const int sw = D == 128 ? (line << 1) : ((line & 1) << 1);
        const uint32_t vd = dst + Smem::kCodes + line * 128 + (((lane & 7) ^ sw) << 4);
        cp_async_16(dst + lane * 16, ks);
        cp_async_16(vd, vs);
        if constexpr (D == 128) {
            cp_async_16(dst + 512 + lane * 16, ks + 512);
            cp_async_16(vd + 512, vs + 512);
        }
        if (lane < 8) {
            const uint32_t* pairs = lane < 4 ? p.k_pairs : p.v_pairs;
            cp_async_16(dst + 2 * Smem::kCodes + lane * 16,
                        pairs + static_cast<size_t>(tile) * kTileRows + (lane & 3) * 4);
        }
    };
    int total = 0, j_next = 1;
    auto own_item = [&](int j) -> int4 {
        const int k = snake_item(c, j, C);
        if (k >= total) return make_int4(-1, 0, 0, 0);
        return j < 2 ? first_items[j] : p.items[k];
    };
    // The next tile of the stream, if any; a commit group in any case.
    auto issue = [&]() {
        while (next_tile == num_tiles && d_next.x >= 0) {
            enter(d_next);
            d_next = d_after;
            fetch(d_next);
            ++j_next;
            d_after = own_item(j_next + 1);
        }
        if (next_tile < num_tiles) {
            copy_tile(__shfl_sync(0xffffffffu, place, next_tile));
            ++next_tile;
        }
        cp_async_commit();
        issue_stage = issue_stage + 1 == STAGES ? 0 : issue_stage + 1;
    };

    // ---- q of an item: raw rows (lane (gid, t4): column gid, D / 4 dims from
    // t4 * D / 4), then the MMA's B fragments and the column's scale and sum.
    uint4 q_raw[D / 32];
    auto load_q = [&](const int4& d) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) q_raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (d.x >= 0 && gid < ncols) {
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(p.q) + query_row(p, d.x, d.y, gid, grp) * D + t4 * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) q_raw[i] = __ldg(src + i);
        }
    };
    uint32_t qb[2 * kKWords][2];
    float qf[2], qsum[2];                  // of columns 2 t4 and 2 t4 + 1
    auto deal_q = [&]() {
        float mx = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t w[4] = {q_raw[i].x, q_raw[i].y, q_raw[i].z, q_raw[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = bf16_lo(w[e]), b = bf16_hi(w[e]);
                mx = fmaxf(mx, fmaxf(fabsf(a), fabsf(b)));
                sum += a + b;
            }
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        }
        // f = 2^k with mx * f in [2^12, 2^13); 1 / f = 2^-k.
        const int ex = max(13, min(253, static_cast<int>(__float_as_uint(mx) >> 23)));
        const float f = __uint_as_float(static_cast<uint32_t>(min(254, 266 - ex)) << 23);
        const float inv = __uint_as_float(static_cast<uint32_t>(max(1, ex - 12)) << 23);
#pragma unroll
        for (int i = 0; i < kKWords; ++i) {
            const uint32_t w[4] = {q_raw[i].x, q_raw[i].y, q_raw[i].z, q_raw[i].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = bf16_lo(w[e]) * f;
                x[2 * e + 1] = bf16_hi(w[e]) * f;
            }
            qb[2 * i][0] = pack_f16x2(x[0], x[4]);
            qb[2 * i][1] = pack_f16x2(x[1] * 0.0625f, x[5] * 0.0625f);
            qb[2 * i + 1][0] = pack_f16x2(x[2], x[6]);
            qb[2 * i + 1][1] = pack_f16x2(x[3] * 0.0625f, x[7] * 0.0625f);
        }
        // S = F (s acc + lo sum'), acc = f 2^-24 q . c: F = scale 2^24 / f.
        const float F = p.scale_log2 * (inv * 16777216.f);
        const float sp = sum * (f * (1.f / 16777216.f));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            qf[i] = __shfl_sync(0xffffffffu, F, 8 * t4 + 4 * i);
            qsum[i] = __shfl_sync(0xffffffffu, sp, 8 * t4 + 4 * i);
        }
    };

    // The first item where the warp can find it without the plan: its tiles
    // and q are on their way while the CTA computes its work list.
    const int4 first = first_item_by_warp(p, c, lane);
    static_assert(STAGES - 1 <= kWarpTiles, "a full partition fills the ring");
    if (first.x >= 0) {
        fetch(first);
        enter(first);
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) issue();
        load_q(first);
    }
    total = plan_cta<__nv_bfloat16, kThreads4>(p, c, C, reinterpret_cast<int*>(merge), first_items);
    int4 it = own_item(0);
    if (it.x < 0) {
        cp_async_wait_group<0>();
        return;
    }
    if (first.x < 0) {
        fetch(it);
        enter(it);
        load_q(it);
    }
    d_next = own_item(1);
    fetch(d_next);
    d_after = own_item(2);
    if (first.x < 0) {
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i) issue();
    }
    __syncthreads();                       // the plan's scratch becomes the merge area

    int stage = 0;
    const int j0 = (2 * t4) / grp, j1 = (2 * t4 + 1) / grp;   // the columns' query tokens
    int4 it_next = own_item(1);
    for (int j = 0; it.x >= 0; ++j) {
        const int n = it.w;
        int lo;
        const int cnt = tiles_of(it, lo);
        const int4 it_after = own_item(j + 2);
        deal_q();
        float o[kMt][4];
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][e] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, ref0 = 0.f, ref1 = 0.f;
        float l0 = 0.f, l1 = 0.f, z0 = 0.f, z1 = 0.f;

        for (int i = 0; i < cnt; ++i) {
            issue();
            cp_async_wait_group<STAGES - 1>();
            __syncwarp();
            const uint32_t kb = ring + stage * Smem::kStage;
            const uint32_t vb = kb + Smem::kCodes;
            const uint32_t pb = vb + Smem::kCodes;
            const int row0 = lo + kTileRows * (warp + kWarps * i);

            // ---- acc = q . c, rows gid and gid + 8, columns 2 t4 and 2 t4 + 1
            uint32_t kw[2][kKWords];
            if constexpr (D == 128) {
                const uint4 a = lds128(kb + lane * 16), b = lds128(kb + 512 + lane * 16);
                kw[0][0] = a.x; kw[0][1] = a.y; kw[0][2] = a.z; kw[0][3] = a.w;
                kw[1][0] = b.x; kw[1][1] = b.y; kw[1][2] = b.z; kw[1][3] = b.w;
            } else {
                const uint2 a = lds64(kb + lane * 8), b = lds64(kb + 256 + lane * 8);
                kw[0][0] = a.x; kw[0][1] = a.y;
                kw[1][0] = b.x; kw[1][1] = b.y;
            }
            float acc[4] = {0.f, 0.f, 0.f, 0.f}, bcc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < kKWords; ++u) {
                const uint32_t a = kw[0][u], b = kw[1][u], a8 = a >> 8, b8 = b >> 8;
                mma_16816_f16(acc, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u,
                              qb[2 * u][0], qb[2 * u][1]);
                mma_16816_f16(bcc, a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u,
                              b8 & 0x00f000f0u, qb[2 * u + 1][0], qb[2 * u + 1][1]);
            }
            const uint32_t kp0 = lds32(pb + 4 * gid), kp1 = lds32(pb + 32 + 4 * gid);
            uint32_t vp0 = lds32(pb + 64 + 4 * gid), vp1 = lds32(pb + 96 + 4 * gid);
            bool see[4] = {true, true, true, true};
            const bool edge = row0 + kTileRows - 1 > n - Q || (window > 0 && row0 <= n - 1 - window);
            if (edge) {
                const int top0 = n - Q + j0, top1 = n - Q + j1;
                const int r = row0 + gid;
                const int w = window > 0 ? window : INT_MAX;
                // differences of rows fit: both are below 2^31
                see[0] = r <= top0 && top0 - r < w;
                see[1] = r <= top1 && top1 - r < w;
                see[2] = r + 8 <= top0 && top0 - r - 8 < w;
                see[3] = r + 8 <= top1 && top1 - r - 8 < w;
                // Rows that no token sees may hold any pair.
                if (r >= n || n - Q - r >= w) vp0 = 0u;
                if (r + 8 >= n || n - Q - r - 8 >= w) vp1 = 0u;
            }
            // ---- T = S + e
            const uint32_t e0 = value_exponent(vp0), e1 = value_exponent(vp1);
            const float x0 = static_cast<float>(static_cast<int>(e0) - 127);
            const float x1 = static_cast<float>(static_cast<int>(e1) - 127);
            const float i0 = __uint_as_float((254u - e0) << 23), i1 = __uint_as_float((254u - e1) << 23);
            float T[4];
            T[0] = fmaf(fmaf(int4_step(kp0), acc[0] + bcc[0], int4_lo(kp0) * qsum[0]), qf[0], x0);
            T[1] = fmaf(fmaf(int4_step(kp0), acc[1] + bcc[1], int4_lo(kp0) * qsum[1]), qf[1], x0);
            T[2] = fmaf(fmaf(int4_step(kp1), acc[2] + bcc[2], int4_lo(kp1) * qsum[0]), qf[0], x1);
            T[3] = fmaf(fmaf(int4_step(kp1), acc[3] + bcc[3], int4_lo(kp1) * qsum[1]), qf[1], x1);
            if (edge) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!see[e]) T[e] = -INFINITY;
            }
            float mx0 = fmaxf(T[0], T[2]), mx1 = fmaxf(T[1], T[3]);
            if (__any_sync(0xffffffffu, mx0 > m0 + kRaise || mx1 > m1 + kRaise)) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
                }
                const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                // A column that has seen no row keeps M = -inf and sums of 0.
                ref0 = n0 == -INFINITY ? 0.f : n0;
                ref1 = n1 == -INFINITY ? 0.f : n1;
                const float a0 = fast_exp2(m0 - ref0), a1 = fast_exp2(m1 - ref1);
                m0 = n0;
                m1 = n1;
                l0 *= a0; z0 *= a0; l1 *= a1; z1 *= a1;
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt) {
                    o[mt][0] *= a0; o[mt][1] *= a1; o[mt][2] *= a0; o[mt][3] *= a1;
                }
            }
            const float E0 = fast_exp2(T[0] - ref0), E1 = fast_exp2(T[1] - ref1);
            const float E2 = fast_exp2(T[2] - ref0), E3 = fast_exp2(T[3] - ref1);
            const float u0 = int4_step(vp0) * i0, u1 = int4_step(vp1) * i1;
            const float y0 = int4_lo(vp0) * i0, y1 = int4_lo(vp1) * i1;
            l0 = fmaf(E2, i1, fmaf(E0, i0, l0));
            l1 = fmaf(E3, i1, fmaf(E1, i0, l1));
            z0 = fmaf(E2, y1, fmaf(E0, y0, z0));
            z1 = fmaf(E3, y1, fmaf(E1, y0, z1));
            // B operand: lane (gid, t4) takes column gid, rows 2 t4, 2 t4 + 1 (+ 8)
            const uint32_t b0 = transpose8x8(pack_f16x2(E0 * u0, E1 * u0));
            const uint32_t b1 = transpose8x8(pack_f16x2(E2 * u1, E3 * u1));

            // ---- o += codes(V)^T . P, rows 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
            uint32_t vw[4][kVWords];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (D == 128) {
                    const int line = t4 + 4 * (q >> 1);
                    const int unit = (((q & 1) << 2) | (gid >> 1)) ^ (t4 << 1);
                    const uint2 v = lds64(vb + line * 128 + unit * 16 + (gid & 1) * 8);
                    vw[q][0] = v.x; vw[q][1] = v.y;
                } else {
                    const int r = 2 * t4 + (q & 1) + 8 * (q >> 1);
                    const int unit = (((r & 3) << 1) | (gid >> 2)) ^ (((r >> 2) & 1) << 1);
                    vw[q][0] = lds32(vb + (r >> 2) * 128 + unit * 16 + (gid & 3) * 4);
                }
            }
#pragma unroll
            for (int u = 0; u < kVWords; ++u) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t sel = hf ? 0x7632u : 0x5410u;
                    const uint32_t x = prmt(vw[0][u], vw[1][u], sel), y = prmt(vw[2][u], vw[3][u], sel);
                    const uint32_t x8 = x >> 8, y8 = y >> 8;
                    mma_16816_f16(o[4 * u + 2 * hf], x & 0x000f000fu, x & 0x00f000f0u,
                                  y & 0x000f000fu, y & 0x00f000f0u, b0, b1);
                    mma_16816_f16(o[4 * u + 2 * hf + 1], x8 & 0x000f000fu, x8 & 0x00f000f0u,
                                  y8 & 0x000f000fu, y8 & 0x00f000f0u, b0, b1);
                }
            }
            __syncwarp();                  // the stage may be filled again
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }

        // ---- the warp's state, then the next item's q while the CTA merges
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
            z0 += __shfl_xor_sync(0xffffffffu, z0, off);
            z1 += __shfl_xor_sync(0xffffffffu, z1, off);
        }
        float* st = merge + warp * Smem::kState;
        float* ml = st + NC * Smem::kCol;
        const int c0 = 2 * t4, c1 = 2 * t4 + 1;
        if (gid == 0) {
            if (c0 < NC) { ml[c0] = m0; ml[NC + c0] = l0; }
            if (c1 < NC) { ml[c1] = m1; ml[NC + c1] = l1; }
        }
        if (c0 < NC) {                     // NC is even: c1 < NC too
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
                const int at = gid * (kLaneDims + 2) + 2 * mt;   // dims gid * kLaneDims + 2 mt, + 1
                *reinterpret_cast<float2*>(st + c0 * Smem::kCol + at) =
                    make_float2(fmaf(o[mt][0], 16777216.f, z0), fmaf(o[mt][2], 1048576.f, z0));
                *reinterpret_cast<float2*>(st + c1 * Smem::kCol + at) =
                    make_float2(fmaf(o[mt][1], 16777216.f, z1), fmaf(o[mt][3], 1048576.f, z1));
            }
        }
        load_q(it_next);
        __syncthreads();
        const int nparts = (n - seq_row_base(n, p.window) + kItemRows - 1) / kItemRows;
        for (int idx = threadIdx.x; idx < ncols * D; idx += kThreads4) {
            const int g = idx / D, d = idx - g * D;
            const float* col = merge + g * Smem::kCol + d / kLaneDims * (kLaneDims + 2) + d % kLaneDims;
            const float* mlg = merge + NC * Smem::kCol + g;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mlg[w * Smem::kState]);
            const float ref = M == -INFINITY ? 0.f : M;
            float L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float cw = fast_exp2(mlg[w * Smem::kState] - ref);
                L = fmaf(cw, mlg[w * Smem::kState + NC], L);
                O = fmaf(cw, col[w * Smem::kState], O);
            }
            const size_t row = query_row(p, it.x, it.y, g, grp);
            if (nparts == 1) {
                static_cast<__nv_bfloat16*>(p.out)[row * D + d] = __float2bfloat16_rn(O / L);
            } else {
                const size_t slot = row * p.max_parts + it.z;
                p.part_o[slot * D + d] = O;
                if (d == 0) {
                    p.part_ml[2 * slot] = M;
                    p.part_ml[2 * slot + 1] = L;
                }
            }
        }
        __syncthreads();                   // the next item's states overwrite the merge area
        it = it_next;
        it_next = it_after;
    }
    cp_async_wait_group<0>();
}

template <int D, int NC, int STAGES, int MIN_CTAS>
cudaError_t run(const DecodeParams& p, int sm_count, cudaStream_t stream) {
    auto kernel = decode_int4_kernel<D, NC, STAGES, MIN_CTAS>;
    constexpr int smem = Smem4<D, NC, STAGES>::kBytes;
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
        return ncols <= 4 ? run<128, 4, 5, 4>(p, sms, stream) : run<128, 8, 4, 4>(p, sms, stream);
    return ncols <= 4 ? run<64, 4, 6, 4>(p, sms, stream) : run<64, 8, 6, 4>(p, sms, stream);
}

}  // namespace pa

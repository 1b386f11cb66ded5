// pa_int4.cuh -- the 4-bit cache row: head_dim codes c in 0..15, two to a byte
// (dim 2j in the low nibble of byte j), and one bf16 pair (lo, s) held as one
// 32-bit word (lo in the low half); value = lo + s * c.
//
//   lo = min x rounded down to bf16, s = (max x - lo) / 15 rounded up to bf16,
//   c = (x - lo) / s rounded half to even, clamped to 0..15 (s = 0: 0).
//
// Differences and quotients are IEEE fp32, so every caller gives the same
// bits. The pair costs 4 bytes a row where fp32 would cost 8 (11 % of a row at
// head dim 128); rounding lo down and s up keeps every x inside the codes'
// range, and codes are computed against the pair that is kept. For a bf16 row lo
// is exact and the step at most 2^-7 of itself wider than (max - min) / 15; for an
// fp32 row rounding lo widens the range by up to 2^-7 |lo|, whatever the row's
// spread: values from 1003.90 to 1003.99 get lo 1000 and a step of 0.27. bf16 and
// not f16, so that any bf16 row with a finite max - min has a finite pair.
#pragma once

#include "pa_common.cuh"

namespace pa {

__device__ __forceinline__ float int4_lo(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float int4_step(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// IEEE quotients d / s by one divisor: with r the correctly rounded 1 / s and
// q0 = d r, the remainder m = d - q0 s is exact in an FMA, and q0 + m r is rounded
// once (the correction step of P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990). Before that
// rounding it is within 2^-22 of a last place of the quotient, and s, 15 or a
// bf16 value, has at most 8 significant bits, so that no quotient comes nearer
// than 2^-9 of a place to a rounding boundary. That needs s, and d where it
// counts, away from underflow.
__device__ __forceinline__ float int4_quotient(float d, float s, float r) {
    const float q = __fmul_rn(d, r);
    return __fmaf_rn(__fmaf_rn(-q, s, d), r, q);
}
// Two fp32 values side by side in one register pair: one instruction each.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Steps (and a row's max - lo) outside these bounds divide instead.
constexpr float kInt4Small = 0x1p-80f, kInt4Large = 0x1p80f;

// The pair of a row from its smallest and largest element (a zero lo is +0), lo
// being exact where the row is bf16.
template <bool BF16>
__device__ __forceinline__ uint32_t int4_pair(float mn, float mx) {
    mn = __fadd_rn(mn, 0.f);
    uint32_t lo = __float_as_uint(mn);
    // Down to bf16: towards zero, and one step on where that went up.
    if constexpr (!BF16) lo = (lo + ((lo >> 31) ? 0xffffu : 0u)) & 0xffff0000u;
    const float d = __fsub_rn(mx, __uint_as_float(lo));
    float s = int4_quotient(d, 15.0f, 1.0f / 15.0f);
    if (!(d >= kInt4Small) && d != 0.f) s = __fdiv_rn(d, 15.0f);
    // Up to bf16 (s is not negative); an infinite or NaN row stays itself.
    const uint32_t up = (__float_as_uint(s) + 0xffffu) & 0xffff0000u;
    return (lo >> 16) | up;
}

// N consecutive dims' codes (N = 8 or 16), dim e in nibble e. A finite row's
// quotients lie in 0..15: lo is at most its minimum, lo + 15 s at least its
// maximum but for rounding that the rounding to an integer removes.
template <int N>
__device__ __forceinline__ void int4_codes(const float* x, uint32_t pair, uint32_t* codes) {
    const float lo = int4_lo(pair), step = int4_step(pair);
    const float r = step > 0.f ? __frcp_rn(step) : 0.f;   // a row of one value: differences 0
    float q[N];
    if (step == 0.f || (step > kInt4Small && step < kInt4Large)) {
        const uint64_t mlo = f32x2(-lo, -lo), ms = f32x2(-step, -step), r2 = f32x2(r, r);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const uint64_t d = add2(f32x2(x[e], x[e + 1]), mlo), q0 = mul2(d, r2);
            const uint64_t q1 = add2(fma2(fma2(q0, ms, d), r2, q0), f32x2(12582912.f, 12582912.f));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(q[e]), "=f"(q[e + 1]) : "l"(q1));
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = __fadd_rn(__fdiv_rn(__fsub_rn(x[e], lo), step), 12582912.f);
    }
    // Adding 1.5 * 2^23 rounds to an integer, half to even, into the low bits; the
    // integers' common upper bits are taken off the sum below, mod 2^32.
    constexpr uint32_t kBits = 0x4b400000u;
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        uint32_t w = 0u;
#pragma unroll
        for (int e = 7; e >= 0; --e) w = w * 16u + __float_as_uint(q[8 * i + e]);
        codes[i] = w - kBits * 0x11111111u;
    }
}

// A row spread over TPR consecutive lanes, 8 dims each (live: this lane holds
// dims of the row): the row's pair, in every lane.
template <int TPR, bool BF16>
__device__ __forceinline__ uint32_t int4_row_pair(const float* x, bool live) {
    float mn = INFINITY, mx = -INFINITY;
    if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mn = fminf(mn, x[e]);
            mx = fmaxf(mx, x[e]);
        }
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    }
    return int4_pair<BF16>(mn, mx);
}

// Row of KV head 0 of a slot in a pool [block][kv_head][block_size]. A 64-bit
// division is some 70 instructions, so only pools that need one pay for it.
__device__ __forceinline__ long long slot_row(long long slot, long long num_slots, int num_kv_heads,
                                              int block_size) {
    if (num_slots <= 0x7fffffffLL) {
        const uint32_t s = static_cast<uint32_t>(slot), bs = static_cast<uint32_t>(block_size);
        const uint32_t blk = s / bs;
        return static_cast<long long>(blk) * num_kv_heads * block_size + (s - blk * bs);
    }
    const long long blk = slot / block_size;
    return blk * num_kv_heads * block_size + (slot - blk * block_size);
}

// Eight consecutive elements as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    ElemTraits<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    ElemTraits<float>::unpack(reinterpret_cast<const uint4*>(p)[0], x);
    ElemTraits<float>::unpack(reinterpret_cast<const uint4*>(p)[1], x + 4);
}

}  // namespace pa

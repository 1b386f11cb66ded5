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
// range, so the coarser pair widens the step by at most 2^-7 of itself and
// adds no error of its own: codes are computed against the pair that is kept.
// bf16 and not f16, so that any finite bf16 row has a finite pair.
#pragma once

#include "pa_common.cuh"

namespace pa {

__device__ __forceinline__ float int4_lo(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float int4_step(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// The pair of a row from its smallest and largest element (a zero lo is +0).
__device__ __forceinline__ uint32_t int4_pair(float mn, float mx) {
    const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rd(__fadd_rn(mn, 0.f)));
    const float step = __fdiv_rn(__fsub_rn(mx, int4_lo(lo)), 15.0f);
    return lo | (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_ru(step))) << 16);
}

// Eight consecutive dims' codes, dim e in nibble e. One reciprocal serves all
// quotients: with r the correctly rounded 1 / s, q0 = d r and the remainder
// m = d - q0 s (exact in an FMA), q0 + m r rounds to the IEEE quotient d / s
// (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990; the one exception there, a
// divisor whose fp32 significand is all ones, is no bf16 value). That needs s
// and the remainder away from underflow: rows whose step is below 2^-90 or above
// 2^90 divide instead. A finite row's quotients lie in 0..15 (lo is at most its
// minimum, lo + 15 s at least its maximum but for rounding that rint removes).
__device__ __forceinline__ uint32_t int4_codes(const float* x, uint32_t pair) {
    const float lo = int4_lo(pair), step = int4_step(pair);
    if (!(step > 0.f)) return 0u;
    float c[8];
    if (step > 0x1p-90f && step < 0x1p90f) {
        const float r = __frcp_rn(step);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = __fsub_rn(x[e], lo);
            const float q = __fmul_rn(d, r);
            c[e] = __fmaf_rn(__fmaf_rn(-q, step, d), r, q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = __fdiv_rn(__fsub_rn(x[e], lo), step);
    }
    // Adding 1.5 * 2^23 rounds to an integer, half to even; four codes are put
    // together in fp32 (below 2^16: exact) and read from the low bits.
    constexpr float kRound = 12582912.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = __fsub_rn(__fadd_rn(c[e], kRound), kRound);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float* k = c + 4 * i;
        const float v = __fmaf_rn(k[3], 4096.f, __fmaf_rn(k[2], 256.f, __fmaf_rn(k[1], 16.f, k[0])));
        w[i] = __float_as_uint(__fadd_rn(v, 8388608.f));
    }
    return __byte_perm(w[0], w[1], 0x5410);
}

// A row spread over TPR consecutive lanes, 8 dims each (live: this lane holds
// dims of the row): the row's pair, in every lane.
template <int TPR>
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
    return int4_pair(mn, mx);
}

// Eight consecutive elements as fp32, and eight fp32 values rounded and stored.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    ElemTraits<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    ElemTraits<float>::unpack(reinterpret_cast<const uint4*>(p)[0], x);
    ElemTraits<float>::unpack(reinterpret_cast<const uint4*>(p)[1], x + 4);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace pa

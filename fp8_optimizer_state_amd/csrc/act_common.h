// The FP8 activation codec's arithmetic, shared by the codec's own kernels and by
// the kernels that store their result in its format.
#pragma once

#include "coat_common.h"

namespace {

// ------------------------------------------------------------------ activation codec
//
// Article, section "Solution: mixed-granularity FP8 precision flow": layer
// inputs are kept in FP8 for the backward pass, with a quantization
// granularity that differs between layers. Plain absmax scaling of bf16
// values with one fp32 scale per tensor or per group of G consecutive values:
// s = RN32(amax / fpmax), code = encode(RN32(x / s)) (the sign alone when
// s = 0), value = RN_bf16(RN32(decode(code) s)); a tensor or group holding a
// NaN or Inf gets s = NaN and every code 0x7F.
//
// RN32(x / s) without a division per value: x has at most 8 significant bits
// and s at most 24, so a quotient that is not an fp32 number lies at least
// 2^-49 (relative) from every midpoint between fp32 neighbours (the distance
// is a nonzero multiple of 2^(e-24) / s's integer significand in the binade
// [2^e, 2^(e+1)), likewise in the subnormal range), while x times 1 / s to
// within 2^-51 of it, rounded to fp64, is within 2^-50. Rounding that product
// to fp32 thus gives RN32(x / s) exactly; the hardware converts round it to the FP8 grid,
// nearest with ties to even, after a clamp to the largest finite magnitude.

// Largest bf16 magnitude bits of the 2 NW values in w.
template <int NW>
__device__ __forceinline__ uint32_t bf16_absmax_bits(const uint32_t (&w)[NW]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const uint32_t a = w[i] & 0x7FFF7FFFu;
        const uint32_t lo = a & 0xFFFFu, hi = a >> 16;
        m = m > lo ? m : lo;
        m = m > hi ? m : hi;
    }
    return m;
}

__device__ __forceinline__ uint32_t group_umax(uint32_t v, int lanes) {
    for (int d = 1; d < lanes; d <<= 1) {
        const uint32_t o = xlane32(v, d);
        v = v > o ? v : o;
    }
    return v;
}

// The scale of a group with magnitude bits `amax_bits`: RN32(amax / fpmax), NaN
// if the group holds an Inf or NaN. The product with RN64(1 / fpmax), rounded to
// fp32, is that quotient by the argument above (amax has 8 significant bits).
template <int F>
__device__ __forceinline__ float act_scale(uint32_t amax_bits) {
    const float amax = __builtin_bit_cast(float, amax_bits << 16);
    return amax_bits >= 0x7F80u ? __builtin_nanf("") : (float)((double)amax * (1.0 / Fmt<F>::FPMAX));
}

// Codes of the 2 NW bf16 values in w (value i in half i & 1 of word i >> 1) for
// a group with magnitude bits `amax_bits` and their scale `sc`; returns the
// NW / 2 code words.
template <int F, int NW>
__device__ __forceinline__ void act_codes(const uint32_t (&w)[NW], uint32_t amax_bits, float sc, uint32_t (&out)[NW / 2]) {
    using T = Fmt<F>;
    if (amax_bits >= 0x7F80u) {  // Inf or NaN in the group
#pragma unroll
        for (int i = 0; i < NW / 2; ++i) out[i] = 0x7F7F7F7Fu;
        return;
    }
    if (sc == 0.0f) {  // all zero: the sign alone
#pragma unroll
        for (int i = 0; i < NW / 2; ++i) {
            uint32_t c = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int j = 4 * i + b;
                c |= ((w[j >> 1] >> (16 * (j & 1) + 15)) & 1u) << (8 * b + 7);
            }
            out[i] = c;
        }
        return;
    }
    // 1 / s by the hardware's estimate and two Newton steps: within 2^-51 of it,
    // x times it within 2^-50, so the argument above holds
    const double s = (double)sc;
    double r = __builtin_amdgcn_rcp(s);
    r = __builtin_fma(__builtin_fma(-s, r, 1.0), r, r);
    r = __builtin_fma(__builtin_fma(-s, r, 1.0), r, r);
#pragma unroll
    for (int i = 0; i < NW / 2; ++i) {
        float y[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int j = 4 * i + b;
            const float x = __builtin_bit_cast(float, (j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
            const float q = (float)((double)x * r);  // RN32(x / s)
            y[b] = __builtin_fminf(__builtin_fmaxf(q, -T::FPMAX_F), T::FPMAX_F);
        }
        uint32_t c = cvt_pk<F, false>(y[0], y[1], 0u);
        out[i] = cvt_pk<F, true>(y[2], y[3], c);
    }
}

}  // namespace

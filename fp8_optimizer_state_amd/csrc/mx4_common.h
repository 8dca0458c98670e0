// Microscaled 4-bit floating point (E2M1 codes, one power-of-two scale byte per
// 32 values): the arithmetic and the memory access shared by the kernels.
#pragma once

#include "coat_common.h"
#include "ops_host.h"

namespace {

// 16-byte accesses at an element's alignment: global memory takes them at any
// byte address, in one instruction (rows of an odd width start anywhere).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef __attribute__((address_space(1))) u32x4_a2 gu32x4_a2;
typedef __attribute__((address_space(1))) u32x4_a4 gu32x4_a4;
typedef __attribute__((address_space(1))) u32x2 gu32x2;

__device__ __forceinline__ float as_float(uint32_t w) { return __builtin_bit_cast(float, w); }
__device__ __forceinline__ bf16x2 word_bf16(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
// Round to nearest even; a NaN stays one.
__device__ __forceinline__ uint32_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Between what lanes of a wavefront write to LDS and what others of it read, either way round:
// LDS keeps a wavefront's order, and this has the compiler keep it too. No instruction.
__device__ __forceinline__ void exchange_between_lanes() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 8 stored elements, as they come from memory.
template <class E>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4 w;
};
template <>
struct Raw8<float> {
    u32x4 lo, hi;
};

__device__ __forceinline__ void expand(const Raw8<uint16_t>& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(r.w[i]);
        v[2 * i + 1] = bf16_hi(r.w[i]);
    }
}
__device__ __forceinline__ void expand(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = as_float(r.lo[i]);
        v[4 + i] = as_float(r.hi[i]);
    }
}

// 8 consecutive elements from p, of which the first n (maybe < 1) exist; the
// others are zero. WHOLE: n is at least 8 or at most 0.
template <bool WHOLE = false>
__device__ __forceinline__ Raw8<uint16_t> load_raw8(const uint16_t* p, int64_t n) {
    Raw8<uint16_t> r;
    if (n >= 8) {
        r.w = *reinterpret_cast<const gu32x4_a2*>(gp(p));
        return r;
    }
    r.w = u32x4{0u, 0u, 0u, 0u};
    if (WHOLE || n < 1) return r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // the first element stands in for those past the end
        const uint32_t e = gp(p)[i < n ? i : 0];
        r.w[i >> 1] |= i < n ? e << (16 * (i & 1)) : 0u;
    }
    return r;
}
template <bool WHOLE = false>
__device__ __forceinline__ Raw8<float> load_raw8(const float* p, int64_t n) {
    Raw8<float> r;
    if (n >= 8) {
        r.lo = *reinterpret_cast<const gu32x4_a4*>(gp(p));
        r.hi = *reinterpret_cast<const gu32x4_a4*>(gp(p) + 4);
        return r;
    }
    r.lo = r.hi = u32x4{0u, 0u, 0u, 0u};
    if (WHOLE || n < 1) return r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float e = gp(p)[i < n ? i : 0];
        const uint32_t b = i < n ? __builtin_bit_cast(uint32_t, e) : 0u;
        if (i < 4) r.lo[i] = b;
        else r.hi[i - 4] = b;
    }
    return r;
}

// The same in two halves, for several loads that shall be under way together: the
// load, of the row's last 8 elements where fewer than 8 are left (the row has
// 8), and what moves those into place once they are there.
__device__ __forceinline__ Raw8<uint16_t> load_end8(const uint16_t* p, int64_t n) {
    return {*reinterpret_cast<const gu32x4_a2*>(gp(p) + (n < 8 ? n - 8 : 0))};
}
__device__ __forceinline__ Raw8<float> load_end8(const float* p, int64_t n) {
    const auto q = gp(p) + (n < 8 ? n - 8 : 0);
    return {*reinterpret_cast<const gu32x4_a4*>(q), *reinterpret_cast<const gu32x4_a4*>(q + 4)};
}
__device__ __forceinline__ void settle8(Raw8<uint16_t>& r, int64_t n) {
    if (n >= 8) return;
    const int k = n > 0 ? 8 - (int)n : 8;  // elements that belong before p
    u32x4 w = r.w;
    if (k & 4) w = u32x4{w[2], w[3], 0u, 0u};
    if (k & 2) w = u32x4{w[1], w[2], w[3], 0u};
    if (k & 1)
        w = u32x4{__builtin_amdgcn_alignbit(w[1], w[0], 16), __builtin_amdgcn_alignbit(w[2], w[1], 16),
                  __builtin_amdgcn_alignbit(w[3], w[2], 16), w[3] >> 16};
    r.w = k < 8 ? w : u32x4{0u, 0u, 0u, 0u};
}
__device__ __forceinline__ void settle8(Raw8<float>& r, int64_t n) {
    if (n >= 8) return;
    const int k = n > 0 ? 8 - (int)n : 8;
    u32x4 a = r.lo, b = r.hi;
    const u32x4 none{0u, 0u, 0u, 0u};
    if (k & 4) {
        a = b;
        b = none;
    }
    if (k & 2) {
        a = u32x4{a[2], a[3], b[0], b[1]};
        b = u32x4{b[2], b[3], 0u, 0u};
    }
    if (k & 1) {
        a = u32x4{a[1], a[2], a[3], b[0]};
        b = u32x4{b[1], b[2], b[3], 0u};
    }
    r.lo = k < 8 ? a : none;
    r.hi = k < 8 ? b : none;
}

// 8 consecutive elements to p, of which the first n exist. WHOLE: as above.
template <bool WHOLE = false>
__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const float (&v)[8]) {
    if (n >= 8) {
        *reinterpret_cast<gu32x4_a2*>(gp(p)) =
            u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    } else if (!WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) gp(p)[i] = (uint16_t)bf16_bits(v[i]);
    }
}
template <bool WHOLE = false>
__device__ __forceinline__ void store8(float* p, int64_t n, const float (&v)[8]) {
    if (n >= 8) {
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __builtin_bit_cast(uint32_t, v[i]);
            b[i] = __builtin_bit_cast(uint32_t, v[4 + i]);
        }
        *reinterpret_cast<gu32x4_a4*>(gp(p)) = a;
        *reinterpret_cast<gu32x4_a4*>(gp(p) + 4) = b;
    } else if (!WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) gp(p)[i] = v[i];
    }
}

// 16 bytes of elements to p, of which the first n exist.
__device__ __forceinline__ void store16(uint16_t* p, int64_t n, const float (&v)[8]) { store8(p, n, v); }
__device__ __forceinline__ void store16(float* p, int64_t n, const float (&v)[4]) {
    if (n >= 4) {
        *reinterpret_cast<gu32x4_a4*>(gp(p)) =
            u32x4{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]), __builtin_bit_cast(uint32_t, v[2]),
                  __builtin_bit_cast(uint32_t, v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) gp(p)[i] = v[i];
    }
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Larger magnitude of each half of two words of bf16 (w's sign bits are dropped, m has none).
__device__ __forceinline__ uint32_t bf16_max2(uint32_t m, uint32_t w) {
    const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}

// fp32 bits of the largest magnitude of 8 stored elements.
__device__ __forceinline__ uint32_t absmax_bits(const Raw8<uint16_t>& r) {
    uint32_t m = bf16_max2(bf16_max2(bf16_max2(bf16_max2(0u, r.w[0]), r.w[1]), r.w[2]), r.w[3]);
    return umax(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t absmax_bits(const Raw8<float>& r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = umax(m, umax(r.lo[i] & 0x7FFFFFFFu, r.hi[i] & 0x7FFFFFFFu));
    return m;
}

// The scale byte of a block whose largest magnitude has these fp32 bits:
// e + 127 with e = floor(log2 amax) - 2 >= -127, 0xFF for an Inf or NaN. The
// exponent field of an fp32 subnormal (0) lies below the limit like its value.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    const uint32_t f = amax_bits >> 23;
    return f >= 255u ? 255u : (f > 2u ? f - 2u : 0u);
}

// The largest fp32 bits of the four lanes that share a block of 32 values.
__device__ __forceinline__ uint32_t block_max(uint32_t am) {
    am = umax(am, xlane32(am, 1));
    return umax(am, xlane32(am, 2));
}

// Codes of 8 elements of a block with scale byte b (not 0xFF), the first in the
// low bits. The convert divides by the power of two whose exponent field is b
// (2^-127 for b = 0), rounds to nearest, ties to the even code, and cuts at 6;
// tests pin that for every bf16 value and for fp32 values about each border.
__device__ __forceinline__ uint32_t mx4_codes8(const Raw8<uint16_t>& r, uint32_t b) {
    const float scale = as_float(b << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, word_bf16(r.w[0]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, word_bf16(r.w[1]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, word_bf16(r.w[2]), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, word_bf16(r.w[3]), scale, 3);
}
__device__ __forceinline__ uint32_t mx4_codes8(const Raw8<float>& r, uint32_t b) {
    const float scale = as_float(b << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(r.lo[0]), as_float(r.lo[1]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(r.lo[2]), as_float(r.lo[3]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(r.hi[0]), as_float(r.hi[1]), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, as_float(r.hi[2]), as_float(r.hi[3]), scale, 3);
}

// Values of 4 codes (the low half of c) of a block with scale byte b.
__device__ __forceinline__ void mx4_values4(uint32_t c, uint32_t b, float (&v)[4]) {
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    v[0] = p0.x; v[1] = p0.y; v[2] = p1.x; v[3] = p1.y;
    const int e = (int)b - 127;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = b == 255u ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(v[i], e);
}

}  // namespace

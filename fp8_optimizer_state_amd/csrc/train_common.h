// What the training products share on the device: random bits of the dropout,
// activations, the epilogues of a bf16 product and the products themselves.
#pragma once

#include "mx4_common.h"
#include "train_host.h"

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(1))) int64_t gi64;
typedef __attribute__((address_space(1))) int32_t gi32;
typedef __attribute__((address_space(1))) f32x2 gf32x2;

// ------------------------------------------------------------------ dropout

// Philox 4x32 with 10 rounds (Salmon et al., "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011): four random words of a counter and a key.
__device__ __forceinline__ u32x4 philox(uint64_t low, uint64_t high, uint64_t key) {
    uint32_t c0 = (uint32_t)low, c1 = (uint32_t)(low >> 32), c2 = (uint32_t)high, c3 = (uint32_t)(high >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

struct Drop {
    const int64_t* rng;
    int64_t offset;
    uint32_t threshold;  // 0: nothing is dropped
    uint64_t key, step;
    __device__ void begin() {
        if (threshold == 0) return;
        key = (uint64_t)gp(rng)[0];
        step = (uint64_t)gp(rng)[1] + (uint64_t)offset;
    }
    // Zeroes what is dropped of a block of 8 columns.
    __device__ __forceinline__ void operator()(uint64_t block, float (&v)[8]) const {
        const u32x4 w = philox(block, step, key);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu) >= threshold ? v[i] : 0.0f;
    }
};

// ------------------------------------------------------------------ activations

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x)); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2). Phi(-|z|) / e falls from 1/2
// like 1 / |z|: it is t P(t) with t = 1 / (1 + 0.3 |z|) and a P of degree 7, whose largest
// relative error up to |z| = 14, where e ends, was made least (1.5e-7; 4e-7 as computed here).
// e itself is off by up to 1.5 z^2 half steps of itself, from its argument's rounding.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float a = fabsf(z);
    e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * a * a);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
    float q = fmaf(t, 0.0356748769f, -0.157203499f);
    q = fmaf(q, t, 0.206354196f);
    q = fmaf(q, t, -0.0536842455f);
    q = fmaf(q, t, 0.128561924f);
    q = fmaf(q, t, 0.0999134088f);
    q = fmaf(q, t, 0.120753968f);
    q = fmaf(q, t, 0.119629298f);
    q = q * t * e;
    return z < 0.0f ? q : 1.0f - q;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == COAT_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == COAT_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if constexpr (ACT == COAT_ACT_GELU_TANH) return z * sigmoid(1.59576912f * fmaf(0.044715f * z * z, z, z));
    if constexpr (ACT == COAT_ACT_SILU) return z * sigmoid(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == COAT_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == COAT_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return fmaf(z * 0.398942280f, e, c);
    }
    if constexpr (ACT == COAT_ACT_GELU_TANH) {
        // past 100 the sigmoid is 0 or 1 to the last digit, and a larger square would only overflow
        const float u2 = fminf(z * z, 1e4f), s = sigmoid(1.59576912f * fmaf(0.044715f * u2, z, z));
        return fmaf(z * s * (1.0f - s), 1.59576912f * fmaf(0.134145f, u2, 1.0f), s);
    }
    if constexpr (ACT == COAT_ACT_SILU) {
        const float s = sigmoid(z);
        return fmaf(z * s, 1.0f - s, s);
    }
    return 1.0f;
}

// f with the activation known to the compiler.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case COAT_ACT_RELU: f(std::integral_constant<int, COAT_ACT_RELU>{}); break;
        case COAT_ACT_GELU: f(std::integral_constant<int, COAT_ACT_GELU>{}); break;
        case COAT_ACT_GELU_TANH: f(std::integral_constant<int, COAT_ACT_GELU_TANH>{}); break;
        case COAT_ACT_SILU: f(std::integral_constant<int, COAT_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, COAT_ACT_NONE>{}); break;
    }
}

// What rounding to bf16 leaves of 8 values (of a NaN or Inf nothing more).
__device__ __forceinline__ void left_of(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float left = v[i] - as_float(bf16_bits(v[i]) << 16);
        v[i] = fabsf(left) < __builtin_inff() ? left : 0.0f;
    }
}

// 8 values in bf16 with zeros for infinities and NaN, beside second terms: the first ones carry
// those, and zero times infinity would make a NaN of them.
__device__ __forceinline__ u32x4 finite_of(u32x4 w) {
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
        if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
    }
    return w;
}

// 8 columns past the caches' usual order where whole lines leave for memory anyway, and
// would drive the operands out of them.
__device__ __forceinline__ void store8_past(bool past, uint16_t* p, int64_t n, const float (&v)[8]) {
    if (past && n >= 8) {
        const u32x4 w{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<gu32x4_a2*>(gp(p)));
    } else {
        store8(p, n, v);
    }
}
__device__ __forceinline__ void store8_past(bool, float* p, int64_t n, const float (&v)[8]) { store8(p, n, v); }

// ------------------------------------------------------------------ epilogues
//
// What becomes of a product's sums. A kernel hands over 8 consecutive columns of a
// row at a time, the first a multiple of 8; n of them exist (n may be over 8). What it
// needs from memory for 8 columns (Column) and for them in one row (Row) is loaded apart
// from that, so that the loads of several rows are under way together. kLarge: its products may be
// made in tiles of 256 x 256.

// y = residual + scale D(act(sum + bias)), z = sum + bias.
template <class T>
struct LinearOut {
    static constexpr bool kLogSum = false, kLarge = true;
    const void* bias;
    const T* residual;
    uint16_t* z;
    T* y;
    int64_t ldr, ldz, ldy, blocks;  // blocks of 8 columns of a row
    Drop drop;
    float scale;  // the dropout's factor in it
    int32_t act, bias_type;
    bool y_past, z_past;
    struct Column {
        float b[8];
    };
    typedef Raw8<T> Row;
    __device__ void begin() { drop.begin(); }
    __device__ __forceinline__ Column column(int64_t col, int64_t n) const {
        Column c = {};
        if (bias) {
            if (bias_type == COAT_FP32) expand(load_raw8(static_cast<const float*>(bias) + col, n), c.b);
            else expand(load_raw8(static_cast<const uint16_t*>(bias) + col, n), c.b);
        }
        return c;
    }
    __device__ __forceinline__ Row row(int64_t row, int64_t col, int64_t n) const {
        return residual ? load_raw8(residual + row * ldr + col, n) : Row{};
    }
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n, const Column& c, const Row& raw) const {
        if (bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += c.b[i];
        }
        if (z) store8_past(z_past, z + row * ldz + col, n, v);
        with_act(act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = activate<a.value>(v[i]);
        });
        if (drop.threshold) drop((uint64_t)(row * blocks + col / 8), v);
        if (residual) {
            float r[8];
            expand(raw, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], scale, r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= scale;
        }
        store8_past(y_past, y + row * ldy + col, n, v);
    }
};

// y = scale sum in bf16.
struct ScaledOut {
    static constexpr bool kLogSum = false, kLarge = true;
    const float* scale_at;  // in device memory, or
    float scale;
    uint16_t* y;
    int64_t ldy;
    struct Column {};
    struct Row {};
    __device__ void begin() {
        if (scale_at) scale = *gp(scale_at);
    }
    __device__ __forceinline__ Column column(int64_t, int64_t) const { return Column{}; }
    __device__ __forceinline__ Row row(int64_t, int64_t, int64_t) const { return Row{}; }
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n, const Column&, const Row&) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
        store8(y + row * ldy + col, n, v);
    }
};

// The same of sums that come in pieces: on top of those of earlier pieces, and into
// those for later ones or, behind the last, to row rows[i] of y for row i.
// With second terms the factor and the rows may be given otherwise, and a second sum changes
// nothing that is not finite already. That is a type of its own: as choices at run time, here
// and in GradOut, it made the gradients of 8192 x 32000 x 5120 take 6370 us instead of 5830.
// In tiles of 256 x 256 eight registers of the addresses go to scratch once a tile, on its way out.
template <bool TWO>
struct PiecesOut {
    static constexpr bool kLogSum = false, kLarge = !TWO;
    const float* scale_at;  // in device memory; with second terms may be NULL: scale
    const int32_t* rows;    // with second terms may be NULL: row i
    uint16_t* y;            // NULL: not the last piece
    int64_t ldy;
    float* acc;
    int64_t lda;
    bool first;
    float scale;
    bool second;            // these are sums of second terms
    struct Column {};
    typedef Raw8<float> Row;
    __device__ void begin() {
        if (!TWO || scale_at) scale = *gp(scale_at);
    }
    __device__ __forceinline__ Column column(int64_t, int64_t) const { return Column{}; }
    __device__ __forceinline__ Row row(int64_t row, int64_t col, int64_t) const {
        return first ? Row{} : load_raw8<true>(acc + row * lda + col, 8);  // its rows hold whole blocks
    }
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n, const Column&, const Row& r) const {
        float a[8];
        expand(r, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = TWO && second && !(fabsf(a[i]) < __builtin_inff()) ? a[i] : v[i] + a[i];
        if (!y) {
            store8<true>(acc + row * lda + col, 8, v);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
        store8(y + (!TWO || rows ? (int64_t)gp(rows)[row] : row) * ldy + col, n, v);
    }
};

// The logits' part of the loss: per row and part of kWidth columns the maximum m and
// the sum of exp(l - m), the label's own logit left out and kept apart (so that the
// loss of a token that the model is sure of keeps its digits).
struct LogSumOut {
    static constexpr bool kLogSum = true, kLarge = true;
    const int32_t* label;
    float* zt;
    f32x2* part;   // [part][row]
    int64_t rows;  // of the workspace's arrays
    __device__ void begin() {}
    __device__ __forceinline__ int32_t label_of(int64_t row) const { return gp(label)[row]; }
    __device__ __forceinline__ void keep(int64_t row, float logit) const { gp(zt)[row] = logit; }
    __device__ __forceinline__ void put(int64_t row, int64_t p, float m, float s) const {
        reinterpret_cast<gf32x2*>(gp(part))[p * rows + row] = f32x2{m, s};
    }
};

// What a row of logits' gradients needs: {lse, weight over the largest weight, label's bits,
// own}. The gradient g = weight (exp(l - lse) - [the label]) in bf16; columns past the end up
// to a whole block are zero. At the label that is -(1 - p) = expm1(-loss), `own`, which keeps
// its digits where exp(l - lse) - 1 cancels (lse's rounding alone moves it by 2^-24 |lse|, of a
// loss of 1e-5 at a logit of 60 a seventh). A positive own: the loss is not known, and the
// difference is taken. With second terms, what the rounding to bf16 leaves goes to row i + *count.
template <bool TWO>
struct GradOut {
    static constexpr bool kLogSum = false, kLarge = !TWO;
    const f32x4* info;
    uint16_t* g;
    int64_t ldg, col0;     // first column of the piece in the vocabulary
    const int32_t* count;  // with second terms
    int64_t second;
    struct Column {};
    typedef f32x4 Row;
    __device__ void begin() {
        if constexpr (TWO) second = (int64_t)*gp(count);
    }
    __device__ __forceinline__ Column column(int64_t, int64_t) const { return Column{}; }
    __device__ __forceinline__ Row row(int64_t row, int64_t, int64_t) const { return reinterpret_cast<const gf32x4*>(gp(info))[row]; }
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n, const Column&, const Row& r) const {
        const float label = r[2];  // a bit cast of an element of a vector would take its first
        const int64_t hit = (int64_t)__builtin_bit_cast(int32_t, label) - col0 - col;
        const float own = r[3] > 0.0f ? -1.0f : r[3], times = r[3] > 0.0f ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = exp_fast(v[i] - r[0]);
            v[i] = i < n ? r[1] * (i == hit ? fmaf(p, times, own) : p) : 0.0f;
        }
        store8<true>(g + row * ldg + col, 8, v);
        if constexpr (TWO) {
            left_of(v);
            store8<true>(g + (row + second) * ldg + col, 8, v);
        }
    }
};

}  // namespace

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

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2), by Hastings'
// rational approximation of the error function (Abramowitz and Stegun 7.1.26, off
// by at most 1.5e-7): Phi(-|z|) = e (a1 t + .. + a5 t^5) / 2, t = 1 / (1 + 0.3275911 |z| / sqrt 2).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float a = fabsf(z);
    e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * a * a);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.231641888f, a, 1.0f));
    float q = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
    q = fmaf(q, t, 0.5f * 1.421413741f);
    q = fmaf(q, t, 0.5f * -0.284496736f);
    q = fmaf(q, t, 0.5f * 0.254829592f);
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

// ------------------------------------------------------------------ epilogues
//
// What becomes of a product's sums. A kernel hands over 8 consecutive columns of a
// row at a time, the first a multiple of 8; n of them exist (n may be over 8).

// y = residual + scale D(act(sum + bias)), z = sum + bias.
template <class T>
struct LinearOut {
    static constexpr bool kLogSum = false;
    const void* bias;
    const T* residual;
    uint16_t* z;
    T* y;
    int64_t ldr, ldz, ldy, blocks;  // blocks of 8 columns of a row
    Drop drop;
    float scale;  // the dropout's factor in it
    int32_t act, bias_type;
    __device__ void begin() { drop.begin(); }
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n) const {
        if (bias) {
            float b[8];
            if (bias_type == COAT_FP32) expand(load_raw8(static_cast<const float*>(bias) + col, n), b);
            else expand(load_raw8(static_cast<const uint16_t*>(bias) + col, n), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
        if (z) store8(z + row * ldz + col, n, v);
        with_act(act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = activate<a.value>(v[i]);
        });
        if (drop.threshold) drop((uint64_t)(row * blocks + col / 8), v);
        float r[8] = {};
        if (residual) {
            expand(load_raw8(residual + row * ldr + col, n), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], scale, r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= scale;
        }
        store8(y + row * ldy + col, n, v);
    }
};

// y = scale sum in bf16, on top of the sums of earlier pieces and into those for later
// ones where there are any; row i of y is row rows[i] of memory.
struct ScaledOut {
    static constexpr bool kLogSum = false;
    const float* scale_at;  // in device memory, or
    float scale;
    const int32_t* rows;
    uint16_t* y;  // NULL: not the last piece
    int64_t ldy;
    float* acc;  // NULL: the only piece
    int64_t lda;
    bool first;
    __device__ void begin() {
        if (scale_at) scale = *gp(scale_at);
    }
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n) const {
        if (acc) {
            float* const at = acc + row * lda + col;  // its rows hold whole blocks
            if (!first) {
                float a[8];
                expand(load_raw8<true>(at, 8), a);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += a[i];
            }
            if (!y) {
                store8<true>(at, 8, v);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
        store8(y + (rows ? (int64_t)gp(rows)[row] : row) * ldy + col, n, v);
    }
};

// The logits' part of the loss: per row and part of kWidth columns the maximum m and
// the sum of exp(l - m), the label's own logit left out and kept apart (so that the
// loss of a token that the model is sure of keeps its digits).
struct LogSumOut {
    static constexpr bool kLogSum = true;
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

// What a row of logits' gradients needs: {lse, weight over the largest weight, label's bits, 0}.
// The gradient g = weight (exp(l - lse) - [the label]) in bf16; columns past the end up to a
// whole block are zero.
struct GradOut {
    static constexpr bool kLogSum = false;
    const f32x4* info;
    uint16_t* g;
    int64_t ldg, col0;  // first column of the piece in the vocabulary
    __device__ void begin() {}
    __device__ __forceinline__ void operator()(int64_t row, int64_t col, float (&v)[8], int64_t n) const {
        const f32x4 r = reinterpret_cast<const gf32x4*>(gp(info))[row];
        const float label = r[2];  // a bit cast of an element of a vector would take its first
        const int64_t hit = (int64_t)__builtin_bit_cast(int32_t, label) - col0 - col;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = exp_fast(v[i] - r[0]);
            v[i] = i < n ? r[1] * (i == hit ? p - 1.0f : p) : 0.0f;
        }
        store8<true>(g + row * ldg + col, 8, v);
    }
};

// ------------------------------------------------------------------ the product
//
// sum over k of A(i, k) B(j, k), A m x k and B n x k in bf16. An operand's memory has
// rows of k (k runs along a row), or of i (k is the row: "tall").

struct Product16 {
    const uint16_t *a, *b;
    int64_t lda, ldb;       // elements from row to row of memory
    const int32_t* a_rows;  // row i of A is row a_rows[i] of memory; NULL: row i (not with a tall A)
    const int32_t* m_at;    // in device memory: the rows of A that exist, at most m; NULL: m
    const int32_t* k_at;    // the same of k
    int64_t m, n, k;
};

__device__ __forceinline__ f32x16 mfma16(const u32x4& b, const u32x4& a, const f32x16& acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
}

// One matrix instruction takes 32 rows of each operand over 16 values of k: lane l
// holds the 8 values k = 8 (l / 32) .. of row l % 32. B is the first operand, so that
// a lane's four consecutive accumulators are four consecutive columns: accumulator r
// of lane l is row l % 32, column 8 (r / 4) + 4 (l / 32) + r % 4.
//
// The plain product, straight from global memory: each wavefront a 32 x 32 tile, a
// workgroup 64 x 64; any strides and alignments.
template <bool TALL_A, bool TALL_B, class Out>
__global__ __launch_bounds__(kBlock) void product_plain_kernel(Product16 p, uint32_t tiles_n, Out out) {
    __shared__ float lds[kWavesPerBlock][32][33];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t tile = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t m = p.m_at ? (int64_t)*gp(p.m_at) : p.m, k = p.k_at ? (int64_t)*gp(p.k_at) : p.k;
    const int64_t n0 = tile % tiles_n * 64 + (wave & 1) * 32, m0 = tile / tiles_n * 64 + (wave >> 1) * 32;
    if (m0 >= m || n0 >= p.n) return;
    out.begin();
    const int row = lane & 31, half = lane >> 5;
    // rows past the end are read as the last one and not used
    const int64_t ra = m0 + row < m ? m0 + row : m - 1, rb = n0 + row < p.n ? n0 + row : p.n - 1;
    const int64_t ma = p.a_rows ? (int64_t)gp(p.a_rows)[ra] : ra;
    const uint16_t* const pa = p.a + (TALL_A ? ra : ma * p.lda);
    const uint16_t* const pb = p.b + (TALL_B ? rb : rb * p.ldb);
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int64_t k0 = 0; k0 < k; k0 += 16) {
        u32x4 a{0u, 0u, 0u, 0u}, b{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = k0 + half * 8 + e;
            if (at < k) {
                a[e / 2] |= (uint32_t)gp(pa)[TALL_A ? at * p.lda : at] << (16 * (e & 1));
                b[e / 2] |= (uint32_t)gp(pb)[TALL_B ? at * p.ldb : at] << (16 * (e & 1));
            }
        }
        acc = mfma16(b, a, acc);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) lds[wave][row][8 * (r / 4) + 4 * half + r % 4] = acc[r];
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if constexpr (Out::kLogSum) {
        static_assert(kLseWidth == 32);
        if (lane < 32 && m0 + lane < m) {
            const int64_t label = out.label_of(m0 + lane) - n0;
            const int cols = (int)(p.n - n0 < 32 ? p.n - n0 : 32);
            float top = -__builtin_inff(), sum = 0.0f;
            for (int c = 0; c < cols; ++c)
                if (c == label) out.keep(m0 + lane, lds[wave][lane][c]);
                else top = fmaxf(top, lds[wave][lane][c]);
            const float from = top == -__builtin_inff() ? 0.0f : top;
            for (int c = 0; c < cols; ++c)
                if (c != label) sum += exp_fast(lds[wave][lane][c] - from);
            out.put(m0 + lane, n0 / 32, from, sum);
        }
    } else {
        for (int i = lane; i < 32 * 4; i += kWave) {
            const int r = i / 4, c = i % 4 * 8;
            if (m0 + r >= m || n0 + c >= p.n) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = lds[wave][r][c + e];
            out(m0 + r, n0 + c, v, p.n - n0 - c);
        }
    }
}

template <bool TALL_A, bool TALL_B, class Out>
int launch_product(const Product16& p, const Out& out, hipStream_t st) {
    if (p.m == 0 || p.n == 0) return COAT_OK;
    const int64_t tn = div_up(p.n, 64), tiles = tn * div_up(p.m, 64);
    if (tiles > 0x7FFFFFFFll * 64) return COAT_EINVAL;
    const Grid g = grid_xy(tiles, kBlock);
    hipLaunchKernelGGL((product_plain_kernel<TALL_A, TALL_B, Out>), dim3(g.x, g.y), dim3(kBlock), 0, st, p, (uint32_t)tn, out);
    return launch_status();
}

}  // namespace

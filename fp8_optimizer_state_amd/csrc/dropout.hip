// HIP (gfx950) dropout without a stored mask.
#include <type_traits>

#include "train_common.h"

namespace {

// y = residual + scale D(x). Bound by HBM: 16384 x 5120 in bf16 with a residual takes 90 us
// (5.6 TB/s), 8191 x 2731 from fp32 25 us. A thread takes blocks of 8 columns of a row,
// whose random bits are one call of the generator: 16 bits an element, since 32 would make
// the generator's 20 wide products twice the work and p needs no finer steps. y may be x or
// residual: each thread has read its 8 columns before it writes them.
template <class X, class T, bool DROP>
__global__ __launch_bounds__(kBlock) void dropout_kernel(const X* x, int64_t ldx, const T* residual, int64_t ldr,
                                                         float scale, Drop drop, T* y, int64_t ldy, int64_t rows, int64_t cols) {
    drop.begin();
    const int64_t blocks = (cols + 7) / 8, total = rows * blocks;
    for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < total; i += (int64_t)gridDim.x * kBlock) {
        const int64_t row = i / blocks, col = (i - row * blocks) * 8, n = cols - col;
        float v[8], r[8];
        expand(load_raw8(x + row * ldx + col, n), v);
        if constexpr (DROP) drop((uint64_t)i, v);
        if (residual) {
            expand(load_raw8(residual + row * ldr + col, n), r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], scale, r[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= scale;
        }
        store8(y + row * ldy + col, n, v);
    }
}

template <class X, class T>
int launch_dropout(const X* x, int64_t rows, int64_t cols, int64_t ldx, const T* residual, int64_t ldr, float scale, const Drop& drop,
                   T* y, int64_t ldy, hipStream_t st) {
    const int64_t groups = div_up(rows * div_up(cols, 8), kBlock);
    const dim3 grid((unsigned)(groups < 64 * kCUs ? groups : 64 * kCUs));
    if (drop.threshold)
        hipLaunchKernelGGL((dropout_kernel<X, T, true>), grid, dim3(kBlock), 0, st, x, ldx, residual, ldr, scale, drop, y, ldy, rows, cols);
    else
        hipLaunchKernelGGL((dropout_kernel<X, T, false>), grid, dim3(kBlock), 0, st, x, ldx, residual, ldr, scale, drop, y, ldy, rows, cols);
    return launch_status();
}

}  // namespace

extern "C" {

int coat_dropout(const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t x_type, const void* residual, int64_t ldr,
                 float scale, float p, const int64_t* rng, int64_t offset, void* y, int64_t ldy, int32_t y_type,
                 coat_stream_t stream) {
    const int rc = check_dropout(x, rows, cols, ldx, x_type, residual, ldr, scale, p, rng, y, ldy, y_type);
    if (rc || rows == 0 || cols == 0) return rc;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const uint32_t t = drop_threshold(p);
    const Drop drop{rng, offset, t, 0, 0};
    const float s = scale * drop_factor(t);
    if (x_type == COAT_FP32) {
        const float* const xf = static_cast<const float*>(x);
        if (y_type == COAT_FP32)
            return launch_dropout(xf, rows, cols, ldx, static_cast<const float*>(residual), ldr, s, drop, static_cast<float*>(y), ldy, st);
        return launch_dropout(xf, rows, cols, ldx, static_cast<const uint16_t*>(residual), ldr, s, drop, static_cast<uint16_t*>(y), ldy, st);
    }
    const uint16_t* const xh = static_cast<const uint16_t*>(x);
    if (y_type == COAT_FP32)
        return launch_dropout(xh, rows, cols, ldx, static_cast<const float*>(residual), ldr, s, drop, static_cast<float*>(y), ldy, st);
    return launch_dropout(xh, rows, cols, ldx, static_cast<const uint16_t*>(residual), ldr, s, drop, static_cast<uint16_t*>(y), ldy, st);
}

}  // extern "C"

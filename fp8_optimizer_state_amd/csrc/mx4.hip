// HIP (gfx950) codec of microscaled 4-bit floating point: bf16 or fp32 matrices
// to E2M1 codes with one power-of-two scale byte per 32 values, along the rows,
// the columns or both, and back.
#include "mx4_common.h"

namespace {

// ------------------------------------------------------------------ along the rows
//
// A wavefront takes a segment of 2048 values of a row, 8 consecutive ones per
// lane and step, so that each load covers consecutive bytes; a block of 32 is
// four lanes. The segments reach over the end of the row to the end of its
// scale bytes (a multiple of 512 values): the lanes behind the data write the
// zeros that the layout asks for.
constexpr int kSeg = 4 * 8 * kWave;

template <class T>
__global__ __launch_bounds__(kBlock) void mx4_quantize_rows_kernel(const T* __restrict__ x, uint32_t items,
                                                                   uint32_t segs, int64_t cols, int64_t ld,
                                                                   uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t nw = gridDim.x * kWavesPerBlock;
    const int64_t qb = mx4_code_bytes(cols), sb = mx4_scale_bytes(cols);
    for (uint64_t it = (uint64_t)wave_id(); it < items; it += nw) {
        const uint32_t row = (uint32_t)it / segs, seg = (uint32_t)it - row * segs;
        const T* xr = x + (int64_t)row * ld;
        uint8_t* qr = q + (int64_t)row * qb;
        uint8_t* sr = s + (int64_t)row * sb;
        const int64_t c0 = (int64_t)seg * kSeg + lane * 8;
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) load8(xr + c0 + i * 8 * kWave, cols - (c0 + i * 8 * kWave), v[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * 8 * kWave;
            uint32_t am = absmax_bits(v[i]);
            uint32_t o = xlane32(am, 1);
            am = am > o ? am : o;
            o = xlane32(am, 2);
            am = am > o ? am : o;
            const uint32_t b = mx4_scale_byte(am);
            const uint32_t code = b == 255u ? 0u : mx4_codes8(v[i], b);
            if (c / 2 < qb) *reinterpret_cast<gu32*>(gp(qr) + c / 2) = code;
            if ((lane & 3) == 0 && c / 32 < sb) gp(sr)[c / 32] = (uint8_t)b;
        }
    }
}

template <class T>
__global__ __launch_bounds__(kBlock) void mx4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                                const uint8_t* __restrict__ s, uint32_t items,
                                                                uint32_t segs, int64_t cols, T* __restrict__ x,
                                                                int64_t ld) {
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t nw = gridDim.x * kWavesPerBlock;
    const int64_t qb = mx4_code_bytes(cols), sb = mx4_scale_bytes(cols);
    for (uint64_t it = (uint64_t)wave_id(); it < items; it += nw) {
        const uint32_t row = (uint32_t)it / segs, seg = (uint32_t)it - row * segs;
        T* xr = x + (int64_t)row * ld;
        const uint8_t* qr = q + (int64_t)row * qb;
        const uint8_t* sr = s + (int64_t)row * sb;
        const int64_t c0 = (int64_t)seg * kSeg + lane * 8;
        uint32_t code[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * 8 * kWave;
            code[i] = c < cols ? *reinterpret_cast<const gu32*>(gp(qr) + c / 2) : 0u;
            b[i] = c < cols ? gp(sr)[c / 32] : 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * 8 * kWave;
            float v[8];
            mx4_values8(code[i], b[i], v);
            if (c < cols) store8(xr + c, cols - c, v);
        }
    }
}

// ------------------------------------------------------------------ along the columns, or both
//
// A workgroup takes a tile of 128 x 128 values: it is read once, row by row,
// into LDS (and quantized along the rows on the way where that is asked for);
// then each thread quantizes blocks of 32 values down a column.
constexpr int kTileRows = 128, kTileCols = 128;

__device__ __forceinline__ void to_lds8(uint16_t* p, const float (&v)[8]) {
    // bf16 values read from bf16: the upper halves are the values
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (__builtin_bit_cast(uint32_t, v[2 * i]) >> 16) | (__builtin_bit_cast(uint32_t, v[2 * i + 1]) & 0xFFFF0000u);
    *reinterpret_cast<u32x4*>(p) = w;
}
__device__ __forceinline__ void to_lds8(float* p, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[i];
}
__device__ __forceinline__ float from_lds(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }
__device__ __forceinline__ float from_lds(float f) { return f; }

template <class T, bool ROWS>
__global__ __launch_bounds__(kBlock) void mx4_quantize_tile_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                                   int64_t ld, uint32_t tiles_r,
                                                                   uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                                                                   uint8_t* __restrict__ qt, uint8_t* __restrict__ st) {
    __shared__ __attribute__((aligned(16))) T tile[kTileRows][kTileCols];
    const int64_t r0 = (int64_t)(blockIdx.x % tiles_r) * kTileRows, c0 = (int64_t)(blockIdx.x / tiles_r) * kTileCols;
    const int tid = threadIdx.x;
    const int64_t qb = mx4_code_bytes(cols), sb = mx4_scale_bytes(cols);
    const int64_t qtb = mx4_code_bytes(rows), stb = mx4_scale_bytes(rows);
#pragma unroll 4
    for (int i = 0; i < kTileRows * kTileCols / 8 / kBlock; ++i) {
        const int lr = i * (kBlock * 8 / kTileCols) + tid / (kTileCols / 8), lc = (tid % (kTileCols / 8)) * 8;
        const int64_t r = r0 + lr, c = c0 + lc;
        float v[8];
        load8(x + r * ld + c, r < rows ? cols - c : 0, v);
        to_lds8(&tile[lr][lc], v);
        if (ROWS) {
            uint32_t am = absmax_bits(v);
            uint32_t o = xlane32(am, 1);
            am = am > o ? am : o;
            o = xlane32(am, 2);
            am = am > o ? am : o;
            const uint32_t b = mx4_scale_byte(am);
            const uint32_t code = b == 255u ? 0u : mx4_codes8(v, b);
            if (r < rows && c / 2 < qb) *reinterpret_cast<gu32*>(gp(q) + r * qb + c / 2) = code;
            if ((tid & 3) == 0 && r < rows && c / 32 < sb) gp(s)[r * sb + c / 32] = (uint8_t)b;
        }
    }
    __syncthreads();
    for (int i = tid; i < kTileCols * (kTileRows / 32); i += kBlock) {
        const int lc = i % kTileCols, rb = i / kTileCols;
        const int64_t c = c0 + lc, r = r0 + rb * 32;
        if (c >= cols) continue;
        float v[4][8];
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[j][k] = from_lds(tile[rb * 32 + j * 8 + k][lc]);
            const uint32_t a = absmax_bits(v[j]);
            am = am > a ? am : a;
        }
        const uint32_t b = mx4_scale_byte(am);
        u32x4 code{0u, 0u, 0u, 0u};
        if (b != 255u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) code[j] = mx4_codes8(v[j], b);
        }
        if (r / 2 < qtb) *reinterpret_cast<gu32x4*>(gp(qt) + c * qtb + r / 2) = code;
        if (r / 32 < stb) gp(st)[c * stb + r / 32] = (uint8_t)b;
    }
}

template <class T>
int launch_quantize(const T* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* q, uint8_t* s, uint8_t* qt,
                    uint8_t* st, hipStream_t stream) {
    if (!qt) {
        const int64_t segs = div_up(32 * mx4_scale_bytes(cols), kSeg);  // 32 values a scale byte
        const int64_t items = rows * segs;
        if (items > 0xFFFFFFFFll) return COAT_EINVAL;
        hipLaunchKernelGGL(mx4_quantize_rows_kernel<T>, dim3(grid_for(items, 128)), dim3(kBlock), 0, stream, x,
                           (uint32_t)items, (uint32_t)segs, cols, ld, q, s);
        return launch_status();
    }
    // the tiles reach to the end of the scale bytes of either direction
    const int64_t tr = div_up(32 * mx4_scale_bytes(rows), kTileRows), tc = div_up(32 * mx4_scale_bytes(cols), kTileCols);
    if (tr * tc > 0x7FFFFFFFll) return COAT_EINVAL;
    if (q)
        hipLaunchKernelGGL((mx4_quantize_tile_kernel<T, true>), dim3((unsigned)(tr * tc)), dim3(kBlock), 0, stream, x,
                           rows, cols, ld, (uint32_t)tr, q, s, qt, st);
    else
        hipLaunchKernelGGL((mx4_quantize_tile_kernel<T, false>), dim3((unsigned)(tr * tc)), dim3(kBlock), 0, stream, x,
                           rows, cols, ld, (uint32_t)tr, q, s, qt, st);
    return launch_status();
}

}  // namespace

// ====================================================================== C ABI

extern "C" {

int64_t coat_mx4_code_bytes(int64_t k) { return k > 0 ? mx4_code_bytes(k) : 0; }
int64_t coat_mx4_scale_bytes(int64_t k) { return k > 0 ? mx4_scale_bytes(k) : 0; }

int coat_mx4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, uint8_t* q, uint8_t* s,
                      uint8_t* q_t, uint8_t* s_t, coat_stream_t stream) {
    const int rc = check_mx4_quantize(x, rows, cols, ld, dtype, q, s, q_t, s_t);
    if (rc || rows == 0 || cols == 0) return rc;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (dtype == COAT_FP32)
        return launch_quantize(static_cast<const float*>(x), rows, cols, ld, q, s, q_t, s_t, st);
    return launch_quantize(static_cast<const uint16_t*>(x), rows, cols, ld, q, s, q_t, s_t, st);
}

int coat_mx4_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, void* x, int64_t ld,
                        int32_t dtype, coat_stream_t stream) {
    const int rc = check_mx4_dequantize(q, s, rows, cols, x, ld, dtype);
    if (rc || rows == 0 || cols == 0) return rc;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const int64_t segs = div_up(cols, kSeg), items = rows * segs;
    if (items > 0xFFFFFFFFll) return COAT_EINVAL;
    const unsigned grid = grid_for(items, 128);
    if (dtype == COAT_FP32)
        hipLaunchKernelGGL(mx4_dequantize_kernel<float>, dim3(grid), dim3(kBlock), 0, st, q, s, (uint32_t)items,
                           (uint32_t)segs, cols, static_cast<float*>(x), ld);
    else
        hipLaunchKernelGGL(mx4_dequantize_kernel<uint16_t>, dim3(grid), dim3(kBlock), 0, st, q, s, (uint32_t)items,
                           (uint32_t)segs, cols, static_cast<uint16_t*>(x), ld);
    return launch_status();
}

}  // extern "C"

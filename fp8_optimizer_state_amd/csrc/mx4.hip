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
// zeros that the layout asks for. Bound by HBM: 16384 x 13824 in bf16 take 105 us
// to quantize (5.5 TB/s) and 101 us back (5.7); 13824 x 5120 take 40 us back to bf16 and
// 66 to fp32 (4.5 and 4.9 TB/s), 27 and 55 where the caches hold the codes.
// A block's maximum is taken over the magnitudes' bits, which order like the
// values, a NaN or infinity above all; the converter rounds to nearest even and
// saturates.
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
        Raw8<T> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_raw8(xr + c0 + i * 8 * kWave, cols - (c0 + i * 8 * kWave));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * 8 * kWave;
            const uint32_t b = mx4_scale_byte(block_max(absmax_bits(v[i])));
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
        // a lane's values of a step fill 16 bytes, so that a store covers consecutive bytes
        constexpr int kPer = 16 / sizeof(T), kSteps = kSeg / kPer / kWave;
        const int64_t c0 = (int64_t)seg * kSeg + lane * kPer;
        uint32_t code[kSteps], b[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t c = c0 + i * kPer * kWave;
            code[i] = b[i] = 0u;
            if (c < cols) {
                if constexpr (kPer == 8) code[i] = *reinterpret_cast<const gu32*>(gp(qr) + c / 2);
                else code[i] = *reinterpret_cast<const gu16*>(gp(qr) + c / 2);
                b[i] = gp(sr)[c / 32];
            }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t c = c0 + i * kPer * kWave;
            float v[kPer];
#pragma unroll
            for (int j = 0; j < kPer; j += 4) {
                float w[4];
                mx4_values4(code[i] >> (4 * j), b[i], w);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[j + k] = w[k];
            }
            if (c < cols) store16(xr + c, cols - c, v);
        }
    }
}

// ------------------------------------------------------------------ along the columns, or both
//
// A workgroup takes a tile of 128 x 128 values: it is read once, row by row,
// into LDS (and quantized along the rows on the way where that is asked for);
// then each thread quantizes blocks of 32 values down a column. Bound by HBM, at a
// lower rate than the rows alone, since the codes leave in runs of 64 bytes a row
// and a column: 16384 x 13824 in bf16 take 163 us both ways (4.3 TB/s), 129 along
// the columns (4.4). Square tiles of 128, because a column's four blocks are then
// a whole run, and five workgroups of bf16 values share a compute unit's LDS.
constexpr int kTileRows = 128, kTileCols = 128;

// Where a block of 32 values down column c goes.
struct Down {
    uint8_t *q, *s;
    int64_t qb, sb, cols;
    __device__ __forceinline__ void put(int64_t r, int64_t c, uint32_t b, const u32x4& code) const {
        if (c >= cols) return;
        if (r / 2 < qb) *reinterpret_cast<gu32x4*>(gp(q) + c * qb + r / 2) = b == 255u ? u32x4{0u, 0u, 0u, 0u} : code;
        if (r / 32 < sb) gp(s)[c * sb + r / 32] = (uint8_t)b;
    }
};

// Quantizes the blocks of a tile in LDS down its columns. Four consecutive lanes
// take the four blocks of a column, so that they store 64 consecutive bytes; to
// spread them over the banks, chunk c (16 bytes) of row r lies at position
// c ^ (4 (r / 32)). bf16: a thread takes two columns, whole words.
template <class T>
__device__ __forceinline__ int tile_col(int r, int c) {
    constexpr int kChunk = 16 / sizeof(T);
    return c ^ (r / 32 * 4 * kChunk);
}
__device__ __forceinline__ void to_lds8(uint16_t* row, int r, int c, const Raw8<uint16_t>& v) {
    *reinterpret_cast<u32x4*>(row + tile_col<uint16_t>(r, c)) = v.w;
}
__device__ __forceinline__ void to_lds8(float* row, int r, int c, const Raw8<float>& v) {
    *reinterpret_cast<u32x4*>(row + tile_col<float>(r, c)) = v.lo;
    *reinterpret_cast<u32x4*>(row + tile_col<float>(r, c + 4)) = v.hi;
}
__device__ __forceinline__ void quantize_down(const uint16_t (&tile)[kTileRows][kTileCols], int64_t r0, int64_t c0, const Down& to) {
    for (int i = threadIdx.x; i < kTileCols / 2 * (kTileRows / 32); i += kBlock) {
        const int lc = i / 4 * 2, lr = i % 4 * 32;
        uint32_t w[32], m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            w[j] = *reinterpret_cast<const uint32_t*>(&tile[lr + j][tile_col<uint16_t>(lr, lc)]);
            m = bf16_max2(m, w[j]);
        }
        const uint32_t b0 = mx4_scale_byte(m << 16), b1 = mx4_scale_byte(m & 0xFFFF0000u);
        u32x4 q0, q1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Raw8<uint16_t> x0, x1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t even = w[8 * j + 2 * k], odd = w[8 * j + 2 * k + 1];
                x0.w[k] = __builtin_amdgcn_perm(odd, even, 0x05040100u);
                x1.w[k] = __builtin_amdgcn_perm(odd, even, 0x07060302u);
            }
            q0[j] = mx4_codes8(x0, b0);
            q1[j] = mx4_codes8(x1, b1);
        }
        to.put(r0 + lr, c0 + lc, b0, q0);
        to.put(r0 + lr, c0 + lc + 1, b1, q1);
    }
}
__device__ __forceinline__ void quantize_down(const float (&tile)[kTileRows][kTileCols], int64_t r0, int64_t c0, const Down& to) {
    for (int i = threadIdx.x; i < kTileCols * (kTileRows / 32); i += kBlock) {
        const int lc = i / 4, lr = i % 4 * 32, at = tile_col<float>(lr, lc);
        Raw8<float> x[4];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[j].lo[k] = __builtin_bit_cast(uint32_t, tile[lr + 8 * j + k][at]);
                x[j].hi[k] = __builtin_bit_cast(uint32_t, tile[lr + 8 * j + 4 + k][at]);
            }
            m = umax(m, absmax_bits(x[j]));
        }
        const uint32_t b = mx4_scale_byte(m);
        to.put(r0 + lr, c0 + lc, b, u32x4{mx4_codes8(x[0], b), mx4_codes8(x[1], b), mx4_codes8(x[2], b), mx4_codes8(x[3], b)});
    }
}

template <class T, bool ROWS>
__global__ __launch_bounds__(kBlock) void mx4_quantize_tile_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                                   int64_t ld, uint32_t tiles_r, uint32_t tiles,
                                                                   uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                                                                   uint8_t* __restrict__ qt, uint8_t* __restrict__ st) {
    __shared__ __attribute__((aligned(16))) T tile[kTileRows][kTileCols];
    // Neighbouring tiles write parts of the same lines of codes and scale bytes
    // (64 bytes and 4 a tile), so patches of 4 x 4 tiles are taken one after the
    // other on one XCD: consecutive workgroups run on different XCDs.
    uint32_t t = blockIdx.x;
    if (gridDim.x % 8 == 0) t = (t & 7) * (gridDim.x / 8) + (t >> 3);
    t += blockIdx.y * gridDim.x;
    if (t >= tiles) return;
    const uint32_t patch = t / 16, patches_r = tiles_r / 4;
    const int64_t r0 = (int64_t)(patch % patches_r * 4 + t % 4) * kTileRows;
    const int64_t c0 = (int64_t)(patch / patches_r * 4 + t / 4 % 4) * kTileCols;
    const int tid = threadIdx.x;
    const int64_t qb = mx4_code_bytes(cols), sb = mx4_scale_bytes(cols);
#pragma unroll 4
    for (int i = 0; i < kTileRows * kTileCols / 8 / kBlock; ++i) {
        const int lr = i * (kBlock * 8 / kTileCols) + tid / (kTileCols / 8), lc = (tid % (kTileCols / 8)) * 8;
        const int64_t r = r0 + lr, c = c0 + lc;
        const Raw8<T> v = load_raw8(x + r * ld + c, r < rows ? cols - c : 0);
        to_lds8(tile[lr], lr, lc, v);
        if (ROWS) {
            const uint32_t b = mx4_scale_byte(block_max(absmax_bits(v)));
            const uint32_t code = b == 255u ? 0u : mx4_codes8(v, b);
            if (r < rows && c / 2 < qb) *reinterpret_cast<gu32*>(gp(q) + r * qb + c / 2) = code;
            if ((tid & 3) == 0 && r < rows && c / 32 < sb) gp(s)[r * sb + c / 32] = (uint8_t)b;
        }
    }
    __syncthreads();
    quantize_down(tile, r0, c0, Down{qt, st, mx4_code_bytes(rows), mx4_scale_bytes(rows), cols});
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
    // the tiles reach to the end of the scale bytes of either direction: four of them, 512 values
    const int64_t tr = div_up(32 * mx4_scale_bytes(rows), kTileRows), tc = div_up(32 * mx4_scale_bytes(cols), kTileCols);
    if (tr * tc > 0x7FFFFFFFll) return COAT_EINVAL;
    const Grid g = grid_xy(tr * tc, kBlock);
    if (q)
        hipLaunchKernelGGL((mx4_quantize_tile_kernel<T, true>), dim3(g.x, g.y), dim3(kBlock), 0, stream, x, rows, cols, ld,
                           (uint32_t)tr, (uint32_t)(tr * tc), q, s, qt, st);
    else
        hipLaunchKernelGGL((mx4_quantize_tile_kernel<T, false>), dim3(g.x, g.y), dim3(kBlock), 0, stream, x, rows, cols, ld,
                           (uint32_t)tr, (uint32_t)(tr * tc), q, s, qt, st);
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

// HIP (gfx950) product of two matrices in microscaled 4-bit floating point.
#include "mx4_common.h"

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// One matrix instruction takes 32 rows of each operand over 64 values of k: lane
// l holds the 32 codes of row l % 32 in block l / 32, and their scale byte.
// Two of them take a row's 64 code bytes and 4 scale bytes: chunk l / 32 and
// scale byte l / 32 first, then chunk 2 + l / 32 and scale byte 2 + l / 32; the
// scale word is shifted by l / 32 bytes once, and the instruction selects its
// byte 0 or 2. B is the first operand, so that a lane's four consecutive
// accumulators are four consecutive columns of y: accumulator r of lane l is
// y[l % 32][8 (r / 4) + 4 (l / 32) + r % 4].
template <int SEL>
__device__ __forceinline__ f32x16 mfma_fp4(const u32x4& b, const u32x4& a, const f32x16& acc, uint32_t sb, uint32_t sa) {
    const i32x8 vb{(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const i32x8 va{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, acc, 4, 4, SEL, (int)sb, SEL, (int)sa);
}

// Small tiles, straight from global memory: each wavefront a 32 x 32 tile, a
// workgroup 64 x 64. Rows past the end are read as the last row and not stored.
template <class T>
__global__ __launch_bounds__(kBlock) void mx4_matmul_small_kernel(const uint8_t* __restrict__ aq,
                                                                  const uint8_t* __restrict__ as, int64_t m,
                                                                  const uint8_t* __restrict__ bq,
                                                                  const uint8_t* __restrict__ bs, int64_t n, int64_t k,
                                                                  uint32_t tiles_n, T* __restrict__ y, int64_t ld) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * 64 + (wave & 1) * 32;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * 64 + (wave >> 1) * 32;
    const int row = lane & 31, half = lane >> 5;
    const int64_t qb = mx4_code_bytes(k), sb = mx4_scale_bytes(k);
    const int64_t ra = m0 + row < m ? m0 + row : m - 1, rb = n0 + row < n ? n0 + row : n - 1;
    const uint8_t *pa = aq + ra * qb + half * 16, *pb = bq + rb * qb + half * 16;
    const uint8_t *psa = as + ra * sb, *psb = bs + rb * sb;
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    const int64_t steps = div_up(k, 128);
    for (int64_t t = 0; t < steps; ++t) {
        const u32x4 a0 = *reinterpret_cast<const gu32x4*>(gp(pa) + t * 64);
        const u32x4 a1 = *reinterpret_cast<const gu32x4*>(gp(pa) + t * 64 + 32);
        const u32x4 b0 = *reinterpret_cast<const gu32x4*>(gp(pb) + t * 64);
        const u32x4 b1 = *reinterpret_cast<const gu32x4*>(gp(pb) + t * 64 + 32);
        const uint32_t sa = *reinterpret_cast<const gu32*>(gp(psa) + t * 4) >> (8 * half);
        const uint32_t sbw = *reinterpret_cast<const gu32*>(gp(psb) + t * 4) >> (8 * half);
        acc = mfma_fp4<0>(b0, a0, acc, sbw, sa);
        acc = mfma_fp4<2>(b1, a1, acc, sbw, sa);
    }
    if (m0 + row >= m) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t c = n0 + 8 * (r / 4) + 4 * half + r % 4;
        if (c < n) {
            if constexpr (sizeof(T) == 4) gp(y)[(m0 + row) * ld + c] = acc[r];
            else gp(y)[(m0 + row) * ld + c] = (uint16_t)bf16_bits(acc[r]);
        }
    }
}

template <class T>
int launch_matmul(const uint8_t* aq, const uint8_t* as, int64_t m, const uint8_t* bq, const uint8_t* bs, int64_t n,
                  int64_t k, T* y, int64_t ld, hipStream_t st) {
    const int64_t tn = div_up(n, 64), tiles = tn * div_up(m, 64);
    if (tiles > 0x7FFFFFFFll) return COAT_EINVAL;
    hipLaunchKernelGGL(mx4_matmul_small_kernel<T>, dim3((unsigned)tiles), dim3(kBlock), 0, st, aq, as, m, bq, bs, n, k,
                       (uint32_t)tn, y, ld);
    return launch_status();
}

}  // namespace

extern "C" {

size_t coat_mx4_matmul_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

int coat_mx4_matmul(const uint8_t* a_q, const uint8_t* a_s, int64_t m, const uint8_t* b_q, const uint8_t* b_s,
                    int64_t n, int64_t k, void* y, int64_t ld, int32_t dtype, void* workspace, size_t workspace_bytes,
                    coat_stream_t stream) {
    const int rc = check_mx4_matmul(a_q, a_s, m, b_q, b_s, n, k, y, ld, dtype);
    if (rc || m == 0 || n == 0) return rc;
    (void)workspace;
    (void)workspace_bytes;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (dtype == COAT_FP32)
        return launch_matmul(a_q, a_s, m, b_q, b_s, n, k, static_cast<float*>(y), ld, st);
    return launch_matmul(a_q, a_s, m, b_q, b_s, n, k, static_cast<uint16_t*>(y), ld, st);
}

}  // extern "C"

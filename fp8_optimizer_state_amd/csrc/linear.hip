// HIP (gfx950) linear layer with its epilogue, and its backward pass.
#include "bf16_product.h"

namespace {

// ------------------------------------------------------------------ the gradient before the activation
//
// dz = D(dy) act'(z) in bf16 (the matrix units' type, and the one rounding on the way to dx
// and dw, unless few values take a second term), without the factors that the products' sums
// are multiplied by, and the sums of a band of rows of it as they were before the rounding.
// A workgroup takes 512 columns of a band: a thread 8 columns of every fourth row, the four
// rows' sums joined through LDS in order. Bound by HBM: 8192 x 13824 in bf16 takes 132 us (5.1 TB/s).
template <class T>
__global__ __launch_bounds__(kBlock) void dz_kernel(const T* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ z, int64_t ldz,
                                                    int32_t act, Drop drop, int64_t m, int64_t n, uint16_t* __restrict__ dz,
                                                    int64_t ld_dz, float* __restrict__ bias_part, int32_t band, bool two) {
    __shared__ float sums[kWavesPerBlock][kWave][9];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    drop.begin();
    const int64_t col = ((int64_t)blockIdx.x * kWave + lane) * 8, left = n - col, blocks = (n + 7) / 8;
    const int64_t r0 = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * band;
    if (r0 >= m) return;
    const int64_t r1 = r0 + band < m ? r0 + band : m;
    float sum[8] = {};
    if (left > 0) {
        for (int64_t row = r0 + wave; row < r1; row += kWavesPerBlock) {
            float v[8];
            expand(load_raw8(dy + row * lddy + col, left), v);
            if (drop.threshold) drop((uint64_t)(row * blocks + col / 8), v);
            if (act != COAT_ACT_NONE) {
                float zv[8];
                expand(load_raw8(z + row * ldz + col, left), zv);
                with_act(act, [&](auto a) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float s = slope<a.value>(zv[i]);
                        // a dropped place stays zero whatever z holds there
                        v[i] = v[i] == 0.0f ? 0.0f : v[i] * s;
                    }
                });
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= left) v[i] = 0.0f;
                sum[i] += v[i];
            }
            if (dz) store8<true>(dz + row * ld_dz + col, 8, v);
            if (dz && two) {  // what the rounding leaves, behind the m rows
                left_of(v);
                store8<true>(dz + (m + row) * ld_dz + col, 8, v);
            }
        }
    }
    if (!bias_part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[wave][lane][i] = sum[i];
    __syncthreads();
    if (wave == 0 && left > 0) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (sums[0][lane][i] + sums[1][lane][i]) + (sums[2][lane][i] + sums[3][lane][i]);
        store8<true>(bias_part + r0 / band * ld_dz + col, 8, v);
    }
}

// dbias = scale times the parts' sums: a workgroup takes 64 columns, its wavefronts every
// fourth part.
template <class T>
__global__ __launch_bounds__(kBlock) void bias_join_kernel(const float* __restrict__ part, int64_t ld, int64_t parts, int64_t n,
                                                           float scale, T* __restrict__ dbias) {
    __shared__ float sums[kWavesPerBlock][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t col = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWave + lane;
    float sum = 0.0f;
    if (col < n) {
#pragma unroll 8
        for (int64_t i = wave; i < parts; i += kWavesPerBlock) sum += gp(part)[i * ld + col];
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || col >= n) return;
    sum = ((sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane])) * scale;
    if constexpr (sizeof(T) == 4) gp(dbias)[col] = sum;
    else gp(dbias)[col] = (uint16_t)bf16_bits(sum);
}

template <class T>
int launch_dz(const T* dy, int64_t lddy, const uint16_t* z, int64_t ldz, int32_t act, const Drop& drop, int64_t m, int64_t n, uint16_t* dz,
              int64_t ld_dz, float* part, bool two, hipStream_t st) {
    const int64_t band = bias_band(m, n), bands = div_up(m, band), most = 32768;
    const dim3 grid((unsigned)div_up(n, kWave * 8), (unsigned)(bands < most ? bands : most), (unsigned)div_up(bands, most));
    hipLaunchKernelGGL(dz_kernel<T>, grid, dim3(kBlock), 0, st, dy, lddy, z, ldz, act, drop, m, n, dz, ld_dz, part,
                       (int32_t)band, two);
    return launch_status();
}

template <class T>
int launch_linear(const Product16& p, const Plan16& plan, float* ws, const coat_epilogue* e, const void* bias, int32_t bias_type, const void* residual, int64_t ldr,
                  uint16_t* z, int64_t ldz, void* y, int64_t ldy, hipStream_t st) {
    const uint32_t t = drop_threshold(e->p);
    // Large outputs of whole lines in bf16: 16384 x 13824 x 5120 with z 1870 -> 1743..1784 us, by
    // box. Small ones stay in the caches for who reads them next.
    auto past = [&](const void* to, int64_t ld) { return aligned(to, 128) && ld % 64 == 0 && p.m * p.n >= (int64_t(1) << 25); };
    const LinearOut<T> out{bias, static_cast<const T*>(residual), z, static_cast<T*>(y), ldr, ldz, ldy, div_up(p.n, 8),
                           Drop{e->rng, e->offset, t, 0, 0}, e->scale * drop_factor(t), e->act, bias_type, past(y, ldy), past(z, ldz)};
    return launch_product<false, false>(p, plan, ws, out, st);
}

}  // namespace

extern "C" {

size_t coat_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t aligned) {
    if (m < 1 || n < 1 || k < 1 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
    return linear_layout(m, n, k, aligned != 0).end;
}

int coat_linear(const uint16_t* x, int64_t m, int64_t k, int64_t ldx, const uint16_t* w, int64_t n, int64_t ldw,
                const coat_epilogue* e, const void* bias, int32_t bias_type, const void* residual, int64_t ldr, uint16_t* z,
                int64_t ldz, void* y, int64_t ldy, int32_t y_type, void* workspace, size_t workspace_bytes, coat_stream_t stream) {
    int rc = check_linear(x, m, k, ldx, w, n, ldw, e, bias, bias_type, residual, ldr, z, ldz, y, ldy, y_type);
    if (rc || m == 0 || n == 0) return rc;
    const bool ready = tiles_take(x, ldx, k) && tiles_take(w, ldw, k);
    const size_t need = coat_linear_workspace_bytes(m, n, k, ready);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return COAT_EINVAL;
        if (!aligned(workspace, 256)) return COAT_EALIGN;
    }
    const LinearLayout l = linear_layout(m, n, k, ready);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    char* const ws = static_cast<char*>(workspace);
    Product16 p{x, w, ldx, ldw, nullptr, nullptr, nullptr, m, n, k};
    if (!ready && l.plan.way != Way16::kPlain && l.plan.way != Way16::kFew) {
        uint16_t *const px = reinterpret_cast<uint16_t*>(ws + l.x), *const pw = reinterpret_cast<uint16_t*>(ws + l.w);
        if ((rc = launch_pack(Pack{x, m, ldx, nullptr, nullptr, px}, Pack{w, n, ldw, nullptr, nullptr, pw}, k, st))) return rc;
        p.a = px;
        p.b = pw;
        p.lda = p.ldb = packed_ld(k);
    }
    float* const part = reinterpret_cast<float*>(ws + l.part);
    if (y_type == COAT_FP32) return launch_linear<float>(p, l.plan, part, e, bias, bias_type, residual, ldr, z, ldz, y, ldy, st);
    return launch_linear<uint16_t>(p, l.plan, part, e, bias, bias_type, residual, ldr, z, ldz, y, ldy, st);
}

size_t coat_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t aligned) {
    if (m < 1 || n < 1 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
    return linear_backward_layout(m, n, k, aligned != 0).end;
}

int coat_linear_backward(const void* dy, int64_t lddy, int32_t dy_type, const uint16_t* x, int64_t m, int64_t k, int64_t ldx,
                         const uint16_t* w, int64_t n, int64_t ldw, const coat_epilogue* e, const uint16_t* z, int64_t ldz,
                         uint16_t* dx, int64_t lddx, uint16_t* dw, int64_t lddw, void* dbias, int32_t dbias_type, void* workspace,
                         size_t workspace_bytes, coat_stream_t stream) {
    int rc = check_linear_backward(dy, lddy, dy_type, x, m, k, ldx, w, n, ldw, e, z, ldz, dx, lddx, dw, lddw, dbias, dbias_type);
    if (rc) return rc;
    const bool ready = tiles_take(x, ldx, k) && tiles_take(w, ldw, k);
    const size_t need = coat_linear_backward_workspace_bytes(m, n, k, ready);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return COAT_EINVAL;
        if (!aligned(workspace, 256)) return COAT_EALIGN;
    }
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const LinearBackwardLayout l = linear_backward_layout(m, n, k, ready);
    char* const ws = static_cast<char*>(workspace);
    uint16_t* const dz_made = reinterpret_cast<uint16_t*>(ws + l.dz);
    float* const part = reinterpret_cast<float*>(ws + l.bias);
    float* const sums = reinterpret_cast<float*>(ws + l.part);
    const uint32_t t = drop_threshold(e->p);
    const Drop drop{e->rng, e->offset, t, 0, 0};
    const float scale = e->scale * drop_factor(t);
    // dy itself is dz up to the factor
    const bool as_it_is = dy_type == COAT_BF16 && e->act == COAT_ACT_NONE && t == 0 && tiles_take(dy, lddy, n);
    const uint16_t* const dz = as_it_is ? static_cast<const uint16_t*>(dy) : dz_made;
    const int64_t ld_dz = as_it_is ? lddy : l.ld_dz;
    // dropping and cutting at zero leave bf16 values as they are
    const bool exact = dy_type == COAT_BF16 && (e->act == COAT_ACT_NONE || e->act == COAT_ACT_RELU);
    const bool two = !exact && m > 0 && n > 0 && k > 0 && dz_takes_two_terms(m, n);
    if (m > 0 && n > 0 && (dbias || !as_it_is)) {
        uint16_t* const to = as_it_is || (!dx && !dw) ? nullptr : dz_made;
        if (dy_type == COAT_FP32)
            rc = launch_dz(static_cast<const float*>(dy), lddy, z, ldz, e->act, drop, m, n, to, l.ld_dz, dbias ? part : nullptr, two, st);
        else
            rc = launch_dz(static_cast<const uint16_t*>(dy), lddy, z, ldz, e->act, drop, m, n, to, l.ld_dz, dbias ? part : nullptr, two, st);
        if (rc) return rc;
    }
    if (dbias && n > 0) {
        const Grid g = grid_xy(div_up(n, kWave), kBlock);
        const dim3 grid(g.x, g.y);
        const int64_t parts = div_up(m, bias_band(m, n));
        if (dbias_type == COAT_FP32)
            hipLaunchKernelGGL(bias_join_kernel<float>, grid, dim3(kBlock), 0, st, part, l.ld_dz, parts, n, scale, static_cast<float*>(dbias));
        else
            hipLaunchKernelGGL(bias_join_kernel<uint16_t>, grid, dim3(kBlock), 0, st, part, l.ld_dz, parts, n, scale,
                               static_cast<uint16_t*>(dbias));
        if ((rc = launch_status())) return rc;
    }
    const bool packs = !ready && m > 0 && n > 0 && k > 0;
    uint16_t *const px = reinterpret_cast<uint16_t*>(ws + l.x), *const pw = reinterpret_cast<uint16_t*>(ws + l.w);
    const Pack of_x{x, m, ldx, nullptr, nullptr, px}, of_w{w, n, ldw, nullptr, nullptr, pw};
    if (packs && dx && (rc = launch_pack(of_w, dw && !two ? of_x : Pack{}, k, st))) return rc;
    if (packs && !dx && dw && !two && (rc = launch_pack(of_x, Pack{}, k, st))) return rc;
    if (dx) {
        const Product16 p{dz, packs ? pw : w, ld_dz, packs ? packed_ld(k) : ldw, nullptr, nullptr, nullptr, m, k, n};
        if (two) {
            float* const acc = reinterpret_cast<float*>(ws + l.acc);
            const PiecesOut<true> first{nullptr, nullptr, nullptr, lddx, acc, packed_ld(k), true, scale, false};
            if ((rc = launch_product<false, true>(p, l.plan_dx, sums, first, st))) return rc;
            const PiecesOut<true> second{nullptr, nullptr, dx, lddx, acc, packed_ld(k), false, scale, true};
            Product16 left = p;
            left.a = dz + m * ld_dz;
            rc = launch_product<false, true>(left, l.plan_dx, sums, second, st);
        } else {
            rc = launch_product<false, true>(p, l.plan_dx, sums, ScaledOut{nullptr, scale, dx, lddx}, st);
        }
        if (rc) return rc;
    }
    if (dw) {
        const ScaledOut out{nullptr, scale, dw, lddw};
        if (two) {  // x's rows stand beside both terms
            Pack again = of_x;
            again.packed = px + m * packed_ld(k);
            again.finite = true;
            if ((rc = launch_pack(of_x, again, k, st))) return rc;
            const Product16 p{dz, px, ld_dz, packed_ld(k), nullptr, nullptr, nullptr, n, k, 2 * m};
            rc = launch_product<true, true>(p, l.plan_dw_two, sums, out, st);
        } else {
            rc = launch_product<true, true>(Product16{dz, packs ? px : x, ld_dz, packs ? packed_ld(k) : ldx, nullptr, nullptr, nullptr, n, k, m},
                                            l.plan_dw, sums, out, st);
        }
    }
    return rc;
}

}  // extern "C"

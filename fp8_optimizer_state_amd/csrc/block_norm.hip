// HIP (gfx950) kernels of the border between two transformer blocks: the norm
// after a block, the gated residual addition and the norm before the next block,
// forward (with the layer input in bf16, FP8 or 4-bit form) and backward.
#include "act_common.h"
#include "mx4_common.h"

namespace {

// A workgroup takes a row at a time; thread i holds the chunks of 8 channels
// i, i + threads, ... of it in registers, so that every matrix is read and
// written once, 16 bytes per lane and access. threads is a multiple of the
// wavefront, so a row reaches over to the next multiple of 512 channels (the
// padding of the 4-bit form); the lanes behind the last channel hold zeros.
constexpr int kMaxWaves = 16;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __builtin_bit_cast(float, xlane32(__builtin_bit_cast(uint32_t, v), d));
    return v;
}

// Sums of two values over the workgroup, the same bits in every thread. `buf`
// alternates between calls, so that one barrier a call is enough: a thread that
// writes a buffer again has passed the other buffer's barrier, which no thread
// reaches before it has read this one.
__device__ __forceinline__ void block_sum2(float (&scratch)[2][kMaxWaves][2], int buf, int waves, float& a, float& b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if (waves == 1) return;
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) {
        scratch[buf][wave][0] = a;
        scratch[buf][wave][1] = b;
    }
    __syncthreads();
    a = scratch[buf][0][0];
    b = scratch[buf][0][1];
    for (int i = 1; i < waves; ++i) {
        a += scratch[buf][i][0];
        b += scratch[buf][i][1];
    }
}

// 8 values of a weight, gate or gradient array of run-time type.
__device__ __forceinline__ void load_param8(const void* p, int32_t type, int64_t at, int64_t n, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    } else if (type == COAT_FP32) {
        load8(static_cast<const float*>(p) + at, n, v);
    } else {
        load8(static_cast<const uint16_t*>(p) + at, n, v);
    }
}
__device__ __forceinline__ void store_grad8(void* p, int32_t type, int64_t at, int64_t n, const float (&v)[8]) {
    if (type == COAT_FP32) store8(static_cast<float*>(p) + at, n, v);
    else store8(static_cast<uint16_t*>(p) + at, n, v);
}

// The value a stored element of the stream stands for.
__device__ __forceinline__ float stored(float v, const uint16_t*) {
    return __builtin_bit_cast(float, bf16_bits(v) << 16);
}
__device__ __forceinline__ float stored(float v, const float*) { return v; }

struct BorderForward {
    int64_t rows, cols, rpg;
    float eps, scale, inv_cols;
    int32_t post, pre, param_type, fmt, lanes;  // lanes: threads that share a group of codes
    const uint16_t* y;
    const void *r, *w_post, *w_pre, *gate;
    void* r_out;
    uint16_t* h;
    uint8_t* q;
    void* q_scale;
};

// Stores 8 channels of a layer input (given as their bf16 bits) in the stored form asked for.
__device__ __forceinline__ void store_codes8(const BorderForward& p, int64_t row, int64_t c, const float (&v)[8]) {
    if (p.fmt == COAT_FMT_MX4) {
        const int64_t qb = mx4_code_bytes(p.cols), sb = mx4_scale_bytes(p.cols);
        uint32_t am = absmax_bits(v);
        uint32_t o = xlane32(am, 1);
        am = am > o ? am : o;
        o = xlane32(am, 2);
        am = am > o ? am : o;
        const uint32_t b = mx4_scale_byte(am);
        const uint32_t code = b == 255u ? 0u : mx4_codes8(v, b);
        if (c / 2 < qb) *reinterpret_cast<gu32*>(gp(p.q) + row * qb + c / 2) = code;
        if ((threadIdx.x & 3) == 0 && c / 32 < sb) gp(static_cast<uint8_t*>(p.q_scale))[row * sb + c / 32] = (uint8_t)b;
        return;
    }
    uint32_t w[4], code[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (__builtin_bit_cast(uint32_t, v[2 * i]) >> 16) | (__builtin_bit_cast(uint32_t, v[2 * i + 1]) & 0xFFFF0000u);
    const uint32_t am = group_umax(bf16_absmax_bits(w), p.lanes);
    float sc;
    if (p.fmt == COAT_FMT_E4M3) {
        act_codes<COAT_FMT_E4M3>(w, am, code);
        sc = act_scale<COAT_FMT_E4M3>(am);
    } else {
        act_codes<COAT_FMT_E5M2>(w, am, code);
        sc = act_scale<COAT_FMT_E5M2>(am);
    }
    if (c >= p.cols) return;
    const int64_t at = row * p.cols + c;  // a multiple of 8: groups divide the row
    *reinterpret_cast<gu32x2*>(gp(p.q) + at) = u32x2{code[0], code[1]};
    if ((threadIdx.x & (p.lanes - 1)) == 0) gp(static_cast<float*>(p.q_scale))[at / (8 * p.lanes)] = sc;
}

template <class S, int NV, int MAXT>
__global__ __launch_bounds__(MAXT) void border_forward_kernel(BorderForward p) {
    __shared__ float scratch[2][kMaxWaves][2];
    const int tid = threadIdx.x, threads = blockDim.x, waves = threads / kWave;
    int buf = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t base = row * p.cols;
        float x[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8;
            load8(static_cast<const S*>(p.r) + base + c, p.cols - c, x[i]);
        }
        if (p.y) {
            float y[NV][8], ss = 0.0f, none = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8;
                load8(p.y + base + c, p.cols - c, y[i]);
            }
            float sig = p.scale;
            if (p.post) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(y[i][j], y[i][j], ss);
                block_sum2(scratch, buf, waves, ss, none);
                buf ^= 1;
                sig *= __builtin_amdgcn_rsqf(__builtin_fmaf(ss, p.inv_cols, p.eps));
            }
            const int64_t grow = p.gate ? row / p.rpg : 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
                float w[8], g[8];
                load_param8(p.w_post, p.param_type, c, n, w);
                load_param8(p.gate, p.param_type, grow * p.cols + c, n, g);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[i][j] = stored(__builtin_fmaf(y[i][j] * sig * w[j], g[j], x[i][j]), static_cast<const S*>(nullptr));
                if (p.r_out) store8(static_cast<S*>(p.r_out) + base + c, n, x[i]);
            }
        }
        if (!p.pre) continue;
        float ss = 0.0f, none = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(x[i][j], x[i][j], ss);
        block_sum2(scratch, buf, waves, ss, none);
        buf ^= 1;
        const float rho = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, p.inv_cols, p.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            float w[8];
            load_param8(p.w_pre, p.param_type, c, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[i][j] = __builtin_bit_cast(float, bf16_bits(j < n ? x[i][j] * rho * w[j] : 0.0f) << 16);
            if (p.h) store8(p.h + base + c, n, x[i]);
            if (p.q) store_codes8(p, row, c, x[i]);
        }
    }
}

struct BorderBackward {
    int64_t rows, cols, rpg, step, chunks;
    float eps, scale, inv_cols;
    int32_t post, param_type, grad_type;
    const uint16_t *y, *dh;
    const void *r, *dr_out, *w_post, *w_pre, *gate;
    void* dr;
    uint16_t* dy;
    void* dgate;
    float *part_pre, *part_post, *part_gate;  // partial sums, a row per workgroup; NULL if not wanted
};

// A workgroup takes consecutive rows and sums the gradients of the weights (and
// of a gate row, while its tokens last) in registers.
//   pre:  with u = w_pre dh, s2 = sum r u:  d = dr_out + rho u - r rho^3 s2 / cols
//   post: with u = w_post scale g d, s4 = sum y u:  dy = sig u - y sig^3 s4 / cols
template <class S, int NV, int MAXT>
__global__ __launch_bounds__(MAXT) void border_backward_kernel(BorderBackward p) {
    __shared__ float scratch[2][kMaxWaves][2];
    const int tid = threadIdx.x, threads = blockDim.x, waves = threads / kWave;
    int buf = 0;
    int64_t row, end;
    if (p.chunks > 0) {
        const int64_t g = blockIdx.x / p.chunks;
        row = g * p.rpg + (blockIdx.x - g * p.chunks) * p.step;
        end = row + p.step < (g + 1) * p.rpg ? row + p.step : (g + 1) * p.rpg;
    } else {
        row = (int64_t)blockIdx.x * p.step;
        end = row + p.step;
    }
    if (end > p.rows) end = p.rows;
    float acc_pre[NV][8], acc_post[NV][8], acc_gate[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_pre[i][j] = acc_post[i][j] = acc_gate[i][j] = 0.0f;
    for (; row < end; ++row) {
        const int64_t base = row * p.cols;
        float d[NV][8], x[NV][8], u[NV][8], y[NV][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            if (p.dr_out) {
                load8(static_cast<const S*>(p.dr_out) + base + c, n, d[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = 0.0f;
            }
            if (p.dh) {
                load8(static_cast<const S*>(p.r) + base + c, n, x[i]);
                load8(p.dh + base + c, n, u[i]);
            }
            if (p.y) load8(p.y + base + c, n, y[i]);
        }
        if (p.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8;
                float w[8];
                load_param8(p.w_pre, p.param_type, c, p.cols - c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s1 = __builtin_fmaf(x[i][j], x[i][j], s1);
                    s2 = __builtin_fmaf(x[i][j] * w[j], u[i][j], s2);
                }
            }
            block_sum2(scratch, buf, waves, s1, s2);
            buf ^= 1;
            const float rho = __builtin_amdgcn_rsqf(__builtin_fmaf(s1, p.inv_cols, p.eps));
            const float back = rho * rho * rho * (s2 * p.inv_cols);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8;
                float w[8];
                load_param8(p.w_pre, p.param_type, c, p.cols - c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float ru = rho * u[i][j];
                    acc_pre[i][j] = __builtin_fmaf(x[i][j], ru, acc_pre[i][j]);
                    d[i][j] += __builtin_fmaf(ru, w[j], -x[i][j] * back);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8;
            store8(static_cast<S*>(p.dr) + base + c, p.cols - c, d[i]);
        }
        if (!p.y) continue;
        const int64_t grow = p.gate ? row / p.rpg : 0;
        float s3 = 0.0f, s4 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            float w[8], g[8];
            load_param8(p.w_post, p.param_type, c, n, w);
            load_param8(p.gate, p.param_type, grow * p.cols + c, n, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[i][j] *= p.scale;  // scale d, from here on
                s3 = __builtin_fmaf(y[i][j], y[i][j], s3);
                s4 = __builtin_fmaf(y[i][j] * w[j], g[j] * d[i][j], s4);
            }
        }
        float sig = 1.0f, back = 0.0f;
        if (p.post) {
            block_sum2(scratch, buf, waves, s3, s4);
            buf ^= 1;
            sig = __builtin_amdgcn_rsqf(__builtin_fmaf(s3, p.inv_cols, p.eps));
            back = sig * sig * sig * (s4 * p.inv_cols);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            float w[8], g[8], out[8];
            load_param8(p.w_post, p.param_type, c, n, w);
            load_param8(p.gate, p.param_type, grow * p.cols + c, n, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float yn = y[i][j] * sig, gd = g[j] * d[i][j];
                acc_post[i][j] = __builtin_fmaf(gd, yn, acc_post[i][j]);
                acc_gate[i][j] = __builtin_fmaf(d[i][j] * w[j], yn, acc_gate[i][j]);
                out[j] = __builtin_fmaf(sig * w[j], gd, -y[i][j] * back);
            }
            store8(p.dy + base + c, n, out);
        }
        if (p.dgate && p.chunks <= 1 && (row + 1 == end || (row + 1) % p.rpg == 0)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8;
                store_grad8(p.dgate, p.grad_type, grow * p.cols + c, p.cols - c, acc_gate[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc_gate[i][j] = 0.0f;
            }
        }
    }
    const int64_t part = (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
        if (p.part_pre) store8(p.part_pre + part + c, n, acc_pre[i]);
        if (p.part_post) store8(p.part_post + part + c, n, acc_post[i]);
        if (p.part_gate) store8(p.part_gate + part + c, n, acc_gate[i]);
    }
}

// Sums the partial rows of each array, in the order of the workgroups: a
// wavefront takes a quarter of the rows of 64 columns, the quarters are added
// in order. blockIdx.y: 0 the pre-norm's weights, 1 the post-norm's, 2 + g gate row g.
struct BorderReduce {
    const float *pre, *post, *gate;
    void *dw_pre, *dw_post, *dgate;
    int64_t blocks, chunks, cols;
    int32_t grad_type;
};
__global__ __launch_bounds__(kBlock) void border_reduce_kernel(BorderReduce p) {
    __shared__ float sums[kWavesPerBlock][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;
    const float* src = p.pre;
    void* dst = p.dw_pre;
    int64_t count = p.blocks, at = c;
    if (blockIdx.y == 1) {
        src = p.post;
        dst = p.dw_post;
    } else if (blockIdx.y > 1) {
        const int64_t g = blockIdx.y - 2;
        count = p.chunks;
        src = p.gate + g * count * p.cols;
        dst = p.dgate;
        at += g * p.cols;
    }
    if (!dst) return;
    const int64_t quarter = (count + kWavesPerBlock - 1) / kWavesPerBlock;
    const int64_t b1 = (wave + 1) * quarter < count ? (wave + 1) * quarter : count;
    float sum = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int64_t b = wave * quarter; b < b1; ++b) sum += gp(src)[b * p.cols + c];
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && c < p.cols) {
        sum = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
        if (p.grad_type == COAT_FP32) gp(static_cast<float*>(dst))[at] = sum;
        else gp(static_cast<uint16_t*>(dst))[at] = (uint16_t)bf16_bits(sum);
    }
}

// Threads of a workgroup that holds NV chunks a thread of a row.
inline int border_threads(int64_t cols, int nv) { return (int)div_up(div_up(cols, 8), (int64_t)kWave * nv) * kWave; }

template <class S>
int launch_forward(const BorderForward& p, hipStream_t st) {
    const int64_t most = (int64_t)kCUs * 8;
    const dim3 grid((unsigned)(p.rows < most ? p.rows : most));
    if (p.cols <= 4096)
        hipLaunchKernelGGL((border_forward_kernel<S, 1, 512>), grid, dim3(border_threads(p.cols, 1)), 0, st, p);
    else if (p.cols <= 8192)
        hipLaunchKernelGGL((border_forward_kernel<S, 2, 512>), grid, dim3(border_threads(p.cols, 2)), 0, st, p);
    else
        hipLaunchKernelGGL((border_forward_kernel<S, 2, 1024>), grid, dim3(border_threads(p.cols, 2)), 0, st, p);
    return launch_status();
}

template <class S>
int launch_backward(const BorderBackward& p, int64_t blocks, hipStream_t st) {
    const dim3 grid((unsigned)blocks);
    if (p.cols <= 4096)
        hipLaunchKernelGGL((border_backward_kernel<S, 1, 512>), grid, dim3(border_threads(p.cols, 1)), 0, st, p);
    else if (p.cols <= 8192)
        hipLaunchKernelGGL((border_backward_kernel<S, 2, 512>), grid, dim3(border_threads(p.cols, 2)), 0, st, p);
    else
        hipLaunchKernelGGL((border_backward_kernel<S, 2, 1024>), grid, dim3(border_threads(p.cols, 2)), 0, st, p);
    return launch_status();
}

}  // namespace

// ====================================================================== C ABI

extern "C" {

int coat_block_norm(const coat_border* b, const uint16_t* y, const void* r, const void* w_post, const void* w_pre,
                    const void* gate, void* r_out, uint16_t* h, uint8_t* q, void* q_scale, int32_t group, int32_t fmt,
                    coat_stream_t stream) {
    const int rc = check_block_norm(b, y, r, w_post, w_pre, gate, r_out, h, q, q_scale, group, fmt);
    if (rc || b->rows == 0) return rc;
    BorderForward p;
    p.rows = b->rows;
    p.cols = b->cols;
    p.rpg = b->rows_per_gate;
    p.eps = b->eps;
    p.scale = b->scale;
    p.inv_cols = (float)(1.0 / (double)b->cols);
    p.post = b->post;
    p.pre = h || q;
    p.param_type = b->param_type;
    p.fmt = fmt;
    p.lanes = q ? group / 8 : 1;
    p.y = y;
    p.r = r;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.gate = gate;
    p.r_out = r_out;
    p.h = h;
    p.q = q;
    p.q_scale = q_scale;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return b->stream_type == COAT_FP32 ? launch_forward<float>(p, st) : launch_forward<uint16_t>(p, st);
}

size_t coat_block_norm_backward_workspace_bytes(const coat_border* b) { return border_workspace_bytes(b); }

int coat_block_norm_backward(const coat_border* b, const uint16_t* y, const void* r_out, const void* dr_out,
                             const uint16_t* dh, const void* w_post, const void* w_pre, const void* gate, void* dr,
                             uint16_t* dy, void* dw_post, void* dw_pre, void* dgate, void* workspace,
                             size_t workspace_bytes, coat_stream_t stream) {
    const int rc = check_block_norm_backward(b, y, r_out, dr_out, dh, w_post, w_pre, gate, dr, dy, dw_post, dw_pre,
                                             dgate, workspace, workspace_bytes);
    if (rc) return rc;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const BorderSplit split = border_split(b->rows, b->rows_per_gate, dgate != nullptr);
    const size_t section = border_section_bytes(split.blocks, b->cols) / sizeof(float);
    float* ws = static_cast<float*>(workspace);
    BorderBackward p;
    p.rows = b->rows;
    p.cols = b->cols;
    p.rpg = b->rows_per_gate < b->rows ? b->rows_per_gate : b->rows;
    p.step = split.step;
    p.chunks = split.chunks;
    p.eps = b->eps;
    p.scale = b->scale;
    p.inv_cols = (float)(1.0 / (double)b->cols);
    p.post = b->post;
    p.param_type = b->param_type;
    p.grad_type = b->grad_type;
    p.y = y;
    p.dh = dh;
    p.r = r_out;
    p.dr_out = dr_out;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.gate = gate;
    p.dr = dr;
    p.dy = dy;
    p.dgate = dgate;
    p.part_pre = dw_pre ? ws : nullptr;
    p.part_post = dw_post ? ws + section : nullptr;
    p.part_gate = dgate && split.chunks > 1 ? ws + 2 * section : nullptr;
    if (b->rows > 0) {
        const int run = b->stream_type == COAT_FP32 ? launch_backward<float>(p, split.blocks, st)
                                                    : launch_backward<uint16_t>(p, split.blocks, st);
        if (run) return run;
    }
    if (!dw_pre && !dw_post && !p.part_gate) return COAT_OK;
    BorderReduce red;
    red.pre = p.part_pre;
    red.post = p.part_post;
    red.gate = p.part_gate;
    red.dw_pre = dw_pre;
    red.dw_post = dw_post;
    red.dgate = p.part_gate ? dgate : nullptr;
    red.blocks = split.blocks;
    red.chunks = split.chunks;
    red.cols = b->cols;
    red.grad_type = b->grad_type;
    const unsigned gates = p.part_gate ? (unsigned)(split.blocks / split.chunks) : 0u;
    hipLaunchKernelGGL(border_reduce_kernel, dim3((unsigned)div_up(b->cols, kWave), 2 + gates), dim3(kBlock), 0, st, red);
    return launch_status();
}

}  // extern "C"

// HIP (gfx950) kernels of the border between two transformer blocks: the norm
// after a block, the gated residual addition and the norm before the next block,
// forward (with the layer input in bf16, FP8 or 4-bit form) and backward.
#include <type_traits>

#include "act_common.h"
#include "mx4_common.h"

namespace {

// A workgroup takes a row at a time; thread i holds the chunks of 8 channels
// i, i + threads, ... of it in registers, so that every matrix is read and
// written once, 16 bytes per lane and access. threads is a multiple of the
// wavefront, so a row reaches over to the next multiple of 512 channels (the
// padding of the 4-bit form); the lanes behind the last channel hold zeros. Bound
// by HBM: 16384 x 5120 in bf16 take 140 us forward (4.8 TB/s; 147 us to FP8, 118 to
// 4 bits) and 212 us backward (4.7 TB/s); a copy of that size runs at 4.7. Rows of
// odd width lie at any byte: 1031 x 2731 takes 29 us backward, the latency of three
// rows one after the other and of the second launch.
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

// A value that every lane holds, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// How a row ends: with a whole chunk, inside one, or before the first one's end.
enum Edge { kWhole, kInside, kTiny };

// 8 elements of a row; settle_row8 finishes what it began.
template <int EDGE, class E>
__device__ __forceinline__ Raw8<E> load_row8(const E* p, int64_t n) {
    if constexpr (EDGE == kInside) return load_end8(p, n);
    else return load_raw8<EDGE == kWhole>(p, n);
}
template <int EDGE, class E>
__device__ __forceinline__ void settle_row8(Raw8<E>& r, int64_t n) {
    if constexpr (EDGE == kInside) settle8(r, n);
}

// The same of a matrix that may be missing (zeros).
template <int EDGE, class E>
__device__ __forceinline__ Raw8<E> load_maybe8(const E* p, int64_t at, int64_t n) {
    if constexpr (EDGE == kInside) {
        if (p) return load_end8(p + at, n);
        return load_raw8<true>(p, 0);
    } else {
        return load_row8<EDGE>(p + at, p ? n : 0);
    }
}

// 8 values of a weight or gate that may be missing (ones).
template <int EDGE, class P>
__device__ __forceinline__ Raw8<P> load_param8(const void* p, int64_t at, int64_t n) {
    if (p) {
        Raw8<P> r = load_row8<EDGE>(static_cast<const P*>(p) + at, n);
        settle_row8<EDGE>(r, n);
        return r;
    }
    Raw8<P> r;
    if constexpr (sizeof(P) == 4) r.lo = r.hi = u32x4{0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u};
    else r.w = u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    return r;
}
template <int EDGE>
__device__ __forceinline__ void store_grad8(void* p, int32_t type, int64_t at, int64_t n, const float (&v)[8]) {
    if (type == COAT_FP32) store8<EDGE == kWhole>(static_cast<float*>(p) + at, n, v);
    else store8<EDGE == kWhole>(static_cast<uint16_t*>(p) + at, n, v);
}

// The value a stored element of the stream stands for.
__device__ __forceinline__ float stored(float v, const uint16_t*) {
    return __builtin_bit_cast(float, bf16_bits(v) << 16);
}
__device__ __forceinline__ float stored(float v, const float*) { return v; }

struct BorderForward {
    int64_t rows, cols, rpg, step;
    float eps, scale, inv_cols;
    int32_t post, pre, fmt, lg2_lanes;  // threads that share a group of codes
    const uint16_t* y;
    const void *r, *w_post, *w_pre, *gate;
    void* r_out;
    uint16_t* h;
    uint8_t* q;
    void* q_scale;
};

// Stores 8 channels of a layer input (given as their bf16 bits) in the stored form asked for.
__device__ __forceinline__ void store_codes8(const BorderForward& p, int64_t row, int64_t c, const float (&v)[8]) {
    Raw8<uint16_t> raw;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        raw.w[i] = (__builtin_bit_cast(uint32_t, v[2 * i]) >> 16) | (__builtin_bit_cast(uint32_t, v[2 * i + 1]) & 0xFFFF0000u);
    if (p.fmt == COAT_FMT_MX4) {
        const int64_t qb = mx4_code_bytes(p.cols), sb = mx4_scale_bytes(p.cols);
        const uint32_t b = mx4_scale_byte(block_max(absmax_bits(raw)));
        const uint32_t code = b == 255u ? 0u : mx4_codes8(raw, b);
        if (c / 2 < qb) *reinterpret_cast<gu32*>(gp(p.q) + row * qb + c / 2) = code;
        if ((threadIdx.x & 3) == 0 && c / 32 < sb) gp(static_cast<uint8_t*>(p.q_scale))[row * sb + c / 32] = (uint8_t)b;
        return;
    }
    const uint32_t w[4] = {raw.w[0], raw.w[1], raw.w[2], raw.w[3]};
    const int lanes = 1 << p.lg2_lanes;
    uint32_t code[2];
    const uint32_t am = group_umax(bf16_absmax_bits(w), lanes);
    float sc;
    if (p.fmt == COAT_FMT_E4M3) {
        sc = act_scale<COAT_FMT_E4M3>(am);
        act_codes<COAT_FMT_E4M3>(w, am, sc, code);
    } else {
        sc = act_scale<COAT_FMT_E5M2>(am);
        act_codes<COAT_FMT_E5M2>(w, am, sc, code);
    }
    if (c >= p.cols) return;
    const int64_t at = row * p.cols + c;  // a multiple of 8: groups divide the row
    *reinterpret_cast<gu32x2*>(gp(p.q) + at) = u32x2{code[0], code[1]};
    if ((threadIdx.x & (lanes - 1)) == 0) gp(static_cast<float*>(p.q_scale))[at >> (3 + p.lg2_lanes)] = sc;
}

// S the stream's type, P the weights' and gate's, NV chunks a thread. A workgroup takes `step` consecutive rows;
// the weights, and the gate row while its tokens last, stay in registers.
template <class S, class P, int NV, int EDGE>
__global__ __launch_bounds__(1024) void border_forward_kernel(BorderForward p) {
    __shared__ float scratch[2][kMaxWaves][2];
    const int tid = threadIdx.x, threads = blockDim.x, waves = threads / kWave;
    int buf = 0;
    int64_t row = (int64_t)blockIdx.x * p.step;
    const int64_t end = row + p.step < p.rows ? row + p.step : p.rows;
    Raw8<P> w_post[NV], w_pre[NV], gate[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
        w_post[i] = load_param8<EDGE, P>(p.w_post, c, n);
        w_pre[i] = load_param8<EDGE, P>(p.w_pre, c, n);
        gate[i] = load_param8<EDGE, P>(nullptr, c, n);
    }
    int64_t gate_end = p.gate ? row : end;  // first row that needs another gate row
    for (; row < end; ++row) {
        const int64_t base = row * p.cols;
        float x[NV][8];
        if (p.y) {
            Raw8<uint16_t> y[NV];
            Raw8<S> r[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
                y[i] = load_row8<EDGE>(p.y + base + c, n);
                r[i] = load_row8<EDGE>(static_cast<const S*>(p.r) + base + c, n);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t n = p.cols - (int64_t)(i * threads + tid) * 8;
                settle_row8<EDGE>(y[i], n);
                settle_row8<EDGE>(r[i], n);
            }
            if (row >= gate_end) {
                const int64_t g = row / p.rpg;
                gate_end = (g + 1) * p.rpg;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int64_t c = (int64_t)(i * threads + tid) * 8;
                    gate[i] = load_param8<EDGE, P>(p.gate, g * p.cols + c, p.cols - c);
                }
            }
            float sig = p.scale;
            if (p.post) {
                float ss = 0.0f, none = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float v[8];
                    expand(y[i], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[j], v[j], ss);
                }
                block_sum2(scratch, buf, waves, ss, none);
                buf ^= 1;
                sig *= __builtin_amdgcn_rsqf(__builtin_fmaf(ss, p.inv_cols, p.eps));
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
                float v[8], w[8], g[8];
                expand(y[i], v);
                expand(w_post[i], w);
                expand(gate[i], g);
                expand(r[i], x[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[i][j] = stored(__builtin_fmaf(v[j] * sig * w[j], g[j], x[i][j]), static_cast<const S*>(nullptr));
                if (p.r_out) store8<EDGE == kWhole>(static_cast<S*>(p.r_out) + base + c, n, x[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
                Raw8<S> r = load_row8<EDGE>(static_cast<const S*>(p.r) + base + c, n);
                settle_row8<EDGE>(r, n);
                expand(r, x[i]);
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
            expand(w_pre[i], w);
            // channels past the end are zeros even where rho is not finite
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[i][j] = __builtin_bit_cast(float, bf16_bits((EDGE == kWhole ? n > 0 : j < n) ? x[i][j] * rho * w[j] : 0.0f) << 16);
            if (p.h) store8<EDGE == kWhole>(p.h + base + c, n, x[i]);
            if (p.q) store_codes8(p, row, c, x[i]);
        }
    }
}

struct BorderBackward {
    int64_t rows, cols, rpg, step, chunks;
    float eps, scale, inv_cols;
    int32_t post, grad_type;
    const uint16_t *y, *dh;
    const void *r, *dr_out, *w_post, *w_pre, *gate;
    void* dr;
    uint16_t* dy;
    void* dgate;
    float *part_pre, *part_post, *part_gate;  // partial sums, a row per workgroup; NULL if not wanted
};

// A workgroup takes consecutive rows and sums the gradients of the weights (and
// of a gate row, while its tokens last) in registers.
//   pre:  with u = w_pre dh, s2 = sum r u:  d = dr_out + rho (u - (r rho) (rho (s2 / cols)))
//   post: with u = w_post scale g d, s4 = sum y u:  dy = sig (u - y (sig (s4 / cols)) sig)
// The products are formed in this order: rho^3 leaves fp32's range for rows of 1e13
// and for rows of zeros with eps under 2e-26, while r rho is at most sqrt(cols).
// (y sig multiplied first, as r rho is, costs registers: 16384 x 13824 650 us.)
// MAXT: threads at most. Up to 768 leave registers for loading a row while the
// one before it is worked on.
template <class S, class P, int NV, int EDGE, int MAXT>
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
    // With two chunks a thread the registers do not hold everything (13824
    // channels: 1667 us for 16384 rows with the spills): the weights are read for
    // each row, and two of the three sums lie in LDS, each thread's own. What is left
    // over still takes 24 to 96 bytes of scratch a thread: 641 us with a bf16 stream
    // (4.2 TB/s), 898 with fp32, 1287 with fp32 weights too and 13823 channels (3.2).
    constexpr bool KEEP = NV == 1;
    __shared__ f32x4 sums[KEEP ? 1 : 2 * NV * 2 * 1024];  // [array][chunk][half chunk][thread]
    auto get = [&](int array, int i, const float (&kept)[8], float (&v)[8]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 q;
            if constexpr (!KEEP) q = sums[((array * NV + i) * 2 + h) * 1024 + tid];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * h + j] = KEEP ? kept[4 * h + j] : q[j];
        }
    };
    auto put = [&](int array, int i, float (&kept)[8], const float (&v)[8]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (!KEEP) {
                sums[((array * NV + i) * 2 + h) * 1024 + tid] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) kept[4 * h + j] = v[4 * h + j];
            }
        }
    };
    const float zeros[8] = {};
    Raw8<P> w_post[NV], w_pre[NV], gate[NV];
    auto weight = [&](const Raw8<P>& kept, const void* from, int64_t at, int64_t c, float (&v)[8]) {
        if constexpr (KEEP) expand(kept, v);
        else expand(load_param8<EDGE, P>(from, at + c, p.cols - c), v);
    };
    float acc_pre[NV][8], acc_post[NV][8], acc_gate[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
        if constexpr (KEEP) {
            w_post[i] = load_param8<EDGE, P>(p.w_post, c, n);
            w_pre[i] = load_param8<EDGE, P>(p.w_pre, c, n);
            gate[i] = load_param8<EDGE, P>(nullptr, c, n);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_pre[i][j] = 0.0f;
        put(0, i, acc_post[i], zeros);
        put(1, i, acc_gate[i], zeros);
    }
    int64_t gate_end = p.gate ? row : end;  // first row that needs another gate row
    // Without the post-norm y plays no part in dy, whatever it holds (its factor is 0,
    // but 0 Inf is not). With one chunk a thread by a branch (16384 x 5120: 212 us, 216
    // with the mask), with two by a mask (16384 x 13824: 640, 687 with the branch).
    const uint32_t post_mask = p.post ? 0xFFFFFFFFu : 0u;
    constexpr bool EARLY = MAXT < 1024;
    Raw8<uint16_t> y[NV], u[NV], y_next[NV], u_next[NV];
    Raw8<S> x[NV], dr[NV], x_next[NV], dr_next[NV];
    auto load_row = [&](int64_t at, Raw8<uint16_t> (&yv)[NV], Raw8<uint16_t> (&uv)[NV], Raw8<S> (&xv)[NV], Raw8<S> (&dv)[NV]) {
        const int64_t from = at * p.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            if (p.dh) {
                xv[i] = load_row8<EDGE>(static_cast<const S*>(p.r) + from + c, n);
                uv[i] = load_row8<EDGE>(p.dh + from + c, n);
            }
            dv[i] = load_maybe8<EDGE>(static_cast<const S*>(p.dr_out), from + c, n);
            yv[i] = load_maybe8<EDGE>(p.y, from + c, n);
        }
    };
    auto settle_row = [&] {
        if (EDGE != kInside) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t n = p.cols - (int64_t)(i * threads + tid) * 8;
            settle_row8<EDGE>(x[i], n);
            settle_row8<EDGE>(u[i], n);
            settle_row8<EDGE>(dr[i], n);
            settle_row8<EDGE>(y[i], n);
        }
    };
    if (EARLY && row < end) load_row(row, y_next, u_next, x_next, dr_next);
    for (; row < end; ++row) {
        const int64_t base = row * p.cols;
        if constexpr (EARLY) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                y[i] = y_next[i];
                u[i] = u_next[i];
                x[i] = x_next[i];
                dr[i] = dr_next[i];
            }
            if (row + 1 < end) load_row(row + 1, y_next, u_next, x_next, dr_next);
        } else {
            load_row(row, y, u, x, dr);
        }
        settle_row();
        const int64_t g_row = p.gate ? row / p.rpg : 0;
        if (row >= gate_end) {
            gate_end = (g_row + 1) * p.rpg;
            if constexpr (KEEP) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int64_t c = (int64_t)(i * threads + tid) * 8;
                    gate[i] = load_param8<EDGE, P>(p.gate, g_row * p.cols + c, p.cols - c);
                }
            }
        }
        float rho = 0.0f, back = 0.0f;
        if (p.dh) {
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8;
                float xv[8], uv[8], w[8];
                expand(x[i], xv);
                expand(u[i], uv);
                weight(w_pre[i], p.w_pre, 0, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s1 = __builtin_fmaf(xv[j], xv[j], s1);
                    s2 = __builtin_fmaf(xv[j] * w[j], uv[j], s2);
                }
            }
            block_sum2(scratch, buf, waves, s1, s2);
            buf ^= 1;
            rho = uniform(__builtin_amdgcn_rsqf(__builtin_fmaf(s1, p.inv_cols, p.eps)));
            back = uniform(rho * (s2 * p.inv_cols));
        }
        float d[NV][8];
        float s3 = 0.0f, s4 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            expand(dr[i], d[i]);
            if (p.dh) {
                float xv[8], uv[8], w[8];
                expand(x[i], xv);
                expand(u[i], uv);
                weight(w_pre[i], p.w_pre, 0, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xn = xv[j] * rho;
                    acc_pre[i][j] = __builtin_fmaf(xn, uv[j], acc_pre[i][j]);
                    d[i][j] = __builtin_fmaf(rho, __builtin_fmaf(uv[j], w[j], -xn * back), d[i][j]);
                }
            }
            store8<EDGE == kWhole>(static_cast<S*>(p.dr) + base + c, n, d[i]);
            if (p.y) {
                float yv[8], w[8], g[8];
                expand(y[i], yv);
                weight(w_post[i], p.w_post, 0, c, w);
                weight(gate[i], p.gate, g_row * p.cols, c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[i][j] *= p.scale;  // scale d, from here on
                    s3 = __builtin_fmaf(yv[j], yv[j], s3);
                    s4 = __builtin_fmaf(yv[j] * w[j], g[j] * d[i][j], s4);
                }
            }
        }
        if (!p.y) continue;
        float sig = 1.0f;
        back = 0.0f;
        if (p.post) {
            block_sum2(scratch, buf, waves, s3, s4);
            buf ^= 1;
            sig = uniform(__builtin_amdgcn_rsqf(__builtin_fmaf(s3, p.inv_cols, p.eps)));
            back = uniform(sig * (s4 * p.inv_cols));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
            float yv[8], w[8], g[8], out[8], post[8], gates[8];
            get(0, i, acc_post[i], post);
            get(1, i, acc_gate[i], gates);
            expand(y[i], yv);
            weight(w_post[i], p.w_post, 0, c, w);
            weight(gate[i], p.gate, g_row * p.cols, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float yn = yv[j] * sig, gd = g[j] * d[i][j];
                post[j] = __builtin_fmaf(gd, yn, post[j]);
                gates[j] = __builtin_fmaf(d[i][j] * w[j], yn, gates[j]);
                const float yp = KEEP ? yv[j] : as_float(__builtin_bit_cast(uint32_t, yv[j]) & post_mask);
                out[j] = sig * __builtin_fmaf(yp * back, -sig, w[j] * gd);
            }
            if (KEEP && !p.post) {
                asm volatile("; dy without the post-norm");  // keeps the branch, which otherwise becomes selects
#pragma unroll
                for (int j = 0; j < 8; ++j) out[j] = g[j] * d[i][j];
            }
            put(0, i, acc_post[i], post);
            put(1, i, acc_gate[i], gates);
            store8<EDGE == kWhole>(p.dy + base + c, n, out);
        }
        if (p.dgate && p.chunks <= 1 && (row + 1 == end || row + 1 == gate_end)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * threads + tid) * 8;
                float gates[8];
                get(1, i, acc_gate[i], gates);
                store_grad8<EDGE>(p.dgate, p.grad_type, g_row * p.cols + c, p.cols - c, gates);
                put(1, i, acc_gate[i], zeros);
            }
        }
    }
    const int64_t part = (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * threads + tid) * 8, n = p.cols - c;
        if (p.part_pre) store8<EDGE == kWhole>(p.part_pre + part + c, n, acc_pre[i]);
        float v[8];
        get(0, i, acc_post[i], v);
        if (p.part_post) store8<EDGE == kWhole>(p.part_post + part + c, n, v);
        get(1, i, acc_gate[i], v);
        if (p.part_gate) store8<EDGE == kWhole>(p.part_gate + part + c, n, v);
    }
}

// Sums the partial rows of each array, in the order of the workgroups: a
// wavefront takes a sixteenth of the rows of 64 columns, the parts are added in
// order. blockIdx.y: 0 the pre-norm's weights, 1 the post-norm's, 2 + g gate row g.
struct BorderReduce {
    const float *pre, *post, *gate;
    void *dw_pre, *dw_post, *dgate;
    int64_t blocks, chunks, cols;
    int32_t grad_type;
};
__global__ __launch_bounds__(kMaxWaves * kWave) void border_reduce_kernel(BorderReduce p) {
    __shared__ float sums[kMaxWaves][kWave];
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
    const int64_t part = (count + kMaxWaves - 1) / kMaxWaves;
    const int64_t b1 = (wave + 1) * part < count ? (wave + 1) * part : count;
    float sum = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int64_t b = wave * part; b < b1; ++b) sum += gp(src)[b * p.cols + c];
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && c < p.cols) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxWaves; ++i) sum += sums[i][lane];
        if (p.grad_type == COAT_FP32) gp(static_cast<float*>(dst))[at] = sum;
        else gp(static_cast<uint16_t*>(dst))[at] = (uint16_t)bf16_bits(sum);
    }
}

// Calls launch(NV, EDGE, threads): the first two as compile-time constants.
template <class F>
void border_shape(int64_t cols, F&& launch) {
    const dim3 threads((unsigned)(border_waves(cols) * kWave));
    using one = std::integral_constant<int, 1>;
    using two = std::integral_constant<int, 2>;
    using whole = std::integral_constant<int, kWhole>;
    using inside = std::integral_constant<int, kInside>;
    if (cols < 8) launch(one{}, std::integral_constant<int, kTiny>{}, threads);
    else if (border_chunks(cols) == 1) cols % 8 == 0 ? launch(one{}, whole{}, threads) : launch(one{}, inside{}, threads);
    else cols % 8 == 0 ? launch(two{}, whole{}, threads) : launch(two{}, inside{}, threads);
}

template <class S, class P>
int launch_forward(BorderForward& p, hipStream_t st) {
    border_shape(p.cols, [&](auto nv, auto edge, dim3 threads) {
        // as many workgroups as run at once (24 wavefronts on a compute unit):
        // 16384 x 5120 takes 144 us with 2 of 10 wavefronts each, 152 with 3, 162
        // with 4; small ones hide their barriers better when there are twice as
        // many (16384 x 1024: 28 us with 16 of 2 wavefronts, 45 with 3, 26 with 32)
        const int64_t waves = threads.x / kWave;
        const int64_t each = waves > 12 ? 1 : 24 / waves;
        p.step = div_up(p.rows, kCUs * (waves <= 4 ? 2 * each : each));
        hipLaunchKernelGGL((border_forward_kernel<S, P, nv.value, edge.value>), dim3((unsigned)div_up(p.rows, p.step)), threads,
                           0, st, p);
    });
    return launch_status();
}

template <class S, class P>
int launch_backward(const BorderBackward& p, int64_t blocks, hipStream_t st) {
    border_shape(p.cols, [&](auto nv, auto edge, dim3 threads) {
        if constexpr (nv.value == 2) {
            hipLaunchKernelGGL((border_backward_kernel<S, P, 2, edge.value, 1024>), dim3((unsigned)blocks), threads, 0, st, p);
        } else if (edge.value == kTiny || threads.x <= 512) {
            hipLaunchKernelGGL((border_backward_kernel<S, P, 1, edge.value, 512>), dim3((unsigned)blocks), threads, 0, st, p);
        } else if constexpr (edge.value == kTiny) {
        } else if (threads.x <= 768) {
            hipLaunchKernelGGL((border_backward_kernel<S, P, 1, edge.value, 768>), dim3((unsigned)blocks), threads, 0, st, p);
        } else {
            hipLaunchKernelGGL((border_backward_kernel<S, P, 1, edge.value, 1024>), dim3((unsigned)blocks), threads, 0, st, p);
        }
    });
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
    p.fmt = fmt;
    p.lg2_lanes = q ? lg2_group_of(group) - 3 : 0;
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
    if (b->param_type == COAT_FP32)
        return b->stream_type == COAT_FP32 ? launch_forward<float, float>(p, st) : launch_forward<uint16_t, float>(p, st);
    return b->stream_type == COAT_FP32 ? launch_forward<float, uint16_t>(p, st) : launch_forward<uint16_t, uint16_t>(p, st);
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
    const BorderSplit split = border_split(b->rows, b->cols, b->rows_per_gate, dgate != nullptr);
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
        const bool s32 = b->stream_type == COAT_FP32;
        const int run = b->param_type == COAT_FP32 ? (s32 ? launch_backward<float, float>(p, split.blocks, st)
                                                          : launch_backward<uint16_t, float>(p, split.blocks, st))
                                                   : (s32 ? launch_backward<float, uint16_t>(p, split.blocks, st)
                                                          : launch_backward<uint16_t, uint16_t>(p, split.blocks, st));
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
    hipLaunchKernelGGL(border_reduce_kernel, dim3((unsigned)div_up(b->cols, kWave), 2 + gates), dim3(kMaxWaves * kWave), 0, st, red);
    return launch_status();
}

}  // extern "C"

// HIP (gfx950) softmax cross entropy of a vocabulary projection, the logits never stored.
#include "bf16_product.h"

// Forward: the tokens that count are listed (one workgroup; 5 us at 1023 tokens, 17 at
// 8192), the logits' tiles leave a maximum and a sum of exponentials for each row of theirs,
// and those are joined (15 us at 8192 tokens): 8192 x 32000 x 5120 takes 1840 us, 1.46
// PFLOP/s, bound as the product is. Listing them lets the tiles pass over the others.
//
// Backward: the rows that count are packed (so that what the others hold, an infinity say,
// reaches no sum), and for one piece of the vocabulary after the other the logits are
// computed again, their gradients stored in bf16 (with second terms where tokens are few) and
// multiplied twice. The logits' second product is a third of the work; storing them would
// take tokens x vocabulary numbers.
namespace {

constexpr int kRowsBlock = 1024;
constexpr int kRowsEach = 8;  // labels of a thread in a turn

// Exclusive prefix of `mine` over the workgroup; `total` is its sum.
__device__ __forceinline__ int32_t block_prefix(int32_t mine, int32_t& total) {
    __shared__ int32_t sums[kRowsBlock / kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int32_t upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int32_t v = __shfl_up(upto, d, kWave);
        if (lane >= d) upto += v;
    }
    __syncthreads();
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    int32_t before = 0;
    total = 0;
    for (int i = 0; i < kRowsBlock / kWave; ++i) {
        if (i < wave) before += sums[i];
        total += sums[i];
    }
    return before + upto - mine;
}

__device__ __forceinline__ int32_t label_in(int64_t label, int64_t vocab) {
    return label >= 0 && label < vocab ? (int32_t)label : -1;
}

// The tokens that count, in order: their places, labels and number. The others' loss
// and lse are zero. One workgroup.
__global__ __launch_bounds__(kRowsBlock) void xent_rows_kernel(const int64_t* __restrict__ labels, int64_t tokens, int64_t ignore,
                                                               int64_t vocab, int32_t* __restrict__ count, int32_t* __restrict__ at,
                                                               int32_t* __restrict__ label, float* __restrict__ zt,
                                                               float* __restrict__ loss, float* __restrict__ lse) {
    int32_t done = 0;
    for (int64_t t0 = 0; t0 < tokens; t0 += kRowsBlock * kRowsEach) {
        int64_t y[kRowsEach];
        int32_t mine = 0;
        const int64_t first = t0 + (int64_t)threadIdx.x * kRowsEach;
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            y[i] = first + i < tokens ? gp(labels)[first + i] : ignore;
            mine += y[i] != ignore;
        }
        int32_t total, j = done + block_prefix(mine, total);
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            if (first + i >= tokens) break;
            if (y[i] == ignore) {
                gp(loss)[first + i] = 0.0f;
                gp(lse)[first + i] = 0.0f;
            } else {
                gp(at)[j] = (int32_t)(first + i);
                gp(label)[j] = label_in(y[i], vocab);
                gp(zt)[j] = __builtin_nanf("");  // until the label's logit is there
                ++j;
            }
        }
        done += total;
    }
    if (threadIdx.x == 0) *gp(count) = done;
}

// lse and loss of the tokens that count from their parts: with S the sum of exp(l - M)
// over all columns but the label's, and d = M - l_label,
//   loss = log(1 + S exp(d)) = d + log(S + exp(-d)),  lse = l_label + loss.
// A workgroup takes kBlock / each rows, `each` (a power of two) threads a row.
__global__ __launch_bounds__(kBlock) void xent_join_kernel(const f32x2* __restrict__ part, int64_t stride, int64_t parts, int each,
                                                           const int32_t* __restrict__ count, const int32_t* __restrict__ at,
                                                           const float* __restrict__ zt, float* __restrict__ loss,
                                                           float* __restrict__ lse) {
    __shared__ f32x2 sums[kBlock];
    const int per = kBlock / each, r = threadIdx.x % per;
    const int64_t rows = (int64_t)*gp(count);
    for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < rows; row0 += (int64_t)gridDim.x * per) {
        const int64_t row = row0 + r;
        float m = -__builtin_inff(), s = 0.0f;
        auto add = [&](const f32x2 v) {
            if (v[1] == 0.0f) return;  // an empty part
            const float top = fmaxf(m, v[0]);
            s = (s == 0.0f ? 0.0f : s * exp_fast(m - top)) + v[1] * exp_fast(v[0] - top);
            m = top;
        };
        if (row < rows)
#pragma unroll 4
            for (int64_t i = threadIdx.x / per; i < parts; i += each) add(reinterpret_cast<const gf32x2*>(gp(part))[i * stride + row]);
        for (int d = each / 2; d > 0; d /= 2) {
            __syncthreads();
            sums[threadIdx.x] = f32x2{m, s};
            __syncthreads();
            if ((int)threadIdx.x < d * per) add(sums[threadIdx.x + d * per]);
        }
        if ((int)threadIdx.x < per && row < rows) {
            const float l = gp(zt)[row], d = m - l;
            float v, whole;
            if (d > 0.0f) {
                const float e = logf(s + expf(-d));
                v = d + e;
                whole = m + e;
            } else {  // also without another column (d = -inf), and where l is NaN
                v = l < __builtin_inff() ? log1pf(s * expf(d)) : __builtin_nanf("");
                whole = l == l ? l + v : m + logf(s);
            }
            const int32_t t = gp(at)[row];
            gp(loss)[t] = v;
            gp(lse)[t] = whole;
        }
    }
}

// The backward pass's view of the tokens: those that count in order, each token's place
// among them (-1: left out), the largest finite magnitude of their losses' weights, and
// each row's {lse, weight over that, label, expm1(-loss)} (without a loss 1). One workgroup.
__global__ __launch_bounds__(kRowsBlock) void xent_back_rows_kernel(const int64_t* __restrict__ labels, int64_t tokens, int64_t ignore,
                                                                    int64_t vocab, const float* __restrict__ lse,
                                                                    const float* __restrict__ loss,
                                                                    const float* __restrict__ dloss, int64_t dloss_count,
                                                                    int32_t* __restrict__ count, int32_t* __restrict__ at,
                                                                    int32_t* __restrict__ place, int32_t* __restrict__ second,
                                                                    f32x4* __restrict__ info) {
    __shared__ float tops[kRowsBlock / kWave];
    float top = 0.0f;
    for (int64_t t = threadIdx.x; t < tokens; t += kRowsBlock)
        if (gp(labels)[t] != ignore) {
            const float d = fabsf(gp(dloss)[dloss_count == 1 ? 0 : t]);
            if (d < __builtin_inff()) top = fmaxf(top, d);
        }
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    if ((threadIdx.x & (kWave - 1)) == 0) tops[threadIdx.x / kWave] = top;
    __syncthreads();
    for (int i = 0; i < kRowsBlock / kWave; ++i) top = fmaxf(top, tops[i]);
    if (top == 0.0f) top = 1.0f;
    int32_t done = 0;
    for (int64_t t0 = 0; t0 < tokens; t0 += kRowsBlock * kRowsEach) {
        int64_t y[kRowsEach];
        int32_t mine = 0;
        const int64_t first = t0 + (int64_t)threadIdx.x * kRowsEach;
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            y[i] = first + i < tokens ? gp(labels)[first + i] : ignore;
            mine += y[i] != ignore;
        }
        int32_t total, j = done + block_prefix(mine, total);
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            const int64_t t = first + i;
            if (t >= tokens) break;
            if (y[i] == ignore) {
                gp(place)[t] = -1;
                continue;
            }
            const int32_t label = label_in(y[i], vocab);
            const float d = gp(dloss)[dloss_count == 1 ? 0 : t];
            const float known = loss ? expm1f(-gp(loss)[t]) : 1.0f, own = loss && known > 0.0f ? 0.0f : known;
            gp(place)[t] = j;
            gp(at)[j] = (int32_t)t;
            reinterpret_cast<gf32x4*>(gp(info))[j] =
                f32x4{gp(lse)[t], label < 0 ? __builtin_nanf("") : d / top, __builtin_bit_cast(float, label), own};
            ++j;
        }
        done += total;
    }
    if (threadIdx.x == 0) {
        *gp(count) = done;
        reinterpret_cast<gfloat*>(gp(count))[1] = top;
        gp(count)[2] = 2 * done;  // rows with second terms
    }
    if (second)
        for (int64_t t = threadIdx.x; t < done; t += kRowsBlock) gp(second)[t] = (int32_t)(done + t);
}

// The rows of x that count, packed, with zeros up to ld (and once more behind them, for second
// terms, if count is given); zeros in the others' rows of dx.
__global__ __launch_bounds__(kBlock) void xent_pack_kernel(const uint16_t* __restrict__ x, int64_t tokens, int64_t cols, int64_t ldx,
                                                           const int32_t* __restrict__ place, uint16_t* __restrict__ packed, int64_t ld,
                                                           uint16_t* __restrict__ dx, int64_t lddx, const int32_t* __restrict__ count) {
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int32_t j = gp(place)[t];
        if (j < 0 && !dx) continue;
        for (int64_t c = threadIdx.x * 8; c < ld; c += kBlock * 8) {
            float v[8] = {};
            if (j >= 0) {
                const u32x4 w = load_raw8(x + t * ldx + c, cols - c).w;
                *reinterpret_cast<gu32x4*>(gp(packed) + j * ld + c) = w;
                if (count) *reinterpret_cast<gu32x4*>(gp(packed) + ((int64_t)*gp(count) + j) * ld + c) = finite_of(w);
            } else {
                store8(dx + t * lddx + c, cols - c, v);
            }
        }
    }
}

}  // namespace

extern "C" {

size_t coat_linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, int32_t aligned) {
    if (tokens < 1 || vocab < 1 || cols < 0 || tokens > kMaxDim || vocab > kMaxDim || cols > kMaxDim) return 0;
    return xent_layout(tokens, vocab, cols, aligned != 0).end;
}

int coat_linear_cross_entropy(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ldx, const uint16_t* w, int64_t vocab,
                              int64_t ldw, const int64_t* labels, int64_t ignore_index, float* loss, float* lse, void* workspace,
                              size_t workspace_bytes, coat_stream_t stream) {
    int rc = check_xent(x, tokens, cols, ldx, w, vocab, ldw, labels, loss, lse);
    if (rc || tokens == 0) return rc;
    const bool ready = tiles_gather(x, tokens, ldx, cols) && tiles_take(w, ldw, cols);
    const XentLayout l = xent_layout(tokens, vocab, cols, ready);
    if (!workspace || workspace_bytes < l.end) return COAT_EINVAL;
    if (!aligned(workspace, 256)) return COAT_EALIGN;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    char* const ws = static_cast<char*>(workspace);
    int32_t* const count = reinterpret_cast<int32_t*>(ws + l.count);
    int32_t* const at = reinterpret_cast<int32_t*>(ws + l.at);
    int32_t* const label = reinterpret_cast<int32_t*>(ws + l.label);
    float* const zt = reinterpret_cast<float*>(ws + l.zt);
    f32x2* const part = reinterpret_cast<f32x2*>(ws + l.part);
    Product16 p{x, w, ldx, ldw, at, count, nullptr, tokens, vocab, cols};
    hipLaunchKernelGGL(xent_rows_kernel, dim3(1), dim3(kRowsBlock), 0, st, labels, tokens, ignore_index, vocab, count, at, label, zt, loss, lse);
    if ((rc = launch_status())) return rc;
    if (!ready && l.plan.way != Way16::kPlain && l.plan.way != Way16::kFew) {
        uint16_t *const px = reinterpret_cast<uint16_t*>(ws + l.x), *const pw = reinterpret_cast<uint16_t*>(ws + l.w);
        if ((rc = launch_pack(Pack{x, tokens, ldx, at, count, px}, Pack{w, vocab, ldw, nullptr, nullptr, pw}, cols, st))) return rc;
        p.a = px;
        p.b = pw;
        p.lda = p.ldb = packed_ld(cols);
        p.a_rows = nullptr;
    }
    if ((rc = launch_product<false, false>(p, l.plan, nullptr, LogSumOut{label, zt, part, tokens}, st))) return rc;
    // threads a row: the whole loss of 8192 x 32000 x 64 takes 177 us with 16 and 186 with 64, of
    // 1023 x 50257 x 64 62 and 50 (53 with 128), of 64 x 50257 x 64 32, 21 and 19
    const int each = tokens >= 4096 ? 16 : (tokens >= 512 ? 64 : 128);
    const int64_t groups = div_up(tokens, kBlock / each);
    hipLaunchKernelGGL(xent_join_kernel, dim3((unsigned)(groups < 16 * kCUs ? groups : 16 * kCUs)), dim3(kBlock), 0, st, part, tokens, l.parts,
                       each, count, at, zt, loss, lse);
    return launch_status();
}

size_t coat_linear_cross_entropy_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, int32_t aligned) {
    if (tokens < 1 || vocab < 1 || cols < 0 || tokens > kMaxDim || vocab > kMaxDim || cols > kMaxDim) return 0;
    return xent_backward_layout(tokens, vocab, cols, aligned != 0).end;
}

int coat_linear_cross_entropy_backward_loss(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ldx, const uint16_t* w, int64_t vocab,
                                            int64_t ldw, const int64_t* labels, int64_t ignore_index, const float* lse, const float* loss,
                                            const float* dloss, int64_t dloss_count, uint16_t* dx, int64_t lddx, uint16_t* dw, int64_t lddw,
                                            void* workspace, size_t workspace_bytes, coat_stream_t stream) {
    int rc = check_xent_backward(x, tokens, cols, ldx, w, vocab, ldw, labels, lse, dloss, dloss_count, dx, lddx, dw, lddw);
    if (!rc && !aligned(loss, 4)) rc = COAT_EALIGN;
    if (rc || cols == 0) return rc;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (tokens == 0) {
        if (!dw) return COAT_OK;
        return launch_product<true, true>(Product16{x, x, 8, 8, nullptr, nullptr, nullptr, vocab, cols, 0}, plan16_of(vocab, cols, 0, false, true, true),
                                          nullptr, ScaledOut{nullptr, 0.0f, dw, lddw}, st);
    }
    const bool ready = tiles_gather(x, tokens, ldx, cols) && tiles_take(w, ldw, cols);
    const XentBackwardLayout l = xent_backward_layout(tokens, vocab, cols, ready);
    if (!workspace || workspace_bytes < l.end) return COAT_EINVAL;
    if (!aligned(workspace, 256)) return COAT_EALIGN;
    char* const ws = static_cast<char*>(workspace);
    int32_t* const count = reinterpret_cast<int32_t*>(ws + l.count);
    const float* const top = reinterpret_cast<const float*>(ws + l.count) + 1;
    int32_t* const at = reinterpret_cast<int32_t*>(ws + l.at);
    int32_t* const place = reinterpret_cast<int32_t*>(ws + l.place);
    int32_t* const second = l.two ? reinterpret_cast<int32_t*>(ws + l.second) : nullptr;
    const int32_t* const two = l.two ? count : nullptr;
    f32x4* const info = reinterpret_cast<f32x4*>(ws + l.info);
    uint16_t* const px = reinterpret_cast<uint16_t*>(ws + l.x);
    uint16_t* const g = reinterpret_cast<uint16_t*>(ws + l.g);
    float* const acc = reinterpret_cast<float*>(ws + l.acc);
    float* const sums = reinterpret_cast<float*>(ws + l.part);
    hipLaunchKernelGGL(xent_back_rows_kernel, dim3(1), dim3(kRowsBlock), 0, st, labels, tokens, ignore_index, vocab, lse, loss, dloss, dloss_count,
                       count, at, place, second, info);
    hipLaunchKernelGGL(xent_pack_kernel, dim3((unsigned)(tokens < 64 * kCUs ? tokens : 64 * kCUs)), dim3(kBlock), 0, st, x, tokens, cols, ldx,
                       place, px, l.ld_x, dx, lddx, two);
    if ((rc = launch_status())) return rc;
    if (!ready) {
        uint16_t* const pw = reinterpret_cast<uint16_t*>(ws + l.w);
        if ((rc = launch_pack(Pack{w, vocab, ldw, nullptr, nullptr, pw}, Pack{}, cols, st))) return rc;
        w = pw;
        ldw = packed_ld(cols);
    }
    for (int64_t v0 = 0; v0 < vocab; v0 += l.piece) {
        const int64_t v1 = v0 + l.piece < vocab ? v0 + l.piece : vocab;
        const uint16_t* const wp = w + v0 * ldw;
        const XentPiece plans = xent_piece_plans(tokens, v1 - v0, cols, l.two);
        const Product16 logits{px, wp, l.ld_x, ldw, nullptr, count, nullptr, tokens, v1 - v0, cols};
        rc = two ? launch_product<false, false>(logits, plans.logits, sums, GradOut<true>{info, g, l.ld_g, v0, two, 0}, st)
                 : launch_product<false, false>(logits, plans.logits, sums, GradOut<false>{info, g, l.ld_g, v0, nullptr, 0}, st);
        if (rc) return rc;
        if (dx) {
            uint16_t* const to = v1 == vocab ? dx : nullptr;
            Product16 p{g, wp, l.ld_g, ldw, nullptr, count, nullptr, tokens, cols, v1 - v0};
            if (two) {
                const PiecesOut<true> first{top, at, nullptr, lddx, acc, l.ld_x, v0 == 0, 0.0f, false};
                if ((rc = launch_product<false, true>(p, plans.dx, sums, first, st))) return rc;
                p.a_rows = second;
                const PiecesOut<true> left{top, at, to, lddx, acc, l.ld_x, false, 0.0f, true};
                rc = launch_product<false, true>(p, plans.dx, sums, left, st);
            } else {
                const PiecesOut<false> out{top, at, to, lddx, acc, l.ld_x, v0 == 0, 0.0f, false};
                rc = launch_product<false, true>(p, plans.dx, sums, out, st);
            }
            if (rc) return rc;
        }
        if (dw) {
            const int64_t rows = l.two ? 2 * tokens : tokens;
            const Product16 p{g, px, l.ld_g, l.ld_x, nullptr, nullptr, l.two ? count + 2 : count, v1 - v0, cols, rows};
            rc = launch_product<true, true>(p, plans.dw, sums, ScaledOut{top, 0.0f, dw + v0 * lddw, lddw}, st);
            if (rc) return rc;
        }
    }
    return COAT_OK;
}

int coat_linear_cross_entropy_backward(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ldx, const uint16_t* w, int64_t vocab,
                                       int64_t ldw, const int64_t* labels, int64_t ignore_index, const float* lse, const float* dloss,
                                       int64_t dloss_count, uint16_t* dx, int64_t lddx, uint16_t* dw, int64_t lddw, void* workspace,
                                       size_t workspace_bytes, coat_stream_t stream) {
    return coat_linear_cross_entropy_backward_loss(x, tokens, cols, ldx, w, vocab, ldw, labels, ignore_index, lse, nullptr, dloss, dloss_count,
                                                   dx, lddx, dw, lddw, workspace, workspace_bytes, stream);
}

}  // extern "C"

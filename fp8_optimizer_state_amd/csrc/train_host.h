// Host-side logic of the training products (linear layer, dropout, cross entropy of
// a vocabulary projection) that touches no GPU: argument checks, sizes and
// workspaces. Plain C++ with no HIP dependency, so that the same code runs in a
// host-only driver under AddressSanitizer and UndefinedBehaviorSanitizer.
#pragma once

#include "ops_host.h"

namespace {

// Dropout: an element is dropped if its 16 bits are under the threshold, which is
// at most 65535 (p rounded to a multiple of 2^-16, something always kept).
inline uint32_t drop_threshold(float p) {
    const double t = (double)p * 65536.0 + 0.5;
    return t >= 65536.0 ? 65535u : (uint32_t)t;
}
inline float drop_factor(uint32_t threshold) { return (float)(65536.0 / (65536.0 - (double)threshold)); }

inline int check_epilogue(const coat_epilogue* e) {
    if (!e) return COAT_EINVAL;
    if (e->act < COAT_ACT_NONE || e->act > COAT_ACT_SILU || !finite_f(e->scale)) return COAT_EINVAL;
    if (!(e->p >= 0.0f && e->p < 1.0f) || (e->p > 0.0f && !e->rng)) return COAT_EINVAL;
    if (!finite_f(e->scale * drop_factor(drop_threshold(e->p)))) return COAT_EINVAL;
    if (!aligned(e->rng, 8)) return COAT_EALIGN;
    return COAT_OK;
}

// A matrix that may be absent; rows = 0 or cols = 0 needs no address.
inline int check_optional(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
    if (!p) return COAT_OK;
    const int rc = check_matrix(rows, cols, ld, dtype);
    if (rc) return rc;
    return aligned(p, type_bytes(dtype)) ? COAT_OK : COAT_EALIGN;
}
inline int check_present(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
    if (!p && rows > 0 && cols > 0) return COAT_EINVAL;
    const int rc = check_matrix(rows, cols, ld, dtype);
    if (rc) return rc;
    return aligned(p, type_bytes(dtype)) ? COAT_OK : COAT_EALIGN;
}
// The first error among several checks, invalid arguments before alignments.
inline int first_error(std::initializer_list<int> all) {
    int align = COAT_OK;
    for (const int rc : all) {
        if (rc == COAT_EINVAL) return rc;
        if (rc) align = rc;
    }
    return align;
}

inline int check_linear(const void* x, int64_t m, int64_t k, int64_t ldx, const void* w, int64_t n, int64_t ldw,
                        const coat_epilogue* e, const void* bias, int32_t bias_type, const void* residual, int64_t ldr,
                        const void* z, int64_t ldz, const void* y, int64_t ldy, int32_t y_type) {
    if (!type_ok(bias_type)) return COAT_EINVAL;
    return first_error({check_epilogue(e), check_present(x, m, k, ldx, COAT_BF16), check_present(w, n, k, ldw, COAT_BF16),
                        check_present(y, m, n, ldy, y_type), check_optional(residual, m, n, ldr, y_type),
                        check_optional(z, m, n, ldz, COAT_BF16),
                        aligned(bias, type_bytes(bias_type)) ? COAT_OK : COAT_EALIGN});
}

inline int check_linear_backward(const void* dy, int64_t lddy, int32_t dy_type, const void* x, int64_t m, int64_t k, int64_t ldx,
                                 const void* w, int64_t n, int64_t ldw, const coat_epilogue* e, const void* z, int64_t ldz,
                                 const void* dx, int64_t lddx, const void* dw, int64_t lddw, const void* dbias,
                                 int32_t dbias_type) {
    if (!type_ok(dbias_type) || (!dx && !dw && !dbias && m > 0 && n > 0 && k > 0)) return COAT_EINVAL;
    const int rc = check_epilogue(e);
    if (rc == COAT_EINVAL) return rc;
    if (e->act != COAT_ACT_NONE && !z && m > 0 && n > 0) return COAT_EINVAL;
    return first_error({rc, check_present(dy, m, n, lddy, dy_type), dw ? check_present(x, m, k, ldx, COAT_BF16) : check_optional(x, m, k, ldx, COAT_BF16),
                        dx ? check_present(w, n, k, ldw, COAT_BF16) : check_optional(w, n, k, ldw, COAT_BF16),
                        check_optional(z, m, n, ldz, COAT_BF16), check_optional(dx, m, k, lddx, COAT_BF16),
                        check_optional(dw, n, k, lddw, COAT_BF16), aligned(dbias, type_bytes(dbias_type)) ? COAT_OK : COAT_EALIGN,
                        m > kMaxDim || n > kMaxDim || k > kMaxDim || m < 0 || n < 0 || k < 0 ? COAT_EINVAL : COAT_OK});
}

inline int check_dropout(const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t x_type, const void* residual,
                         int64_t ldr, float scale, float p, const int64_t* rng, const void* y, int64_t ldy, int32_t y_type) {
    if (!finite_f(scale) || !(p >= 0.0f && p < 1.0f) || (p > 0.0f && !rng)) return COAT_EINVAL;
    if (!finite_f(scale * drop_factor(drop_threshold(p)))) return COAT_EINVAL;
    return first_error({check_present(x, rows, cols, ldx, x_type), check_present(y, rows, cols, ldy, y_type),
                        check_optional(residual, rows, cols, ldr, y_type), aligned(rng, 8) ? COAT_OK : COAT_EALIGN});
}

// ------------------------------------------------------------------ products of bf16 matrices

// How a product m x n over k is computed: in tiles of 256 x 256 or 128 x 128, whose k
// may be dealt to `splits` workgroups of per_split steps of 64 values (their sums go
// to the workspace, `stride` apart in rows of ld, and are added by another kernel), in
// 16 rows of B a workgroup (kFew), or one 32 x 32 tile a wavefront straight from memory.
enum class Way16 { kPlain, kTile256, kTile128, kFew };
struct Plan16 {
    Way16 way;
    uint32_t tiles_m, tiles_n, splits, per_split;
    int64_t ld, stride;
};

constexpr int64_t kMaxLd = int64_t(1) << 22;  // of a tile's operand: 256 rows' bytes stay within 32 bits

// Whether tiles can take an operand as it lies: rows of whole 16-byte chunks.
inline bool tiles_take(const void* p, int64_t ld, int64_t cols) {
    return aligned16(p) && ld % 8 == 0 && cols % 8 == 0 && ld < kMaxLd;
}

// Estimated microseconds of 128 x 128 tiles with their k in `splits` parts: a compute
// unit takes 0.83 a step of 64 values with two of them, 0.47 with one, and 4.3 a round to
// begin and end; with splits the partial sums' way out and back on top. Measured:
// 1500 x 5120 x 13824 (480 tiles, 216 steps) 179, 4096 x 5120 x 5120 (three rounds of 80)
// 208, 333 x 5120 x 13824 (120 tiles) 104 in one part, 64 in two, 55 in four.
inline double tile128x_time(int64_t tiles, int64_t m, int64_t ld, int64_t steps, int64_t splits) {
    const int64_t items = tiles * splits, each = div_up(steps, splits);
    const double work = items <= kCUs ? 0.47 * (double)each + 4.3 : (double)div_up(items, 2 * kCUs) * (0.83 * (double)each + 4.3);
    return splits == 1 ? work : work + 4.0 + (double)splits * (double)m * (double)ld / 1e6;
}
// The same of 256 x 256 tiles: 1.3 a step with all compute units at work (the card's power
// sets the clock), 1.0 with half of them, and 14 to write a tile out. Measured: 16384 x
// 13824 x 5120 (14 rounds of 80) 1629, 4096 x 5120 x 5120 (two rounds) 233, 1023 x 50257
// x 768 (four rounds of 12) 124 and 100 in small tiles.
inline double tile256x_time(int64_t tiles, int64_t steps) {
    const int64_t left = tiles % kCUs;
    const double step = tiles > kCUs ? 1.3 : (left <= kCUs / 2 ? 1.0 : 0.7 + 0.6 * (double)left / kCUs);
    return (double)(tiles / kCUs) * (1.3 * (double)steps + 14.0) + (left ? step * (double)steps + 14.0 : 0.0);
}

// can_split: the sums of a part of k may leave on their own. tall_a, tall_b: an operand
// whose rows in memory are those of k. large: whether tiles of 256 x 256 may be taken (products
// of second terms have no code for them: their few rows or columns never pay for one).
inline Plan16 plan16_of(int64_t m, int64_t n, int64_t k, bool can_split, bool tall_a, bool tall_b, bool large = true) {
    Plan16 p{Way16::kPlain, 0, 0, 1, 0, 0, 0};
    if (m < 1 || n < 1 || k < 1 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return p;
    if ((tall_a ? m : k) >= kMaxLd || (tall_b ? n : k) >= kMaxLd) return p;
    const bool rows = !tall_a && !tall_b;
    // Few rows of A. Each 16 rows of B read all of A again, so that more rows pay only where
    // B is small: 4 x 13824 x 5120 takes 30 us this way and 29 in tiles, 16 40 and 30, 1 x
    // 4096 x 4096 9 and 17. Where tiles cannot share k they pay later: the loss of 1 x
    // 32000 x 4096 takes 57 us and 72, of 16 x 32000 x 4096 71 and 54, of 16 x 13824 x 5120
    // 48 and 52, of 16 x 5120 x 13824 59 and 110.
    if (rows && m <= 16 && (m <= 4 || (can_split ? n * k <= (1 << 24) : n <= 25600))) {
        p.way = Way16::kFew;
        return p;
    }
    if (div_up(m, 128) * div_up(n, 128) > 0x3FFFFFFF) return p;
    const int64_t steps = div_up(k, 64), tiles256 = div_up(m, 256) * div_up(n, 256), tiles = div_up(m, 128) * div_up(n, 128);
    p.ld = div_up(n, 64) * 64;
    p.stride = m * p.ld;
    int64_t best = 1;
    if (can_split) {
        for (int64_t s = 2; s <= steps / 4 && tiles * s <= 2 * kCUs; ++s)
            if (tile128x_time(tiles, m, p.ld, steps, s) < tile128x_time(tiles, m, p.ld, steps, best)) best = s;
    }
    p.per_split = (uint32_t)div_up(steps, best);
    p.splits = (uint32_t)div_up(steps, p.per_split);
    p.way = Way16::kTile128;
    p.tiles_m = (uint32_t)div_up(m, 128);
    p.tiles_n = (uint32_t)div_up(n, 128);
    if (large && tile256x_time(tiles256, steps) < tile128x_time(tiles, m, p.ld, steps, best)) {
        p.way = Way16::kTile256;
        p.tiles_m = (uint32_t)div_up(m, 256);
        p.tiles_n = (uint32_t)div_up(n, 256);
        p.splits = 1;
        p.per_split = (uint32_t)steps;
    }
    return p;
}
inline size_t plan16_bytes(const Plan16& p) {
    return p.splits > 1 ? align_up((size_t)p.splits * (size_t)p.stride * sizeof(float), 256) : 0;
}

// An operand that tiles do not take is copied to rows of whole 128 bytes first, with
// zeros behind its columns.
inline int64_t packed_ld(int64_t cols) { return div_up(cols, 64) * 64; }
inline size_t packed_bytes(int64_t rows, int64_t cols) { return align_up((size_t)rows * (size_t)packed_ld(cols) * 2, 256); }

struct LinearLayout {
    Plan16 plan;
    size_t part, x, w, end;
};
inline LinearLayout linear_layout(int64_t m, int64_t n, int64_t k, bool ready) {
    LinearLayout l;
    l.plan = plan16_of(m, n, k, true, false, false);
    const bool pack = !ready && l.plan.way != Way16::kPlain && l.plan.way != Way16::kFew;
    l.part = 0;
    l.x = plan16_bytes(l.plan);
    l.w = l.x + (pack ? packed_bytes(m, k) : 0);
    l.end = l.w + (pack ? packed_bytes(n, k) : 0);
    return l;
}

// ------------------------------------------------------------------ backward pass of the linear layer

// Rows of a band, whose part of the bias gradient one workgroup adds up: 64, or fewer
// where those would leave compute units without work (1031 x 2731: 32 us with 64, 9 with 8).
inline int64_t bias_band(int64_t m, int64_t n) {
    int64_t band = 64;
    while (band > 8 && div_up(m, band) * div_up(n, 512) < 4 * kCUs) band /= 2;
    return band;
}

// A rounding to bf16 on the way to a gradient and the one that stores it are independent and
// alike: together they leave the gradients off by sqrt 2 of what storing leaves, in the mean
// of squares and at any size. Over many values that is what every call sees (1.4 from 4096
// on); over few it spreads (1 x 8 values up to 2.6 times, 64 to 1024 1.5 to 1.6; a loss of 1
// token 1.6, of 16 1.3, of 64 1.1). Where there are few the products take what the rounding
// leaves as well, a second bf16 term, and are off by 1.0 times: of up to 2048 values, and of the
// logits of up to 16 tokens, whose labels' own gradients are most of them. So the error steps
// from 1.0 to 1.5 at 2049 values; a limit further up would cost more: launches (the gradients of
// 16 x 128 values 19 -> 31 us), twice the products over the tokens, and reading the weights once
// more (a loss of 1 x 32000 x 4096 with its gradients 208 -> 260 us).
constexpr int64_t kTwoTermValues = 2048, kTwoTermTokens = 16;
inline bool dz_takes_two_terms(int64_t m, int64_t n) { return m <= kTwoTermValues && n <= kTwoTermValues && m * n <= kTwoTermValues; }
inline bool xent_takes_two_terms(int64_t tokens, int64_t vocab) { return tokens <= kTwoTermTokens || dz_takes_two_terms(tokens, vocab); }

// Workspace of the backward pass: dz in bf16 with rows of whole 128 bytes (its second terms
// behind it), the partial sums of the bias gradient and of the products, copies of x
// and w, and the sums of dx over the two terms.
struct LinearBackwardLayout {
    Plan16 plan_dx, plan_dw, plan_dw_two;
    int64_t ld_dz;
    size_t dz, bias, part, x, w, acc, end;
};
inline LinearBackwardLayout linear_backward_layout(int64_t m, int64_t n, int64_t k, bool ready) {
    LinearBackwardLayout l;
    const bool two = dz_takes_two_terms(m, n);
    l.plan_dx = plan16_of(m, k, n, true, false, true, !two);
    l.plan_dw = plan16_of(n, k, m, true, true, true);
    l.plan_dw_two = plan16_of(n, k, 2 * m, true, true, true);
    size_t part = plan16_bytes(l.plan_dx);
    if (plan16_bytes(l.plan_dw) > part) part = plan16_bytes(l.plan_dw);
    if (two && plan16_bytes(l.plan_dw_two) > part) part = plan16_bytes(l.plan_dw_two);
    l.ld_dz = packed_ld(n);
    l.dz = 0;
    l.bias = packed_bytes(two ? 2 * m : m, n);
    l.part = l.bias + align_up((size_t)div_up(m, bias_band(m, n)) * (size_t)l.ld_dz * sizeof(float), 256);
    l.x = l.part + part;
    l.w = l.x + (two ? packed_bytes(2 * m, k) : (ready ? 0 : packed_bytes(m, k)));
    l.acc = l.w + (ready ? 0 : packed_bytes(n, k));
    l.end = l.acc + (two ? 2 * packed_bytes(m, k) : 0);
    return l;
}

// ------------------------------------------------------------------ cross entropy of a vocabulary projection

inline int check_xent(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* w, int64_t vocab, int64_t ldw,
                      const int64_t* labels, const float* loss, const float* lse) {
    if (vocab < 1 || (tokens > 0 && (!labels || !loss || !lse))) return COAT_EINVAL;
    return first_error({check_present(x, tokens, cols, ldx, COAT_BF16), check_present(w, vocab, cols, ldw, COAT_BF16),
                        aligned(labels, 8) ? COAT_OK : COAT_EALIGN, aligned(loss, 4) && aligned(lse, 4) ? COAT_OK : COAT_EALIGN});
}

inline int check_xent_backward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* w, int64_t vocab, int64_t ldw,
                               const int64_t* labels, const float* lse, const float* dloss, int64_t dloss_count, const void* dx,
                               int64_t lddx, const void* dw, int64_t lddw) {
    if (dloss_count != 1 && dloss_count != tokens) return COAT_EINVAL;
    if (tokens > 0 && !dloss) return COAT_EINVAL;
    if (!dx && !dw && tokens > 0 && cols > 0) return COAT_EINVAL;
    return first_error({check_xent(x, tokens, cols, ldx, w, vocab, ldw, labels, lse, lse), check_optional(dx, tokens, cols, lddx, COAT_BF16),
                        check_optional(dw, vocab, cols, lddw, COAT_BF16), aligned(dloss, 4) ? COAT_OK : COAT_EALIGN});
}

// Columns of a partial log sum, by the way the logits are computed.
constexpr int64_t log_sum_width(Way16 way) { return way == Way16::kTile256 ? 128 : (way == Way16::kTile128 ? 64 : (way == Way16::kFew ? 16 : 32)); }

// Workspace of the loss: number of tokens that count, their places and labels, the
// logits of their labels, a (maximum, sum) for each of them and each part of the
// vocabulary, and copies of x and w.
struct XentLayout {
    Plan16 plan;
    int64_t parts;
    size_t count, at, label, zt, part, x, w, end;
};
inline XentLayout xent_layout(int64_t tokens, int64_t vocab, int64_t cols, bool ready) {
    XentLayout l;
    const size_t t = (size_t)tokens;
    l.plan = plan16_of(tokens, vocab, cols, false, false, false);
    const bool pack = !ready && l.plan.way != Way16::kPlain && l.plan.way != Way16::kFew;
    l.parts = div_up(vocab, log_sum_width(l.plan.way));
    l.count = 0;
    l.at = 256;
    l.label = l.at + align_up(t * 4, 256);
    l.zt = l.label + align_up(t * 4, 256);
    l.part = l.zt + align_up(t * 4, 256);
    l.x = l.part + align_up((size_t)l.parts * t * 8, 256);
    l.w = l.x + (pack ? packed_bytes(tokens, cols) : 0);
    l.end = l.w + (pack ? packed_bytes(vocab, cols) : 0);
    return l;
}

// Whether the loss's tiles can gather x's rows as they lie: their byte offsets have 32 bits.
inline bool tiles_gather(const void* x, int64_t tokens, int64_t ldx, int64_t cols) {
    return tiles_take(x, ldx, cols) && tokens * ldx < (int64_t(1) << 31);
}

// Columns of the vocabulary that the backward pass takes at a time. The gradients of
// a piece's logits are 2^27 numbers (256 MB) or 2048 columns wide; pieces are of equal
// size. 8192 x 32000 x 5120 takes 6300 us in pieces of 2^26, 5900 of 2^27 and 5740 of
// 2^28, which would be all of its logits.
inline int64_t xent_piece(int64_t tokens, int64_t vocab) {
    int64_t most = ((int64_t)1 << 27) / (tokens > 0 ? tokens : 1) / 256 * 256;
    if (most < 2048) most = 2048;
    if (most > kMaxLd / 2) most = kMaxLd / 2;
    if (most >= vocab) return vocab;
    return div_up(div_up(vocab, div_up(vocab, most)), 256) * 256;
}

// Workspace of the backward pass: number of tokens that count, the largest weight of a
// loss and twice that number, the tokens' places in the packed rows and back, the rows of
// their second terms if they have any, what a row of logits needs, the packed rows of x and a piece's
// gradients (each twice with second terms), the sums of dx over pieces and terms, the
// partial sums of products and a copy of w.
struct XentBackwardLayout {
    bool two;
    int64_t piece, ld_x, ld_g;
    size_t count, at, place, second, info, x, g, acc, part, w, end;
};
// The products of a piece of `width` columns.
struct XentPiece {
    Plan16 logits, dx, dw;
};
inline XentPiece xent_piece_plans(int64_t tokens, int64_t width, int64_t cols, bool two) {
    return XentPiece{plan16_of(tokens, width, cols, true, false, false, !two), plan16_of(tokens, cols, width, true, false, true, !two),
                     plan16_of(width, cols, two ? 2 * tokens : tokens, true, true, true)};
}
inline XentBackwardLayout xent_backward_layout(int64_t tokens, int64_t vocab, int64_t cols, bool ready) {
    XentBackwardLayout l;
    const size_t t = (size_t)tokens;
    l.two = xent_takes_two_terms(tokens, vocab);
    l.piece = xent_piece(tokens, vocab);
    l.ld_x = packed_ld(cols);
    l.ld_g = packed_ld(l.piece);
    size_t part = 0;
    for (const int64_t width : {l.piece, vocab - (vocab - 1) / l.piece * l.piece}) {
        const XentPiece p = xent_piece_plans(tokens, width, cols, l.two);
        for (const Plan16& q : {p.logits, p.dx, p.dw})
            if (plan16_bytes(q) > part) part = plan16_bytes(q);
    }
    const size_t rows = l.two ? 2 * t : t;
    l.count = 0;
    l.at = 256;
    l.place = l.at + align_up(t * 4, 256);
    l.second = l.place + align_up(t * 4, 256);
    l.info = l.second + (l.two ? align_up(t * 4, 256) : 0);
    l.x = l.info + align_up(t * 16, 256);
    l.g = l.x + align_up(rows * (size_t)l.ld_x * 2, 256);
    l.acc = l.g + align_up(rows * (size_t)l.ld_g * 2, 256);
    l.part = l.acc + (l.two || l.piece < vocab ? align_up(t * (size_t)l.ld_x * 4, 256) : 0);
    l.w = l.part + part;
    l.end = l.w + (ready ? 0 : packed_bytes(vocab, cols));
    return l;
}

}  // namespace

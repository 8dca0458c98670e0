// Host-side logic of the layer-input operators that touches no GPU: sizes,
// argument checks and launch shapes. Plain C++ with no HIP dependency, so that
// the same code runs in a host-only driver under AddressSanitizer and
// UndefinedBehaviorSanitizer.
#pragma once

#include <float.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "coat_fp8.h"
#include "coat_host.h"

namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFF;
constexpr int kCUs = 256;  // of an MI355X; launch shapes that decide an order of sums use this, not the device's count

constexpr int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch of `count` workgroups, numbered x first. One axis of a grid holds fewer
// than 2^32 work-items, so more workgroups go over y; those behind `count` return.
struct Grid {
    uint32_t x, y;
};
inline Grid grid_xy(int64_t count, int64_t threads) {
    const int64_t most = 0xFFFFFFFFll / threads / 16 * 16;  // whole patches of 16 workgroups
    const int64_t x = count < most ? count : most;
    return Grid{(uint32_t)x, (uint32_t)div_up(count, x)};
}

constexpr int64_t mx4_code_bytes(int64_t k) { return 64 * div_up(k, 128); }
constexpr int64_t mx4_scale_bytes(int64_t k) { return 16 * div_up(k, 512); }

inline bool type_ok(int32_t t) { return t == COAT_BF16 || t == COAT_FP32; }
inline size_t type_bytes(int32_t t) { return t == COAT_FP32 ? 4 : 2; }

// ------------------------------------------------------------------ 4-bit codec and product

// A matrix of `rows` x `cols` elements with `ld` elements from row to row.
inline int check_matrix(int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim || ld < cols || !type_ok(dtype)) return COAT_EINVAL;
    if (rows > 0 && ld > (INT64_MAX / 8) / rows) return COAT_EINVAL;
    return COAT_OK;
}

inline int check_mx4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, const uint8_t* q,
                              const uint8_t* s, const uint8_t* q_t, const uint8_t* s_t) {
    const int rc = check_matrix(rows, cols, ld, dtype);
    if (rc) return rc;
    if ((q == nullptr) != (s == nullptr) || (q_t == nullptr) != (s_t == nullptr)) return COAT_EINVAL;
    if (rows == 0 || cols == 0) return COAT_OK;
    if (!x || (!q && !q_t)) return COAT_EINVAL;
    if (!aligned(x, type_bytes(dtype)) || !aligned16(q) || !aligned16(s) || !aligned16(q_t) || !aligned16(s_t))
        return COAT_EALIGN;
    return COAT_OK;
}

inline int check_mx4_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, const void* x,
                                int64_t ld, int32_t dtype) {
    const int rc = check_matrix(rows, cols, ld, dtype);
    if (rc) return rc;
    if (rows == 0 || cols == 0) return COAT_OK;
    if (!x || !q || !s) return COAT_EINVAL;
    if (!aligned(x, type_bytes(dtype)) || !aligned16(q) || !aligned16(s)) return COAT_EALIGN;
    return COAT_OK;
}

inline int check_mx4_matmul(const uint8_t* a_q, const uint8_t* a_s, int64_t m, const uint8_t* b_q, const uint8_t* b_s,
                            int64_t n, int64_t k, const void* y, int64_t ld, int32_t dtype) {
    const int rc = check_matrix(m, n, ld, dtype);
    if (rc) return rc;
    if (k < 0 || k > kMaxDim) return COAT_EINVAL;
    if (m == 0 || n == 0) return COAT_OK;
    if (!y) return COAT_EINVAL;
    if (k > 0 && (!a_q || !a_s || !b_q || !b_s)) return COAT_EINVAL;
    if (!aligned16(a_q) || !aligned16(a_s) || !aligned16(b_q) || !aligned16(b_s) || !aligned(y, type_bytes(dtype)))
        return COAT_EALIGN;
    return COAT_OK;
}

// How a product is computed.
enum class Way { kSmall, kFew, kTile128, kTile256 };
struct Product {
    Way way;
    uint32_t tiles_m, tiles_n, splits, per_split;
    int64_t lw, part;  // of the partial sums: elements of a row and of a split
    int64_t head_m, head_n;  // kTile256: the part of y in large tiles; the rest, rows or columns, follows in small ones
};

// Estimated microseconds of 128 x 128 tiles with their k in `splits` parts: 0.27
// a step of 128 values in each round of workgroups and 3 to begin and end; with
// splits the second launch and the partial sums' way out and back on top.
// Measured: 128 x 13824 x 5120 (108 tiles) 16.3 in one part, 19.2 in two;
// 512 x 4096 x 4096 14.7 and 18.8; 333 x 5120 x 13824 36 and 32;
// 64 x 5120 x 13824 34 and, in six, 17.5.
inline double tile128_time(int64_t tiles, int64_t m, int64_t lw, int64_t steps, int64_t splits) {
    const double rounds = (double)div_up(tiles * splits, kCUs);
    const double work = rounds * (double)div_up(steps, splits) * 0.27 + 3.0;
    return splits == 1 ? work : work + 6.0 + 8.0 * (double)splits * (double)m * (double)lw / 3.5e6;
}

// The same of 256 x 256 tiles, with all compute units at work: 13824 x 5120 x 8191
// (five rounds of 64 steps) takes 294, 16384 x 13824 x 5120 (14 of 40) 550.
inline double tile256_time(int64_t tiles, int64_t steps) {
    return (double)div_up(tiles, kCUs) * (0.81 * (double)steps + 7.0);
}

inline Product product_of(int64_t m, int64_t n, int64_t k) {
    Product p{Way::kSmall, 0, 0, 1, 0, 0, 0, m, n};
    if (k == 0 || k >= (1 << 22)) return p;  // longer rows than 32-bit offsets within a tile reach
    // Few rows of A, which each 16 rows of B read again: 1 x 13824 x 5120 takes 9 us
    // this way and 15 in tiles, 16 12 and 15, 32 17 and 15; 24 x 10000 x 5120 12 and
    // 15, 16 x 32000 x 4096 20 and 15.
    if (m <= 32 && m * n * k <= int64_t(7) << 28) {
        p.way = Way::kFew;
        return p;
    }
    if (div_up(m, 128) * div_up(n, 128) > 0x3FFFFFFF) return p;
    const int64_t groups = div_up(k, 512);
    p.per_split = (uint32_t)groups;
    p.way = Way::kTile256;
    p.tiles_m = (uint32_t)div_up(m, 256);
    p.tiles_n = (uint32_t)div_up(n, 256);
    // Large tiles where they fill most of the card: 2048 x 5120 x 5120 (160 of them)
    // takes 40 us and 46 in small ones, 1500 x 5120 x 13824 (120) 87 and 77. Not where
    // one row of small ones covers a side, and half of each large one would lie past
    // it: 128 x 128256 x 5120 takes 108 and 89, 33 x 65536 x 5120 42 and 34, 2^18 x 33
    // x 8200 350 and 262; 129 x 65536 x 5120 49 and 52, 192 x 65536 x 5120 52 and 58.
    const int64_t large = (int64_t)p.tiles_m * p.tiles_n, steps = div_up(k, 128);
    if (large >= 160 && m > 128 && n > 128) {
        const int64_t full = large / kCUs * kCUs;  // of them in whole rounds of workgroups
        // A last round of few large tiles is done in small ones instead, if the
        // estimate gains 6 % or more (the card is bound by power, and a round with
        // few workgroups runs faster than the estimate): 4096 x 5120 x 5120 takes 86
        // us whole and 67 so, 2600 x 13824 x 5120 134 and 121, 13824 x 5120 x 16384
        // 582 and 556; 10000 x 7000 x 2000 (4.5 % by the estimate) 131 and 141.
        double best = 0.94 * tile256_time(large, steps);
        for (const bool rows : {true, false}) {
            const int64_t across = rows ? p.tiles_n : p.tiles_m, lines = full / across;
            if (lines == 0 || full == large) continue;
            const int64_t left_m = rows ? m - 256 * lines : m, left_n = rows ? n : n - 256 * lines;
            const double t = tile256_time(lines * across, steps) + 4.0 +
                             tile128_time(div_up(left_m, 128) * div_up(left_n, 128), 0, 0, steps, 1);
            if (t >= best) continue;
            best = t;
            p.head_m = rows ? 256 * lines : m;
            p.head_n = rows ? n : 256 * lines;
        }
        return p;
    }
    p.way = Way::kTile128;
    p.tiles_m = (uint32_t)div_up(m, 128);
    p.tiles_n = (uint32_t)div_up(n, 128);
    p.lw = div_up(n, 64) * 64;
    p.part = m * p.lw;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    int64_t best = 1;
    for (int64_t s = 2; s <= groups / 2 && tiles * s <= kCUs; ++s)
        if (tile128_time(tiles, m, p.lw, steps, s) < tile128_time(tiles, m, p.lw, steps, best)) best = s;
    p.per_split = (uint32_t)div_up(groups, best);
    p.splits = (uint32_t)div_up(groups, p.per_split);
    return p;
}

inline size_t product_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m < 1 || n < 1 || k < 1 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
    const Product p = product_of(m, n, k);
    return p.splits > 1 ? (size_t)p.splits * (size_t)p.part * sizeof(float) : 0;
}

// ------------------------------------------------------------------ block border

inline int check_border(const coat_border* b) {
    if (!b) return COAT_EINVAL;
    if (b->rows < 0 || b->rows > kMaxDim || b->cols < 1 || b->cols > COAT_BORDER_MAX_COLS || b->rows_per_gate < 1)
        return COAT_EINVAL;
    // the reciprocal root takes no subnormal, and beside a smaller eps the squares that fp32 loses would count
    if (!finite_f(b->eps) || !(b->eps >= FLT_MIN) || !finite_f(b->scale)) return COAT_EINVAL;
    if ((b->post != 0 && b->post != 1) || !type_ok(b->stream_type) || !type_ok(b->param_type) ||
        !type_ok(b->grad_type))
        return COAT_EINVAL;
    return COAT_OK;
}

inline int check_block_norm(const coat_border* b, const void* y, const void* r, const void* w_post, const void* w_pre,
                            const void* gate, const void* r_out, const void* h, const void* q, const void* q_scale,
                            int32_t group, int32_t fmt) {
    const int rc = check_border(b);
    if (rc) return rc;
    if ((q == nullptr) != (q_scale == nullptr)) return COAT_EINVAL;
    if (q) {
        if (fmt == COAT_FMT_MX4) {
            if (group != 32) return COAT_EINVAL;
        } else if (fmt == COAT_FMT_E4M3 || fmt == COAT_FMT_E5M2) {
            if (lg2_group_of(group) < 0 || group > 512 || b->cols % group != 0) return COAT_EINVAL;
        } else {
            return COAT_EINVAL;
        }
    }
    if (w_post && !b->post) return COAT_EINVAL;
    if (b->rows == 0) return COAT_OK;  // a matrix without rows may have no address
    if (!y && (gate || w_post || b->post || r_out)) return COAT_EINVAL;
    if (w_pre && !h && !q) return COAT_EINVAL;
    if (!r_out && !h && !q) return COAT_EINVAL;
    if (!r) return COAT_EINVAL;
    const size_t st = type_bytes(b->stream_type), pt = type_bytes(b->param_type);
    if (!aligned(y, 2) || !aligned(r, st) || !aligned(r_out, st) || !aligned(h, 2) || !aligned(w_post, pt) ||
        !aligned(w_pre, pt) || !aligned(gate, pt) || !aligned16(q) ||
        !aligned(q_scale, fmt == COAT_FMT_MX4 ? 16 : 4))
        return COAT_EALIGN;
    return COAT_OK;
}

// Wavefronts of a workgroup that holds one or two chunks of 8 channels a thread.
constexpr int border_chunks(int64_t cols) { return cols <= 8 * 1024 ? 1 : 2; }
constexpr int64_t border_waves(int64_t cols) { return div_up(div_up(cols, 8), 64 * border_chunks(cols)); }

// How the backward pass deals the rows to workgroups. A workgroup sums the
// weight gradients of its rows in registers and writes one row of partial sums,
// so there are as many as run at once (16 wavefronts on a compute unit, four
// workgroups at most) and not more: 16384 x 5120 takes 242 us with 256, 250 with
// 512, 261 with 1024; 16384 x 1024 takes 122, 72 and 51.
// No workgroup holds rows of two gate rows that both reach into others:
//   chunks > 0: a gate row's tokens are cut into `chunks` workgroups of `step`
//               rows (the last may be shorter or empty);
//   chunks = 0: a workgroup takes `step` rows, whole gate rows (or any rows, if
//               no gate gradient is wanted).
struct BorderSplit {
    int64_t step, chunks, blocks;
};
inline BorderSplit border_split(int64_t rows, int64_t cols, int64_t rows_per_gate, bool dgate) {
    if (rows == 0) return BorderSplit{1, 0, 0};
    const int64_t waves = border_waves(cols), each = waves > 8 ? 1 : (waves > 4 ? 2 : 4);
    const int64_t want = div_up(rows, kCUs * each);  // rows of a workgroup
    if (!dgate) return BorderSplit{want, 0, div_up(rows, want)};
    const int64_t rpg = rows_per_gate < rows ? rows_per_gate : rows, gates = div_up(rows, rpg);
    // Gate rows seldom divide evenly. Of the ways that fill one to three rounds of
    // workgroups the one with the fewest rows after one another is taken, a
    // workgroup's beginning and end counting as two: 8000 x 8000 with 301 tokens a
    // gate row takes 194 us in 243 workgroups of 34 rows, 303 in 270 of 31.
    BorderSplit best{0, 0, 0};
    int64_t least = INT64_MAX;
    auto consider = [&](int64_t step, int64_t chunks, int64_t blocks) {
        const int64_t cost = div_up(blocks, kCUs * each) * (step + 2);
        if (cost < least) {
            least = cost;
            best = BorderSplit{step, chunks, blocks};
        }
    };
    for (int64_t round = 1; round <= 3; ++round) {
        const int64_t slots = round * kCUs * each;
        if (gates <= slots) {
            const int64_t step = div_up(rpg, slots / gates), chunks = div_up(rpg, step);
            consider(step, chunks, gates * chunks);
        } else {
            const int64_t step = div_up(gates, slots) * rpg;
            consider(step, 0, div_up(rows, step));
        }
    }
    return best;
}

// Partial sums of the backward pass: up to three sections of blocks x cols fp32.
inline size_t border_section_bytes(int64_t blocks, int64_t cols) {
    return align_up((size_t)blocks * (size_t)cols * sizeof(float), 256);
}
inline size_t border_workspace_bytes(const coat_border* b) {
    if (check_border(b) != COAT_OK) return 0;
    const int64_t with = border_split(b->rows, b->cols, b->rows_per_gate, true).blocks;
    const int64_t without = border_split(b->rows, b->cols, b->rows_per_gate, false).blocks;
    return 3 * border_section_bytes(with > without ? with : without, b->cols);
}

inline int check_block_norm_backward(const coat_border* b, const void* y, const void* r_out, const void* dr_out,
                                     const void* dh, const void* w_post, const void* w_pre, const void* gate,
                                     const void* dr, const void* dy, const void* dw_post, const void* dw_pre,
                                     const void* dgate, const void* workspace, size_t workspace_bytes) {
    const int rc = check_border(b);
    if (rc) return rc;
    if (w_post && !b->post) return COAT_EINVAL;
    if ((dw_post && !w_post) || (dw_pre && !w_pre) || (dgate && !gate)) return COAT_EINVAL;
    const size_t st = type_bytes(b->stream_type), pt = type_bytes(b->param_type), gt = type_bytes(b->grad_type);
    if (b->rows > 0) {  // a matrix without rows may have no address
        if (!y && (gate || w_post || b->post || dy)) return COAT_EINVAL;
        if (!dh && (w_pre || !dr_out)) return COAT_EINVAL;
        if (!dr || (y && !dy) || (dh && !r_out)) return COAT_EINVAL;
        const size_t need = border_workspace_bytes(b);
        if ((dw_post || dw_pre || dgate) && (!workspace || workspace_bytes < need)) return COAT_EINVAL;
    }
    if (!aligned(y, 2) || !aligned(dh, 2) || !aligned(dy, 2) || !aligned(r_out, st) || !aligned(dr_out, st) ||
        !aligned(dr, st) || !aligned(w_post, pt) || !aligned(w_pre, pt) || !aligned(gate, pt) ||
        !aligned(dw_post, gt) || !aligned(dw_pre, gt) || !aligned(dgate, gt) || !aligned(workspace, 256))
        return COAT_EALIGN;
    return COAT_OK;
}

}  // namespace

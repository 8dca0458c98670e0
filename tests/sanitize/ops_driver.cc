// The host logic of the layer-input operators (ops_host.h) on the CPU: argument
// checks, and how the border's backward pass and the product deal their work out.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "ops_host.h"

#define EXPECT(c)                                                    \
    do {                                                             \
        if (!(c)) {                                                  \
            fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); \
            exit(1);                                                 \
        }                                                            \
    } while (0)

static const void* at(uintptr_t a) { return reinterpret_cast<const void*>(a); }
static const uint8_t* bytes(uintptr_t a) { return reinterpret_cast<const uint8_t*>(a); }

// Every row belongs to one workgroup, none to two; no workgroup holds rows of two
// gate rows that both reach into others; partial sums of a gate row are consecutive.
static void border(int64_t rows, int64_t cols, int64_t rpg, bool dgate) {
    const BorderSplit s = border_split(rows, cols, rpg, dgate);
    const int64_t eff = rpg < rows ? rpg : rows;
    std::vector<int> seen((size_t)rows, 0);
    for (int64_t b = 0; b < s.blocks; ++b) {
        int64_t r0, r1;
        if (s.chunks > 0) {
            const int64_t g = b / s.chunks;
            r0 = g * eff + (b - g * s.chunks) * s.step;
            r1 = r0 + s.step < (g + 1) * eff ? r0 + s.step : (g + 1) * eff;
        } else {
            r0 = b * s.step;
            r1 = r0 + s.step;
        }
        if (r1 > rows) r1 = rows;
        for (int64_t r = r0; r < r1; ++r) ++seen[(size_t)r];
        if (dgate && r1 > r0) {
            const bool cut = r0 % eff != 0 || (r1 % eff != 0 && r1 != rows);
            if (cut) EXPECT(s.chunks > 0 && r0 / eff == (r1 - 1) / eff);
        }
    }
    for (int v : seen) EXPECT(v == 1);
    if (s.chunks > 0) EXPECT((s.chunks - 1) * s.step < eff && s.chunks * s.step >= eff);  // no empty part of a whole gate row
    EXPECT(s.blocks <= 3 * 4 * kCUs);
    coat_border d{};
    d.rows = rows;
    d.cols = cols;
    d.rows_per_gate = rpg;
    d.eps = 1e-5f;
    d.scale = 1.0f;
    EXPECT(border_workspace_bytes(&d) >= 3 * border_section_bytes(s.blocks, cols));
}

// The parts of k that the splits take cover its groups of steps, none is empty, and
// the workspace holds them.
static void product(int64_t m, int64_t n, int64_t k) {
    const Product p = product_of(m, n, k);
    const size_t need = product_workspace_bytes(m, n, k);
    EXPECT((need > 0) == (p.splits > 1));
    if (p.way != Way::kTile128 && p.way != Way::kTile256) return;
    const int64_t tile = p.way == Way::kTile256 ? 256 : 128, groups = div_up(k, 512);
    EXPECT((int64_t)p.tiles_m * tile >= m && ((int64_t)p.tiles_m - 1) * tile < m);
    EXPECT((int64_t)p.tiles_n * tile >= n && ((int64_t)p.tiles_n - 1) * tile < n);
    EXPECT((int64_t)p.splits * p.per_split >= groups && ((int64_t)p.splits - 1) * p.per_split < groups);
    EXPECT((int64_t)p.tiles_m * p.tiles_n * p.splits <= 0x7FFFFFFF);
    EXPECT(p.head_m >= 1 && p.head_m <= m && p.head_n >= 1 && p.head_n <= n && (p.head_m == m || p.head_n == n));
    if (p.head_m < m) EXPECT(p.way == Way::kTile256 && p.head_m % 256 == 0);
    if (p.head_n < n) EXPECT(p.way == Way::kTile256 && p.head_n % 256 == 0);
    if (p.splits > 1) EXPECT(p.lw >= n && p.lw % 4 == 0 && need == (size_t)p.splits * (size_t)m * (size_t)p.lw * 4);
}

// Every workgroup has a number, none of them is far behind, and no axis holds 2^32 work-items.
static void grid(int64_t count, int64_t threads) {
    const Grid g = grid_xy(count, threads);
    EXPECT((uint64_t)g.x * (uint64_t)threads < (uint64_t(1) << 32) && g.y < 65536);
    EXPECT((int64_t)g.x * g.y >= count && (int64_t)g.x * (g.y - 1) < count && (uint64_t)g.x * g.y < (uint64_t(1) << 32));
    EXPECT(g.y == 1 || g.x % 16 == 0);
}

int main() {
    for (int64_t count : {int64_t(1), int64_t(17), int64_t(256), (int64_t(1) << 24) - 16, int64_t(1) << 24, (int64_t(1) << 24) + 32,
                          (int64_t(1) << 26) + 3, int64_t(0x7FFFFFFF)})
        for (int64_t threads : {64, 256, 512}) grid(count, threads);
    for (int64_t rows : {1, 2, 7, 255, 256, 257, 600, 700, 1031, 4096, 5001, 8000})
        for (int64_t cols : {1, 64, 512, 1024, 2731, 5120, 8192, 16384})
            for (int64_t rpg : {int64_t(1), int64_t(2), int64_t(3), int64_t(5), int64_t(31), int64_t(64), int64_t(257), rows / 2 + 1, rows, rows + 9})
                for (bool dgate : {false, true}) border(rows, cols, rpg, dgate);
    EXPECT(border_split(0, 64, 1, true).blocks == 0);

    for (int64_t m : {1, 32, 33, 64, 100, 333, 2048, 16384, 1 << 20, 0x7FFFFFFF})
        for (int64_t n : {1, 17, 300, 5120, 13824, 0x7FFFFFFF})
            for (int64_t k : {1, 128, 511, 513, 5120, 13824, (1 << 22) - 1, 1 << 22, 0x7FFFFFFF}) product(m, n, k);
    EXPECT(product_of(4096, 5120, 5120).head_n == 16 * 256 && product_of(5120, 4096, 5120).head_m == 16 * 256);
    EXPECT(product_of(16384, 5120, 13824).head_n == 5120);  // whole rounds
    // the products whose every element the GPU tests compare, k as the codes hold it: large
    // tiles in more than one round, over several groups of steps but for one; the last four with a rest
    struct Case {
        int64_t m, n, k;
        bool rest;
    };
    for (const Case& c : {Case{8192, 8192, 1152, false}, Case{8192, 8192, 1280, false}, Case{8192, 8192, 1408, false},
                          Case{8192, 8192, 1536, false}, Case{8192, 8192, 384, false}, Case{16384, 4000, 1152, false},
                          Case{8000, 8300, 1152, true}, Case{4096, 5120, 5120, true}, Case{5120, 4096, 5120, true}, Case{2600, 13824, 5120, true}}) {
        const Product p = product_of(c.m, c.n, c.k);
        EXPECT(p.way == Way::kTile256 && p.splits == 1);
        EXPECT((p.head_m < c.m || p.head_n < c.n) == c.rest);
        EXPECT(div_up(p.head_m, 256) * div_up(p.head_n, 256) > (c.rest ? kCUs - 1 : 2 * kCUs));
    }
    // one side within a small tile: small ones, here in more than one round of workgroups
    for (const Case& c : {Case{128, 40000, 1152, false}, Case{100, 40000, 1280, false}, Case{64, 40001, 1408, false}, Case{40000, 128, 1536, false},
                          Case{70000, 33, 384, false}, Case{20, 128256, 5120, false}, Case{1 << 18, 33, 8200, false}}) {
        const Product p = product_of(c.m, c.n, c.k);
        EXPECT(p.way == Way::kTile128 && p.splits == 1 && p.tiles_m * p.tiles_n > (uint32_t)kCUs);
    }
    EXPECT(product_of(129, 65536, 5120).way == Way::kTile256 && product_of(65536, 129, 5120).way == Way::kTile256);
    EXPECT(product_workspace_bytes(0, 5, 5) == 0 && product_workspace_bytes(5, 5, -1) == 0);

    EXPECT(mx4_code_bytes(1) == 64 && mx4_code_bytes(129) == 128 && mx4_scale_bytes(512) == 16 && mx4_scale_bytes(513) == 32);
    const uintptr_t a = 0x10000;
    EXPECT(check_mx4_quantize(at(a), 4, 64, 64, COAT_BF16, bytes(a), bytes(a), nullptr, nullptr) == COAT_OK);
    EXPECT(check_mx4_quantize(at(a), 4, 64, 63, COAT_BF16, bytes(a), bytes(a), nullptr, nullptr) == COAT_EINVAL);
    EXPECT(check_mx4_quantize(at(a), kMaxDim, 64, INT64_MAX / 2, COAT_BF16, bytes(a), bytes(a), nullptr, nullptr) == COAT_EINVAL);
    EXPECT(check_mx4_quantize(at(a + 1), 4, 64, 64, COAT_BF16, bytes(a), bytes(a), nullptr, nullptr) == COAT_EALIGN);
    EXPECT(check_mx4_matmul(bytes(a), bytes(a), 4, bytes(a), bytes(a), 8, 64, at(a), 8, COAT_FP32) == COAT_OK);
    EXPECT(check_mx4_matmul(nullptr, nullptr, 4, nullptr, nullptr, 8, 0, at(a), 8, COAT_FP32) == COAT_OK);
    EXPECT(check_mx4_dequantize(bytes(a), bytes(a), 0, 64, nullptr, 64, COAT_FP32) == COAT_OK);
    coat_border d{};
    EXPECT(check_border(nullptr) == COAT_EINVAL && check_border(&d) == COAT_EINVAL && border_workspace_bytes(&d) == 0);
    d.rows = 4;
    d.cols = 64;
    d.rows_per_gate = 4;
    d.eps = 1e-5f;
    d.post = 1;
    EXPECT(check_block_norm(&d, at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), 32, COAT_FMT_E4M3) == COAT_OK);
    EXPECT(check_block_norm(&d, at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), 128, COAT_FMT_E4M3) == COAT_EINVAL);
    EXPECT(check_block_norm(&d, nullptr, at(a), nullptr, nullptr, nullptr, nullptr, at(a), nullptr, nullptr, 0, 0) == COAT_EINVAL);
    const size_t need = border_workspace_bytes(&d);
    EXPECT(check_block_norm_backward(&d, at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a),
                                     need) == COAT_OK);
    EXPECT(check_block_norm_backward(&d, at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a), at(a),
                                     need - 1) == COAT_EINVAL);
    printf("ok\n");
    return 0;
}

// Host logic of the gradients' second bf16 terms under the sanitizers: which sizes take them, and
// that every section of the workspaces holds what is written to it.
#include <stdio.h>
#include <stdlib.h>

#include "train_host.h"

#define CHECK(c)                                                             \
    do {                                                                     \
        if (!(c)) {                                                          \
            printf("line %d: %s (%lld %lld %lld)\n", __LINE__, #c, (long long)m, (long long)n, (long long)k); \
            return 1;                                                        \
        }                                                                    \
    } while (0)

// The partial sums of a plan's splits, one behind the other, as the tiles write them.
static size_t sums_bytes(const Plan16& p, int64_t rows) {
    return p.splits > 1 ? ((size_t)(p.splits - 1) * (size_t)p.stride + (size_t)rows * (size_t)p.ld) * 4 : 0;
}

static int linear_ok(int64_t m, int64_t n, int64_t k, bool ready) {
    const LinearBackwardLayout b = linear_backward_layout(m, n, k, ready);
    const bool two = dz_takes_two_terms(m, n);
    CHECK(two == ((double)m * (double)n <= 2048));
    const size_t rows = (size_t)(two ? 2 * m : m);
    CHECK(b.bias - b.dz >= rows * (size_t)b.ld_dz * 2);
    CHECK(b.x - b.part >= sums_bytes(b.plan_dx, m) && b.x - b.part >= sums_bytes(b.plan_dw, n));
    CHECK(b.w - b.x >= (two || !ready ? rows * (size_t)packed_ld(k) * 2 : 0));
    CHECK(b.acc - b.w >= (ready ? 0 : (size_t)n * (size_t)packed_ld(k) * 2));
    if (!two) {
        CHECK(b.end == b.acc);
        return 0;
    }
    CHECK(b.x - b.part >= sums_bytes(b.plan_dw_two, n));
    CHECK(b.end - b.acc >= (size_t)m * (size_t)packed_ld(k) * 4);
    CHECK(b.plan_dx.way != Way16::kTile256);
    return 0;
}

static int xent_ok(int64_t m, int64_t n, int64_t k, bool ready) {
    const XentBackwardLayout d = xent_backward_layout(m, n, k, ready);
    CHECK(d.two == (m <= 16 || (double)m * (double)n <= 2048));
    const size_t t = (size_t)m, rows = d.two ? 2 * t : t;
    CHECK(d.at >= d.count + 3 * 4 && d.place - d.at >= t * 4 && d.second - d.place >= t * 4);
    CHECK(d.info - d.second >= (d.two ? t * 4 : 0) && d.x - d.info >= t * 16);
    CHECK(d.g - d.x >= rows * (size_t)d.ld_x * 2 && d.acc - d.g >= rows * (size_t)d.ld_g * 2);
    CHECK((!d.two && d.piece == n) || d.part - d.acc >= t * (size_t)d.ld_x * 4);
    CHECK(d.end - d.w >= (ready ? 0 : (size_t)n * (size_t)packed_ld(k) * 2));
    int64_t last = n % d.piece == 0 ? d.piece : n % d.piece;
    for (const int64_t width : {d.piece, last}) {
        const XentPiece p = xent_piece_plans(m, width, k, d.two);
        CHECK(d.w - d.part >= sums_bytes(p.logits, m) && d.w - d.part >= sums_bytes(p.dx, m) && d.w - d.part >= sums_bytes(p.dw, width));
        CHECK(!d.two || (p.logits.way != Way16::kTile256 && p.dx.way != Way16::kTile256));
    }
    return 0;
}

int main() {
    const int64_t sizes[] = {1, 2, 3, 7, 8, 15, 16, 17, 31, 32, 40, 64, 65, 127, 128, 255, 256, 257, 1000, 1024, 2047, 2048, 2049, 4096, 5120, 13824, 32000,
                             50257, 128256, (1 << 20) + 3, (1 << 21) - 1, 1 << 21, (1 << 21) + 300, (1 << 22) - 1, 1 << 22, (1 << 23) + 9, (1 << 24) + 1};
    long twos = 0, pieces = 0;
    for (const int64_t m : sizes)
        for (const int64_t n : sizes)
            for (const int64_t k : sizes) {
                if (4.0 * ((double)m * n + (double)m * k + (double)n * k) > 4e12) continue;  // more than any card holds
                for (const bool ready : {false, true})
                    if (linear_ok(m, n, k, ready) || xent_ok(m, n, k, ready)) return 1;
                const XentBackwardLayout d = xent_backward_layout(m, n, k, true);
                twos += d.two;
                pieces += d.two && d.piece < n;
            }
    // a plan without large tiles is the one with them wherever second terms are taken
    for (int64_t m = 1; m <= 2048; ++m)
        for (const int64_t k : sizes) {
            const int64_t n = 2048 / m;
            CHECK(plan16_of(m, k, n, true, false, true, true).way != Way16::kTile256);
        }
    const int64_t m = twos, n = pieces, k = 0;
    CHECK(twos > 1000 && pieces > 10);
    printf("ok\n");
    return 0;
}

// Host logic of the training products under the sanitizers: every plan covers its product,
// every workspace section lies behind the one before.
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

static int plan_ok(int64_t m, int64_t n, int64_t k, bool split, bool ta, bool tb) {
    const Plan16 p = plan16_of(m, n, k, split, ta, tb);
    if (p.way == Way16::kPlain || p.way == Way16::kFew) {
        CHECK(p.splits == 1);
        CHECK(plan16_bytes(p) == 0);
        CHECK(p.way == Way16::kPlain || (!ta && !tb && m <= 16));
        return 0;
    }
    const int64_t side = p.way == Way16::kTile256 ? 256 : 128, steps = div_up(k, 64);
    CHECK(p.tiles_m * side >= m && (int64_t)(p.tiles_m - 1) * side < m);
    CHECK(p.tiles_n * side >= n && (int64_t)(p.tiles_n - 1) * side < n);
    CHECK((int64_t)p.splits * p.per_split >= steps && (int64_t)(p.splits - 1) * p.per_split < steps);
    CHECK(split || p.splits == 1);
    CHECK(p.splits == 1 || (p.ld >= n && p.ld % 64 == 0 && p.stride >= m * p.ld));
    CHECK((int64_t)p.tiles_m * p.tiles_n * p.splits < (int64_t(1) << 31));
    // a tile's byte offsets stay within 32 bits
    CHECK((ta ? m : k) < kMaxLd && (tb ? n : k) < kMaxLd);
    return 0;
}

int main() {
    const int64_t sizes[] = {1, 2, 7, 8, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 1023, 4096, 5120, 13824, 16384, 32000, 50257,
                             128256, (1 << 20) + 3, (1 << 22) - 1, 1 << 22, (1 << 24) + 1, 0x7FFFFFFF};
    for (const int64_t m : sizes)
        for (const int64_t n : sizes)
            for (const int64_t k : sizes) {
                for (int f = 0; f < 8; ++f)
                    if (plan_ok(m, n, k, f & 1, f & 2, f & 4)) return 1;
                const double bytes = 4.0 * ((double)m * n + (double)m * k + (double)n * k);
                if (bytes > 4e12) continue;  // more than any card holds
                for (const bool ready : {false, true}) {
                    const LinearLayout a = linear_layout(m, n, k, ready);
                    CHECK(a.part <= a.x && a.x <= a.w && a.w <= a.end && a.end % 256 == 0);
                    const LinearBackwardLayout b = linear_backward_layout(m, n, k, ready);
                    CHECK(b.dz <= b.bias && b.bias <= b.part && b.part <= b.x && b.x <= b.w && b.w <= b.end && b.ld_dz >= n);
                    CHECK(b.part - b.bias >= (size_t)div_up(m, bias_band(m, n)) * (size_t)n * 4);
                    CHECK(b.x - b.part >= plan16_bytes(b.plan_dx) && b.x - b.part >= plan16_bytes(b.plan_dw));
                    const XentLayout c = xent_layout(m, n, k, ready);
                    CHECK(c.parts * log_sum_width(c.plan.way) >= n && c.x - c.part >= (size_t)c.parts * (size_t)m * 8);
                    CHECK(c.count < c.at && c.at < c.label && c.label < c.zt && c.zt < c.part && c.x <= c.w && c.w <= c.end);
                    const XentBackwardLayout d = xent_backward_layout(m, n, k, ready);
                    CHECK(d.piece >= 1 && d.piece <= n && d.ld_g >= d.piece && d.piece < kMaxLd && d.ld_x >= k);
                    CHECK(d.at < d.place && d.place < d.info && d.info < d.x && d.x < d.g && d.g < d.acc && d.acc <= d.part && d.part <= d.w && d.w <= d.end);
                    CHECK(d.piece == n || d.part - d.acc >= (size_t)m * (size_t)d.ld_x * 4);
                    CHECK(d.piece <= 2048 || d.piece * m <= (int64_t(1) << 27) + 256 * m);
                }
            }
    const int64_t m = 0, n = 0, k = 0;
    for (const float p : {0.0f, 0x1p-18f, 0.1f, 0.5f, 0.999f, 0x1.fffffep-1f}) {
        const uint32_t t = drop_threshold(p);
        CHECK(t <= 65535 && drop_factor(t) >= 1.0f);
    }
    CHECK(drop_threshold(0.5f) == 32768 && drop_threshold(0x1p-18f) == 0 && drop_threshold(0x1.fffffep-1f) == 65535);
    coat_epilogue e{0, 1.0f, 0.0f, 0, nullptr};
    static char at[64] __attribute__((aligned(64)));
    CHECK(check_linear(at, 2, 3, 3, at, 2, 3, &e, nullptr, 0, nullptr, 2, nullptr, 2, at, 2, 0) == COAT_OK);
    CHECK(check_linear(at, 2, 3, 2, at, 2, 3, &e, nullptr, 0, nullptr, 2, nullptr, 2, at, 2, 0) == COAT_EINVAL);
    CHECK(check_linear(at + 1, 2, 3, 3, at, 2, 3, &e, nullptr, 0, nullptr, 2, nullptr, 2, at, 2, 0) == COAT_EALIGN);
    CHECK(tiles_take(at, 64, 64) && !tiles_take(at, 63, 56) && !tiles_take(at + 2, 64, 64) && !tiles_take(at, 64, 63) && !tiles_take(at, kMaxLd, 64));
    CHECK(tiles_gather(at, 1 << 20, 64, 64) && !tiles_gather(at, 1 << 25, 64, 64));
    printf("ok\n");
    return 0;
}

// Products of bf16 matrices on the matrix units (gfx950), with an epilogue of the caller's.
#pragma once

#include <type_traits>

#include "train_common.h"

namespace {

// ------------------------------------------------------------------ the product
//
// sum over k of A(i, k) B(j, k), A m x k and B n x k in bf16. An operand's memory has
// rows of k (k runs along a row), or of i (k is the row: "tall").

struct Product16 {
    const uint16_t *a, *b;
    int64_t lda, ldb;       // elements from row to row of memory
    const int32_t* a_rows;  // row i of A is row a_rows[i] of memory; NULL: row i (not with a tall A)
    const int32_t* m_at;    // in device memory: the rows of A that exist, at most m; NULL: m
    const int32_t* k_at;    // the same of k
    int64_t m, n, k;
};

// The same of 16 rows of each operand over 32 values of k: lane l holds the 8 values
// k = 8 (l / 16) .. of row l % 16; accumulator r of lane l is row l % 16, column
// 4 (l / 16) + r. Written out, because the compiler moves 64 such accumulators about
// between accumulation registers. It knows of no wait for it: who reads a result waits,
// and no vector instruction may have written an operand in the two states before (the
// fragments come from LDS reads alone; a test looks at the compiled code). Waiting here
// would cost 5 % (8192 x 8192 x 8192 732 -> 772 us).
__device__ __forceinline__ void mfma16x16(const u32x4& b, const u32x4& a, f32x4& acc) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

__device__ __forceinline__ f32x16 mfma16(const u32x4& b, const u32x4& a, const f32x16& acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
}

template <class Out>
__device__ __forceinline__ void finish(const Out& out, int64_t row, int64_t col, float (&v)[8], int64_t n) {
    out(row, col, v, n, out.column(col, n), out.row(row, col, n));
}

// One matrix instruction takes 32 rows of each operand over 16 values of k: lane l
// holds the 8 values k = 8 (l / 32) .. of row l % 32. B is the first operand, so that
// a lane's four consecutive accumulators are four consecutive columns: accumulator r
// of lane l is row l % 32, column 8 (r / 4) + 4 (l / 32) + r % 4.
//
// The plain product, straight from global memory: each wavefront a 32 x 32 tile, a
// workgroup 64 x 64; any strides and alignments.
template <bool TALL_A, bool TALL_B, class Out>
__global__ __launch_bounds__(kBlock) void product_plain_kernel(Product16 p, uint32_t tiles_n, Out out) {
    __shared__ float lds[kWavesPerBlock][32][33];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t tile = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t m = p.m_at ? (int64_t)__builtin_amdgcn_readfirstlane(*gp(p.m_at)) : p.m, k = p.k_at ? (int64_t)__builtin_amdgcn_readfirstlane(*gp(p.k_at)) : p.k;
    const int64_t n0 = tile % tiles_n * 64 + (wave & 1) * 32, m0 = tile / tiles_n * 64 + (wave >> 1) * 32;
    if (m0 >= m || n0 >= p.n) return;
    out.begin();
    const int row = lane & 31, half = lane >> 5;
    // rows past the end are read as the last one and not used
    const int64_t ra = m0 + row < m ? m0 + row : m - 1, rb = n0 + row < p.n ? n0 + row : p.n - 1;
    const int64_t ma = p.a_rows ? (int64_t)gp(p.a_rows)[ra] : ra;
    const uint16_t* const pa = p.a + (TALL_A ? ra : ma * p.lda);
    const uint16_t* const pb = p.b + (TALL_B ? rb : rb * p.ldb);
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int64_t k0 = 0; k0 < k; k0 += 16) {
        u32x4 a{0u, 0u, 0u, 0u}, b{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = k0 + half * 8 + e;
            if (at < k) {
                a[e / 2] |= (uint32_t)gp(pa)[TALL_A ? at * p.lda : at] << (16 * (e & 1));
                b[e / 2] |= (uint32_t)gp(pb)[TALL_B ? at * p.ldb : at] << (16 * (e & 1));
            }
        }
        acc = mfma16(b, a, acc);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) lds[wave][row][8 * (r / 4) + 4 * half + r % 4] = acc[r];
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if constexpr (Out::kLogSum) {
        if (lane < 32 && m0 + lane < m) {
            const int64_t label = out.label_of(m0 + lane) - n0;
            const int cols = (int)(p.n - n0 < 32 ? p.n - n0 : 32);
            float top = -__builtin_inff(), sum = 0.0f;
            for (int c = 0; c < cols; ++c)
                if (c == label) out.keep(m0 + lane, lds[wave][lane][c]);
                else top = fmaxf(top, lds[wave][lane][c]);
            const float from = top == -__builtin_inff() ? 0.0f : top;
            for (int c = 0; c < cols; ++c)
                if (c != label) sum += exp_fast(lds[wave][lane][c] - from);
            out.put(m0 + lane, n0 / 32, from, sum);
        }
    } else {
        for (int i = lane; i < 32 * 4; i += kWave) {
            const int r = i / 4, c = i % 4 * 8;
            if (m0 + r >= m || n0 + c >= p.n) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = lds[wave][r][c + e];
            finish(out, m0 + r, n0 + c, v, p.n - n0 - c);
        }
    }
}

// ------------------------------------------------------------------ tiles
//
// A workgroup of WN x WM wavefronts, each with 32 FN rows of B by 32 FM rows of A,
// computes tiles one after the other; the k of all its tiles forms one stream of
// steps of 64 values. An operand's part of a step (128 bytes for each row of the tile)
// goes straight from global memory into one of five parts of LDS, two steps before it
// is used; the fifth lets the loads run on evenly, and between two tiles the sums leave
// through it. A step is computed in four phases of 16 values: while one phase's matrix
// instructions run, the fragments of the one after the next are read from LDS. One
// barrier a step, in its middle: behind it every wavefront has read the step (its parts
// may be refilled) and the next one has arrived.
//
// In LDS an operand whose k runs along its rows lies as rows of 128 bytes, chunk c of
// row r at position c ^ (r / 2 % 8), so that 16 rows' reads reach 16 different 16-byte
// columns of the banks. A tall one lies as 64 rows of k, its 32-byte runs r at
// r ^ (k % 4 * 2 + k / 8 % 2): the transposing read takes 4 rows of k by 16 columns from 16
// lanes, and 32 lanes reach every bank once. The counters show no bank conflict in either.
//
// Tiles of 256 x 256 (four wavefronts of 128 x 128 sums in accumulation registers, all 160
// KB of LDS) are bound by the card's power and the matrix units: 8192 x 8192 x 8192 takes
// 732 us (1.50 PFLOP/s; a library's 680), the units busy for 0.77 of the cycles at 1.8 GHz;
// on zeros the clock is 2.3. What was measured on the way there, in us of that size: loads
// in one burst instead of spread over the step 947 against 917, a fifth part of LDS for
// them 863, no scalar work between phases 805, instructions of 16 x 16 instead of 32 x 32
// (half as many accumulator reads and writes) 732. Eight wavefronts of 64 x 128 read half
// as much again from LDS and gain nothing (1137 against 874 at the time).
// Tiles of 128 x 128 (two workgroups a compute unit) hide one's beginning and end behind
// the other: 1023 x 50257 x 768 takes 100 us in them and 124 in large ones.
template <int N>
__device__ __forceinline__ void wait_vm_and_lds_then_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes a lane from base + off to LDS, lane after lane from byte address lds + AT.
template <uint32_t AT>
__device__ __forceinline__ void load_to_lds16(uint32_t lds, uint32_t off, const uint8_t* base) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base), "n"(AT)
                 : "memory", "scc");
}
// f(0), f(1), ... f(N - 1) with the index known to the compiler.
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<N, I + 1>(f);
    }
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// Items: with splits > 1 item t is the product over the steps [s per_split, (s + 1)
// per_split), s = t / tiles, of tile t % tiles, and goes to part + s stride (sums that
// another kernel adds).
struct Items {
    uint32_t tiles_n, splits, per_split;
    float* part;
    int64_t ld, stride;
};

template <int WN_, int WM_, int FN_, int FM_>
struct TileShape {
    static constexpr int WN = WN_, WM = WM_, FN = FN_, FM = FM_, WAVES = WN * WM, BN = 16 * WN * FN, BM = 16 * WM * FM;
    static constexpr int kPart = BN * 128, kLds = 5 * kPart;  // bytes of an operand's part of a step; of LDS
    static constexpr int PIECE = kPart / WAVES / 128;         // fp32 columns of 32 rows that a wavefront writes out at a time
    static constexpr int kWavesPerSimd = WAVES / 4 * (kLds <= 81920 ? 2 : 1);
};
typedef TileShape<2, 2, 8, 8> Tile256;
typedef TileShape<2, 2, 4, 4> Tile128;

template <class S, bool TALL_A, bool TALL_B, class Out>
__global__ __launch_bounds__(S::WAVES* kWave) __attribute__((amdgpu_waves_per_eu(S::kWavesPerSimd, S::kWavesPerSimd))) void product_tile_kernel(
    Product16 p, Items items_of, Out out) {
    constexpr int WN = S::WN, FN = S::FN, FM = S::FM, PIECE = S::PIECE;
    constexpr int WAVES = S::WAVES, BN = S::BN, BM = S::BM;
    constexpr int LA = BM / 8 / WAVES, LB = BN / 8 / WAVES;  // loads of a step by each wavefront
    static_assert(BN == BM && LB * 8 * WAVES == BN && LB % 4 == 0 && WAVES % 2 == 0, "loads are dealt evenly");
    constexpr uint32_t kPart = S::kPart;
    __shared__ __attribute__((aligned(16))) uint8_t lds[S::kLds];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int quad = lane >> 4, l16 = lane & 15;
    const int64_t m = p.m_at ? (int64_t)__builtin_amdgcn_readfirstlane(*gp(p.m_at)) : p.m, n = p.n, k = p.k_at ? (int64_t)__builtin_amdgcn_readfirstlane(*gp(p.k_at)) : p.k;
    const uint32_t tiles_n = items_of.tiles_n, tiles_m = (uint32_t)((m + BM - 1) / BM);
    const uint32_t tiles = tiles_m * tiles_n, items = tiles * items_of.splits;
    const uint32_t steps = (uint32_t)((k + 63) / 64), per_split = items_of.per_split;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

    // tile t: patches of 8 x 4 tiles are consecutive
    auto place = [&](uint32_t t, int64_t& m0, int64_t& n0) __attribute__((always_inline)) {
        const uint32_t per = 8 * tiles_n, band = t / per, in = t - band * per;
        const uint32_t high = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8;
        m0 = (int64_t)(band * 8 + in % high) * BM;
        n0 = (int64_t)(in / high) * BN;
    };
    // values of k in step g, at most 64 (none only if k is 0 or a split's part is empty)
    auto values_of = [&](uint32_t g) __attribute__((always_inline)) {
        const int64_t left = k - (int64_t)g * 64;
        return (uint32_t)(left < 0 ? 0 : (left < 64 ? left : 64));
    };
    auto first_step = [&](uint32_t t) __attribute__((always_inline)) { return items_of.splits == 1 ? 0 : t / tiles * per_split; };
    auto last_step = [&](uint32_t t) __attribute__((always_inline)) {  // one past it; an item has one step at least
        const uint32_t g0 = first_step(t), g1 = g0 + per_split < steps ? g0 + per_split : steps;
        return g1 > g0 ? g1 : g0 + 1;
    };

    // Byte offsets of this lane's 16 bytes in each load. What is past the end of the
    // matrix or of k is not read: another row, column or value is fetched in its place,
    // and not used, or zeroed in LDS.
    uint32_t off_a[LA], off_b[LB];
    auto offsets = [&](int64_t m0, int64_t n0, uint32_t values) __attribute__((always_inline)) {
        each<LA + LB>([&](auto i) __attribute__((always_inline)) {
            constexpr bool is_b = i < LB, tall = is_b ? TALL_B : TALL_A;
            constexpr int own = is_b ? i : i - LB, width = is_b ? BN : BM;
            uint32_t& off = is_b ? off_b[is_b ? own : 0] : off_a[is_b ? 0 : own];
            const uint32_t ld2 = (uint32_t)(is_b ? p.ldb : p.lda) * 2;
            const int64_t left = is_b ? n - n0 : m - m0;
            if constexpr (tall) {
                constexpr int lanes = width / 8, rows = kWave / lanes;  // lanes of a row of k, rows of a load
                uint32_t row = (own * WAVES + wave) * rows + lane / lanes;
                const uint32_t at = lane % lanes, run = (at >> 1) ^ ((row & 3) * 2 + (row >> 3 & 1));
                uint32_t col = (run * 2 + (at & 1)) * 8;
                if (col >= left) col = 0;
                if (row >= values) row = values > 0 ? values - 1 : 0;
                off = row * ld2 + col * 2;
            } else {
                uint32_t row = (own * WAVES + wave) * 8 + lane / 8, chunk = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
                if (row >= left) row = (uint32_t)left - 1;
                if (chunk * 8 >= values) chunk = 0;
                if (!is_b && p.a_rows) off = (uint32_t)gp(p.a_rows)[m0 + row] * ld2 + chunk * 16;
                else off = row * ld2 + chunk * 16;
            }
        });
    };
    const uint8_t *next_a, *next_b;  // first row of the step that is fetched next
    auto start = [&](int64_t m0, int64_t n0, uint32_t g) __attribute__((always_inline)) {
        const uint8_t *a = reinterpret_cast<const uint8_t*>(p.a), *b = reinterpret_cast<const uint8_t*>(p.b);
        next_b = TALL_B ? b + ((int64_t)g * 64 * p.ldb + n0) * 2 : b + (n0 * p.ldb + (int64_t)g * 64) * 2;
        next_a = TALL_A ? a + ((int64_t)g * 64 * p.lda + m0) * 2 : a + ((p.a_rows ? 0 : m0 * p.lda) + (int64_t)g * 64) * 2;
    };
    const uint32_t lds_wave = lds0 + wave * 1024;
    // `part`: an offset into LDS
    auto fetch_a = [&](uint32_t part, auto i) __attribute__((always_inline)) {
        load_to_lds16<i * WAVES * 1024>(lds_wave + part, off_a[i], next_a);
    };
    auto fetch_b = [&](uint32_t part, auto i) __attribute__((always_inline)) {
        load_to_lds16<i * WAVES * 1024>(lds_wave + part, off_b[i], next_b);
    };

    const int wn = wave % WN * FN * 16, wm = wave / WN * FM * 16;
    u32x4 fb[2][FN], fa[2][FM];  // fragments of the phases
    auto read_one = [&](const uint8_t* base, auto tall, auto width, int w0, int i, int f) __attribute__((always_inline)) {
        if constexpr (tall.value) {
            const int row = 32 * f + 8 * quad + (l16 >> 2), run = (w0 / 16 + i) ^ ((l16 >> 2) * 2 + (quad & 1));
            const uint8_t* at = base + row * (width.value * 2) + run * 32 + (l16 & 3) * 8;
            const u32x2 lo = read_transposed(at), hi = read_transposed(at + 4 * width.value * 2);
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        } else {
            return *reinterpret_cast<const u32x4*>(base + (w0 + i * 16 + l16) * 128 + ((4 * f + quad) ^ (l16 >> 1)) * 16);
        }
    };
    // fragment i of phase f, A's first, which every row of matrix instructions needs
    auto read_frag = [&](uint32_t part_a, uint32_t part_b, int f, int i) __attribute__((always_inline)) {
        if (i < FM) fa[f][i] = read_one(lds + part_a, std::bool_constant<TALL_A>{}, std::integral_constant<int, BM>{}, wm, i, f);
        else fb[f][i - FM] = read_one(lds + part_b, std::bool_constant<TALL_B>{}, std::integral_constant<int, BN>{}, wn, i - FM, f);
    };
    // Zeroes what a step of fewer than 64 values has fetched in excess.
    auto clear_excess = [&](uint32_t part_a, uint32_t part_b, uint32_t values) __attribute__((always_inline)) {
        const u32x4 none{0u, 0u, 0u, 0u};
        for (uint32_t c = threadIdx.x; c < BN * 8; c += WAVES * kWave) {
            const uint32_t tall = c / (BN / 8), wide = ((c & 7) ^ (c >> 4 & 7)) * 8;
            if ((TALL_A ? tall : wide) >= values) *reinterpret_cast<u32x4*>(lds + part_a + c * 16) = none;
            if ((TALL_B ? tall : wide) >= values) *reinterpret_cast<u32x4*>(lds + part_b + c * 16) = none;
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };

    // consecutive workgroups run on different XCDs: each XCD takes consecutive items of a round
    const uint32_t first = gridDim.x % 8 == 0 ? (blockIdx.x & 7) * (gridDim.x / 8) + (blockIdx.x >> 3) : blockIdx.x;
    if (first >= items) return;
    out.begin();
    uint32_t ft = first, fg = first_step(first), fg_end = last_step(first);  // step fg of item ft is fetched next
    int64_t m0, n0;
    place(ft % tiles, m0, n0);
    offsets(m0, n0, values_of(fg));
    start(m0, n0, fg);
    auto advance = [&]() __attribute__((always_inline)) {
        if (++fg < fg_end) {
            next_b += TALL_B ? p.ldb * 128 : 128;
            next_a += TALL_A ? p.lda * 128 : 128;
            if (values_of(fg) < 64) offsets(m0, n0, values_of(fg));
            return;
        }
        if (ft + gridDim.x < items) {  // behind the last item its steps are fetched once more and not used
            ft += gridDim.x;
            place(ft % tiles, m0, n0);
        }
        fg = first_step(ft);
        fg_end = last_step(ft);
        offsets(m0, n0, values_of(fg));
        start(m0, n0, fg);
    };
    each<2>([&](auto s) __attribute__((always_inline)) {
        if constexpr (s > 0) advance();
        each<LA>([&](auto i) __attribute__((always_inline)) { fetch_a(2 * s * kPart, i); });
        each<LB>([&](auto i) __attribute__((always_inline)) { fetch_b((2 * s + 1) * kPart, i); });
    });
    wait_vm_and_lds_then_barrier<0>();
    if (values_of(first_step(first)) < 64) clear_excess(0, kPart, values_of(first_step(first)));
#pragma unroll
    for (int i = 0; i < FN + FM; ++i) read_frag(0, kPart, 0, i);
    // The parts of LDS in the order of their use: A's and B's of the step in work and of
    // the next, and a free one.
    uint32_t ring[5] = {0, kPart, 2 * kPart, 3 * kPart, 4 * kPart};

    f32x4 acc[FN][FM];
    // Between what the compiler knows to be done with the accumulators and what it does
    // not. Behind that they are read by lines of their own, where they are needed: the
    // compiler would read all of them first, and spill.
    auto settle = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) asm volatile("" : "+a"(acc[i][j]));
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    };
    auto sums = [&](int i, int j) __attribute__((always_inline)) {
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float one;
            asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(one) : "a"(acc[i][j][r]));
            v[r] = one;
        }
        return v;
    };
    // A phase. A wavefront issues in order, and a matrix instruction occupies its unit
    // for 16 cycles: the few other instructions that the phase needs are dealt out
    // between them, reads of the next phase's fragments and loads, A's of a step in its
    // first phase and B's in the second.
    auto phase = [&](auto f) __attribute__((always_inline)) {
        constexpr int D = FN + FM, kInstr = FN * FM, kLoads = f == 0 ? LA : LB, kItems = D + kLoads, kRun = D / kLoads + 1;
        each<kInstr>([&](auto q) __attribute__((always_inline)) {
            each<(q + 1) * kItems / kInstr - q * kItems / kInstr>([&](auto r) __attribute__((always_inline)) {
                constexpr int item = q * kItems / kInstr + r;
                if constexpr (item % kRun < kRun - 1) read_frag(ring[f == 0 ? 0 : 2], ring[f == 0 ? 1 : 3], 1 - f, item - item / kRun);
                else if constexpr (f == 0) fetch_a(ring[4], std::integral_constant<int, item / kRun>{});
                else fetch_b(ring[0], std::integral_constant<int, item / kRun>{});
            });
            __builtin_amdgcn_sched_barrier(0);
            constexpr int i = q / FM, j = q % FM;
            mfma16x16(fb[f][i], fa[f][j], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    for (uint32_t t = first; t < items; t += gridDim.x) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.0f;
        settle();
        int64_t cm0 = m0, cn0 = n0;
        if (ft != t) place(t % tiles, cm0, cn0);
        // A step. Scalar work between two phases would let the matrix unit run empty: in the
        // plain ones, whose fetched step lies 64 whole values on, there is next to none.
        uint32_t g = first_step(t);
        const uint32_t g1 = last_step(t);
        auto step = [&](auto plain) __attribute__((always_inline)) {
            if constexpr (plain) {
                next_b += TALL_B ? p.ldb * 128 : 128;
                next_a += TALL_A ? p.lda * 128 : 128;
            } else {
                advance();
            }
            phase(std::integral_constant<int, 0>{});
            // still running at most: A's loads of the step after the next
            wait_vm_and_lds_then_barrier<LA>();
            if constexpr (!plain) {
                const uint32_t values = g + 1 < g1 ? values_of(g + 1) : (t + gridDim.x < items ? values_of(first_step(t + gridDim.x)) : 64);
                if (values < 64) clear_excess(ring[2], ring[3], values);
            }
            phase(std::integral_constant<int, 1>{});
            const uint32_t r0 = ring[0], r1 = ring[1];
            ring[0] = ring[2];
            ring[1] = ring[3];
            ring[2] = ring[4];
            ring[3] = r0;
            ring[4] = r1;
        };
        const uint32_t whole = fg_end == steps && (k & 63) != 0 ? fg_end - 1 : fg_end;
        uint32_t plain = ft == t && fg + 1 < whole ? whole - 1 - fg : 0;
        fg += plain;
        g += plain;
#pragma nounroll
        for (; plain > 0; --plain) step(std::true_type{});
#pragma nounroll
        for (; g < g1; ++g) step(std::false_type{});
        settle();
        if constexpr (Out::kLogSum) {
            constexpr int kCols = FN * 16;
            static_assert(kCols == log_sum_width(BN == 256 ? Way16::kTile256 : Way16::kTile128), "as the workspace is laid out");
            const int64_t col0 = cn0 + wn;
            const int cols = (int)(n - col0 < kCols ? n - col0 : kCols);
            if (cols > 0) {
                int32_t labels[FM];
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const int64_t row = cm0 + wm + j * 16 + l16;
                    labels[j] = out.label_of(row < m ? row : m - 1);
                }
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const int64_t row = cm0 + wm + j * 16 + l16;
                    const int64_t label = row < m ? (int64_t)labels[j] - col0 : -1;
                    const float ninf = -__builtin_inff();
                    f32x4 v[FN];
#pragma unroll
                    for (int i = 0; i < FN; ++i) v[i] = sums(i, j);
                    if (cols < kCols) {
#pragma unroll
                        for (int i = 0; i < FN; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (i * 16 + 4 * quad + r >= cols) v[i][r] = ninf;
                    }
                    const bool holds = label >= 0 && label < cols;
                    if (__any(holds)) {
                        float own = 0.0f;
#pragma unroll
                        for (int i = 0; i < FN; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const bool hit = i * 16 + 4 * quad + r == label;
                                own = hit ? v[i][r] : own;
                                v[i][r] = hit ? ninf : v[i][r];
                            }
                        if (holds && quad == (label >> 2 & 3)) out.keep(row, own);
                    }
                    float top = ninf, sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < FN; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) top = fmaxf(top, v[i][r]);
                    top = fmaxf(top, __shfl_xor(top, 16, kWave));
                    top = fmaxf(top, __shfl_xor(top, 32, kWave));
                    if (top == ninf) top = 0.0f;
#pragma unroll
                    for (int i = 0; i < FN; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) sum += exp_fast(v[i][r] - top);
                    sum += __shfl_xor(sum, 16, kWave);
                    sum += __shfl_xor(sum, 32, kWave);
                    if (quad == 0 && row < m) out.put(row, col0 / kCols, top, sum);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        } else {
            // Out through LDS of this wavefront's own, 32 rows of PIECE fp32 at a time, so that
            // a lane has 8 columns of a row: chunk c of row r lies at position c ^ (r % chunks).
            uint8_t* const mine = lds + ring[4] + wave * 32 * PIECE * 4;
            constexpr int kChunks = PIECE / 4, kLanes = PIECE / 8, kFrags = PIECE / 16, kRows = 32 * kLanes / kWave;
            constexpr int kAcross = FN / kFrags, kPieces = FM / 2 * kAcross;
            const int lr = lane / kLanes, lc = lane % kLanes;
            float* const part = items_of.splits > 1 ? items_of.part + t / tiles * items_of.stride : nullptr;
#pragma nounroll
            for (int piece = 0; piece < kPieces; ++piece) {
                const int64_t row0 = cm0 + wm + piece / kAcross * 32 + lr, col = cn0 + wn + piece % kAcross * PIECE + lc * 8;
                const bool here = col < n;
                typename Out::Column column = {};
                typename Out::Row rows[kRows] = {};
                if (!part && here) {
                    column = out.column(col, n - col);
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (row0 + r * (32 / kRows) < m) rows[r] = out.row(row0 + r * (32 / kRows), col, n - col);
                }
                each<kPieces>([&](auto which) __attribute__((always_inline)) {
                    if (which == piece) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int b = 0; b < kFrags; ++b) {
                                const int row = h * 16 + l16, c = b * 4 + quad;
                                *reinterpret_cast<f32x4*>(mine + row * PIECE * 4 + (c ^ (row & (kChunks - 1))) * 16) =
                                    sums(which % kAcross * kFrags + b, which / kAcross * 2 + h);
                            }
                    }
                });
                exchange_between_lanes();
                float v[kRows][8];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int row = lr + r * (32 / kRows);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f32x4 q = *reinterpret_cast<const f32x4*>(mine + row * PIECE * 4 + ((2 * lc + h) ^ (row & (kChunks - 1))) * 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[r][4 * h + e] = q[e];
                    }
                }
                exchange_between_lanes();  // the next piece's take the place of these
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int64_t row = row0 + r * (32 / kRows);
                    if (here && row < m) {
                        if (part) store8<true>(part + row * items_of.ld + col, 8, v[r]);
                        else out(row, col, v[r], n - col, column, rows[r]);
                    }
                }
            }
            // the free part is every wavefront's before the next step is loaded into it
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    }
    // nothing may still be on its way into LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Adds the partial sums of the splits, in their order: 8 columns a thread.
template <class Out>
__global__ __launch_bounds__(kBlock) void product_join_kernel(Items items, const int32_t* __restrict__ m_at, int64_t m, int64_t n, Out out) {
    if (m_at) m = (int64_t)*gp(m_at);
    const int64_t blocks = items.ld / 8, total = m * blocks;
    out.begin();
    for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < total; i += (int64_t)gridDim.x * kBlock) {
        const int64_t row = i / blocks, col = (i - row * blocks) * 8;
        if (col >= n) continue;
        const float* const at = items.part + row * items.ld + col;
        float v[8];
        expand(load_raw8<true>(at, 8), v);
        for (uint32_t s = 1; s < items.splits; ++s) {
            float w[8];
            expand(load_raw8<true>(at + s * items.stride, 8), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += w[e];
        }
        finish(out, row, col, v, n - col);
    }
}

// ------------------------------------------------------------------ few rows of A
//
// Bound by reading B once: 1 x 13824 x 5120 (142 MB) takes 28 us in the kernel (5.0 TB/s) and 32.4 as
// a call. A workgroup takes 16 rows of B; its wavefronts take a part of k each, straight from
// global memory into registers at any alignment, and add their sums through LDS in order. Up to
// 16 rows of A; rows past the end are read as the last one and not used.
constexpr int kFewWaves = 8;
constexpr int kFewAhead = 4;  // loads of each operand under way together

template <class Out>
__global__ __launch_bounds__(kFewWaves* kWave) void product_few_kernel(Product16 p, int64_t per, Out out) {
    __shared__ float sums[kFewWaves][4][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, quad = lane >> 4, l16 = lane & 15;
    const int64_t n0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 16;
    const int64_t m = p.m_at ? (int64_t)__builtin_amdgcn_readfirstlane(*gp(p.m_at)) : p.m, n = p.n;
    if (n0 >= n || m == 0) return;
    const int64_t ra = l16 < m ? l16 : m - 1, rb = n0 + l16 < n ? n0 + l16 : n - 1;
    const int64_t k1 = (wave + 1) * per < p.k ? (wave + 1) * per : p.k;  // a multiple of 8, or the end
    const uint16_t* const pa = p.a + (p.a_rows ? (int64_t)gp(p.a_rows)[ra] : ra) * p.lda;
    const uint16_t* const pb = p.b + rb * p.ldb;
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    int64_t k0 = wave * per + quad * 8;
    for (; k0 - quad * 8 + 32 * kFewAhead <= k1; k0 += 32 * kFewAhead) {
        u32x4 a[kFewAhead], b[kFewAhead];
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) b[i] = *reinterpret_cast<const gu32x4_a2*>(gp(pb) + k0 + 32 * i);
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) a[i] = *reinterpret_cast<const gu32x4_a2*>(gp(pa) + k0 + 32 * i);
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[i]), __builtin_bit_cast(bf16x8, a[i]), acc, 0, 0, 0);
    }
    for (; k0 - quad * 8 < k1; k0 += 32) {  // values past the end of the part are zero
        const u32x4 b = load_raw8(pb + k0, k1 - k0).w, a = load_raw8(pa + k0, k1 - k0).w;
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wave][r][lane] = acc[r];
    __syncthreads();
    const int waves = blockDim.x / kWave;
    auto total = [&](int row, int col) {  // accumulator r of lane l is row l % 16, column 4 (l / 16) + r
        const int r = col & 3, at = (col >> 2) * 16 + row;
        float v = sums[0][r][at];
        for (int w = 1; w < waves; ++w) v += sums[w][r][at];
        return v;
    };
    if constexpr (Out::kLogSum) {
        static_assert(log_sum_width(Way16::kFew) == 16);
        // 16 lanes a row, a column each
        const int row = threadIdx.x / 16, col = threadIdx.x & 15;
        if (row >= 16) return;
        const int64_t label = row < m ? (int64_t)out.label_of(row) - n0 : -1;
        float v = -__builtin_inff();
        if (n0 + col < n) {
            v = total(row, col);
            if (col == label) {
                out.keep(row, v);
                v = -__builtin_inff();
            }
        }
        float top = v;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
        if (top == -__builtin_inff()) top = 0.0f;
        float sum = exp_fast(v - top);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d, kWave);
        if (col == 0 && row < m) out.put(row, n0 / 16, top, sum);
    } else {
        const int row = threadIdx.x >> 1, col = (threadIdx.x & 1) * 8;
        if (row >= m || n0 + col >= n) return;
        out.begin();
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = total(row, col + e);
        finish(out, row, n0 + col, v, n - n0 - col);
    }
}

template <class Out>
int launch_few(const Product16& p, const Out& out, hipStream_t st) {
    // whole turns of the loop for each wavefront but the last
    const int64_t turn = 32 * kFewAhead, per = div_up(p.k, kFewWaves * turn) * turn;
    const unsigned threads = (unsigned)div_up(p.k, per) * kWave < 256u ? 256u : (unsigned)div_up(p.k, per) * kWave;
    const Grid g = grid_xy(div_up(p.n, 16), threads);
    hipLaunchKernelGGL((product_few_kernel<Out>), dim3(g.x, g.y), dim3(threads), 0, st, p, per, out);
    return launch_status();
}

// The product by the plan that the host logic makes for it; ws: the partial sums of its splits.
template <class S, bool TALL_A, bool TALL_B, class Out>
int launch_tiles(const Product16& p, const Plan16& plan, float* ws, const Out& out, hipStream_t st) {
    const Items items{plan.tiles_n, plan.splits, plan.per_split, ws, plan.ld, plan.stride};
    const int64_t count = (int64_t)plan.tiles_m * plan.tiles_n * plan.splits, most = kCUs * (S::kWavesPerSimd * 4 / S::WAVES);
    hipLaunchKernelGGL((product_tile_kernel<S, TALL_A, TALL_B, Out>), dim3((unsigned)(count < most ? count : most)), dim3(S::WAVES * kWave), 0, st,
                       p, items, out);
    if constexpr (!Out::kLogSum) {
        if (plan.splits > 1) {
            const int64_t groups = div_up(p.m * (plan.ld / 8), kBlock);
            hipLaunchKernelGGL(product_join_kernel<Out>, dim3((unsigned)(groups < 16 * kCUs ? groups : 16 * kCUs)), dim3(kBlock), 0, st, items,
                               p.m_at, p.m, p.n, out);
        }
    }
    return launch_status();
}

// Rows of an operand that tiles do not take: the first `cols` values of each, to rows of ld
// (a multiple of 8) with zeros behind them; of rows at[0] .. at[*count - 1], if they are given.
struct Pack {
    const uint16_t* x;
    int64_t rows, ldx;
    const int32_t *at, *count;
    uint16_t* packed;
    bool finite = false;  // with zeros for infinities and NaN
};
// Up to two operands in one launch, 8 values a thread.
__global__ __launch_bounds__(kBlock) void pack_rows_kernel(Pack first, Pack second, int64_t cols, int64_t ld) {
    const Pack p = blockIdx.y == 0 ? first : second;
    const int64_t rows = p.count ? (int64_t)*gp(p.count) : p.rows;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const uint16_t* const from = p.x + (p.at ? (int64_t)gp(p.at)[r] : r) * p.ldx;
        for (int64_t c = threadIdx.x * 8; c < ld; c += kBlock * 8) {
            const u32x4 v = load_raw8(from + c, cols - c).w;
            *reinterpret_cast<gu32x4*>(gp(p.packed) + r * ld + c) = p.finite ? finite_of(v) : v;
        }
    }
}
inline int launch_pack(const Pack& first, const Pack& second, int64_t cols, hipStream_t st) {
    const int64_t rows = first.rows > second.rows ? first.rows : second.rows;
    hipLaunchKernelGGL(pack_rows_kernel, dim3((unsigned)(rows < 64 * kCUs ? rows : 64 * kCUs), second.rows > 0 ? 2u : 1u), dim3(kBlock), 0, st,
                       first, second, cols, packed_ld(cols));
    return launch_status();
}

template <bool TALL_A, bool TALL_B, class Out>
int launch_product(const Product16& p, const Plan16& plan, float* ws, const Out& out, hipStream_t st) {
    if (p.m == 0 || p.n == 0) return COAT_OK;
    if constexpr (Out::kLarge) {
        if (plan.way == Way16::kTile256) return launch_tiles<Tile256, TALL_A, TALL_B>(p, plan, ws, out, st);
    }
    if (plan.way == Way16::kTile128) return launch_tiles<Tile128, TALL_A, TALL_B>(p, plan, ws, out, st);
    if constexpr (!TALL_A && !TALL_B) {
        if (plan.way == Way16::kFew) return launch_few(p, out, st);
    }
    const int64_t tn = div_up(p.n, 64), tiles = tn * div_up(p.m, 64);
    if (tiles > 0x7FFFFFFFll * 64) return COAT_EINVAL;
    const Grid g = grid_xy(tiles, kBlock);
    hipLaunchKernelGGL((product_plain_kernel<TALL_A, TALL_B, Out>), dim3(g.x, g.y), dim3(kBlock), 0, st, p, (uint32_t)tn, out);
    return launch_status();
}

}  // namespace

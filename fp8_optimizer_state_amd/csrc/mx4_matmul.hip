// HIP (gfx950) product of two matrices in microscaled 4-bit floating point.
#include <type_traits>

#include "mx4_common.h"

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// One matrix instruction takes 32 rows of each operand over 64 values of k: lane
// l holds the 32 codes of row l % 32 in block l / 32, and their scale byte.
// Two of them take a row's 64 code bytes and 4 scale bytes: chunk l / 32 and
// scale byte l / 32 first, then chunk 2 + l / 32 and scale byte 2 + l / 32; the
// scale word is shifted by l / 32 bytes once, and the instruction selects its
// byte 0 or 2. B is the first operand, so that a lane's four consecutive
// accumulators are four consecutive columns of y: accumulator r of lane l is
// y[l % 32][8 (r / 4) + 4 (l / 32) + r % 4].
template <int SEL>
__device__ __forceinline__ f32x16 mfma_fp4(const u32x4& b, const u32x4& a, const f32x16& acc, uint32_t sb, uint32_t sa) {
    const i32x8 vb{(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const i32x8 va{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, acc, 4, 4, SEL, (int)sb, SEL, (int)sa);
}

// The plain product, straight from global memory: each wavefront a 32 x 32 tile, a
// workgroup 64 x 64. Rows past the end are read as the last row and not stored.
// For what the others do not take: k = 0 (zeros), rows of 2^22 values or more,
// whose bytes pass the 32-bit offsets within a tile, and more tiles than a 32-bit
// count. Bound by its own loads' latency: nothing is fetched ahead.
template <class T>
__global__ __launch_bounds__(kBlock) void mx4_matmul_small_kernel(const uint8_t* __restrict__ aq,
                                                                  const uint8_t* __restrict__ as, int64_t m,
                                                                  const uint8_t* __restrict__ bq,
                                                                  const uint8_t* __restrict__ bs, int64_t n, int64_t k,
                                                                  uint32_t tiles_n, T* __restrict__ y, int64_t ld) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint32_t tile = blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t n0 = (int64_t)(tile % tiles_n) * 64 + (wave & 1) * 32;
    const int64_t m0 = (int64_t)(tile / tiles_n) * 64 + (wave >> 1) * 32;
    if (m0 >= m) return;
    const int row = lane & 31, half = lane >> 5;
    const int64_t qb = mx4_code_bytes(k), sb = mx4_scale_bytes(k);
    const int64_t ra = m0 + row < m ? m0 + row : m - 1, rb = n0 + row < n ? n0 + row : n - 1;
    const uint8_t *pa = aq + ra * qb + half * 16, *pb = bq + rb * qb + half * 16;
    const uint8_t *psa = as + ra * sb, *psb = bs + rb * sb;
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    const int64_t steps = div_up(k, 128);
    for (int64_t t = 0; t < steps; ++t) {
        const u32x4 a0 = *reinterpret_cast<const gu32x4*>(gp(pa) + t * 64);
        const u32x4 a1 = *reinterpret_cast<const gu32x4*>(gp(pa) + t * 64 + 32);
        const u32x4 b0 = *reinterpret_cast<const gu32x4*>(gp(pb) + t * 64);
        const u32x4 b1 = *reinterpret_cast<const gu32x4*>(gp(pb) + t * 64 + 32);
        const uint32_t sa = *reinterpret_cast<const gu32*>(gp(psa) + t * 4) >> (8 * half);
        const uint32_t sbw = *reinterpret_cast<const gu32*>(gp(psb) + t * 4) >> (8 * half);
        acc = mfma_fp4<0>(b0, a0, acc, sbw, sa);
        acc = mfma_fp4<2>(b1, a1, acc, sbw, sa);
    }
    if (m0 + row >= m) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t c = n0 + 8 * (r / 4) + 4 * half + r % 4;
        if (c < n) {
            if constexpr (sizeof(T) == 4) gp(y)[(m0 + row) * ld + c] = acc[r];
            else gp(y)[(m0 + row) * ld + c] = (uint16_t)bf16_bits(acc[r]);
        }
    }
}

// ------------------------------------------------------------------ large tiles
//
// A workgroup of WN x WM wavefronts, each with 32 FN rows of B by 32 FM rows of
// A, computes tiles one after the other; the k of all its tiles forms one stream
// of steps of 128 values, two steps a pair, four a group. A pair's codes (128
// bytes a row, B's rows before A's) go straight from global memory into one of
// PAIRS slots of LDS, PAIRS pairs before they are used; a group's scale bytes
// (16 a row) likewise. 128 bytes a row, because a compute unit takes in 130
// bytes a nanosecond in such runs and 80 in runs of 64.
//
// A pair is computed in phases: while one phase's matrix instructions run, the
// next one's fragments are read from LDS. One barrier a pair, before its last
// phase: behind it every wavefront has read the pair (its slot may be refilled)
// and the next pair has arrived.
//
// LDS reads are 16 bytes a lane from 32 rows 128 bytes apart; chunk c of row r
// lies at position c ^ (r / 2 % 8), so that any 16 rows reach 16 different
// 16-byte columns of the banks. The loads write LDS in lane order, so the lane
// that fills position p of row r fetches chunk p ^ (r / 2 % 8).
//
// Tiles of 256 x 256 (four wavefronts of 128 x 128 values, 160 KB of LDS) are bound
// by the matrix units: 16384 x 13824 x 5120 takes 550 us (4.2 PFLOP/s). They are
// busy for 57 % of the cycles, at 1.7 to 1.85 GHz: on codes of zero, which switch
// nothing, the same launch runs at 2.4 GHz and 5.3 PFLOP/s. What is left of the
// cycles goes to writing y (5 to 7 us a tile, in part under the next one's loads).
// Tiles of 128 x 128 are bound by latency, with one wavefront a SIMD and a barrier a
// pair: reads of LDS are active in 0.39 of the cycles, the matrix units in 0.39, and the
// wavefronts wait in 0.28 (1500 x 5120 x 13824, 77 us). 16384 x 13824 x 5120 takes 747 us
// in them.
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

__device__ __forceinline__ uint32_t float_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

// A 16-byte chunk of y. PAST: written past the caches' usual order, where y would
// drive the operands out of them (16384 x 16384 x 512 to bf16 in large tiles: 158
// us against 214). Not where the pieces of a row end within a line, whose halves
// would go to memory one by one (4097 x 5001 x 2000 to fp32: 77 us against 50;
// 16384 x 13823 x 5120 643 against 594).
template <bool PAST>
__device__ __forceinline__ void store_chunk(float* p, const u32x4& w) {
    if constexpr (PAST) __builtin_nontemporal_store(w, reinterpret_cast<gu32x4_a4*>(gp(p)));
    else *reinterpret_cast<gu32x4_a4*>(gp(p)) = w;
}
template <bool PAST>
__device__ __forceinline__ void store_chunk(uint16_t* p, const u32x4& w) {
    if constexpr (PAST) __builtin_nontemporal_store(w, reinterpret_cast<gu32x4_a2*>(gp(p)));
    else *reinterpret_cast<gu32x4_a2*>(gp(p)) = w;
}

// The same, or nothing if `on` is 0 (one branch within a long run of code).
template <uint32_t AT>
__device__ __forceinline__ void load_to_lds16_if(uint32_t on, uint32_t lds, uint32_t off, const uint8_t* base) {
    asm volatile(
        "s_cmp_eq_u32 %4, 0\n\ts_cbranch_scc1 .Lskip%=\n\ts_add_u32 m0, %0, %3\n\ts_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2\n.Lskip%=:" ::"s"(lds), "v"(off), "s"(base), "n"(AT), "s"(on)
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

// Where a workgroup reads its next group of steps.
struct Stream {
    const uint8_t *bq, *aq, *bs, *as;  // first rows of the tile, at the group's first step
    uint32_t left;                     // steps from there to the end of k
    // Byte offset of the second pair, and for each pair what this lane's offset is
    // too large by, if the pair's second step is past the end of k. What is past
    // the end is not read: the first pair, or step, is fetched instead and not used.
    uint32_t second, back[2];
};

// With splits > 1 item t is the product over the groups of four steps
// [s per_split, (s + 1) per_split), s = t / tiles, of tile t % tiles, and goes to
// y + s part (partial sums, added by another kernel).
template <int WN, int WM, int FN, int FM, int PAIRS, int PIECE, class T>
__global__ __launch_bounds__(WN* WM* kWave) __attribute__((amdgpu_waves_per_eu(WN* WM / 4, WN* WM / 4))) void mx4_matmul_tile_kernel(
    const uint8_t* __restrict__ aq, const uint8_t* __restrict__ as, int64_t m, const uint8_t* __restrict__ bq,
    const uint8_t* __restrict__ bs, int64_t n, int64_t k, uint32_t tiles_m, uint32_t tiles_n, uint32_t splits,
    uint32_t per_split, T* __restrict__ y, int64_t ld, int64_t part) {
    // D fragments of a half step; L loads of a pair (LB of them B's) and SC of a group's scale bytes by each wavefront
    constexpr int WAVES = WN * WM, BN = 32 * WN * FN, BM = 32 * WM * FM, D = FN + FM, SETS = PAIRS / 2;
    constexpr int L = (BN + BM) / 8 / WAVES, LB = BN / 8 / WAVES, kScaleLoads = (BN + BM) / 64;
    constexpr int SC = kScaleLoads < WAVES ? 1 : kScaleLoads / WAVES;
    static_assert(LB * 8 * WAVES == BN && L * 8 * WAVES == BN + BM && L % 2 == 0 && BN % 64 == 0, "loads are dealt evenly");
    static_assert(kScaleLoads % WAVES == 0 || WAVES % kScaleLoads == 0, "scale loads too, or repeated");
    constexpr bool AHEAD = FN * FM <= 4;  // a phase is a step, not half a step
    constexpr int PHASES = AHEAD ? 2 : 4;
    constexpr uint32_t kSlotBytes = (BN + BM) * 128, kScaleBytes = (BN + BM) * 16;
    // stores of a whole tile, an exact count: later waits let them run
    constexpr int kStores = FN * FM * (sizeof(T) == 4 ? 4 : 2);
    __shared__ __attribute__((aligned(16))) uint8_t lds[PAIRS * kSlotBytes + (SETS + 1) * kScaleBytes + WAVES * 32 * PIECE];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int half = lane >> 5, l32 = lane & 31;
    const int64_t qb = mx4_code_bytes(k), sb = mx4_scale_bytes(k);
    const uint32_t steps = (uint32_t)(qb / 64), groups = (steps + 3) / 4;
    const uint32_t tiles = tiles_m * tiles_n, items = tiles * splits;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

    // tile t: patches of 8 x 4 tiles are consecutive
    auto place = [&](uint32_t t, int64_t& m0, int64_t& n0) {
        const uint32_t per = 8 * tiles_n, band = t / per, in = t - band * per;
        const uint32_t high = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8;
        m0 = (int64_t)(band * 8 + in % high) * BM;
        n0 = (int64_t)(in / high) * BN;
    };
    // byte offsets of this lane's chunks and scale words from the tile's first rows
    const uint32_t chunk = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
    const uint32_t back = chunk >= 4 ? 64 : 0;  // to the same chunk of the pair's first step
    uint32_t off[L], soff[SC];
    // with more wavefronts than loads of scale bytes they are made twice, so that every wavefront counts alike
    const int swave = wave % kScaleLoads;
    auto offsets = [&](int64_t m0, int64_t n0) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const uint32_t row = (uint32_t)(i * WAVES + wave) * 8 + lane / 8 - (i < LB ? 0 : BN);
            const int64_t left = (i < LB ? n - n0 : m - m0) - 1;  // the last row stands in for those past the end
            off[i] = (row < left ? row : (uint32_t)left) * (uint32_t)qb + chunk * 16;
        }
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            uint32_t row = (uint32_t)(i * WAVES + swave) * 64 + lane;
            const bool is_b = row < BN;
            if (!is_b) row -= BN;
            const int64_t left = (is_b ? n - n0 : m - m0) - 1;
            soff[i] = (row < left ? row : (uint32_t)left) * (uint32_t)sb;
        }
    };
    const uint32_t lds_wave = lds0 + wave * 1024;
    auto fetch_part = [&](const Stream& at, int set, auto pair, auto i, uint32_t on = 1) {
        const uint8_t* from = (i < LB ? at.bq : at.aq) + (pair == 1 ? at.second : 0);
        const uint32_t to = lds_wave + set * 2 * kSlotBytes, lane_off = off[i] - at.back[pair];
        if (__builtin_constant_p(on)) load_to_lds16<pair * kSlotBytes + i * WAVES * 1024>(to, lane_off, from);
        else load_to_lds16_if<pair * kSlotBytes + i * WAVES * 1024>(on, to, lane_off, from);
    };
    auto fetch_scales = [&](const Stream& at, int slot) {
        each<SC>([&](auto i) {
            load_to_lds16<PAIRS * kSlotBytes + i * WAVES * 1024>(lds0 + swave * 1024 + slot * kScaleBytes, soff[i],
                                                                 (i * WAVES + swave) * 64 < BN ? at.bs : at.as);
        });
    };
    auto settle = [&](Stream& at) {
        at.second = at.left > 2 ? 128 : 0;
        at.back[0] = at.left == 1 ? back : 0;
        at.back[1] = at.left == 1 || at.left == 3 ? back : 0;
        asm volatile("" : "+v"(at.back[0]), "+v"(at.back[1]));  // held, not computed at each use
    };
    auto stream_of = [&](int64_t m0, int64_t n0, uint32_t g) {
        Stream at{bq + n0 * qb + g * 256, aq + m0 * qb + g * 256, bs + n0 * sb + g * 16, as + m0 * sb + g * 16, steps - 4 * g, 0, {0, 0}};
        settle(at);
        return at;
    };

    u32x4 fb[AHEAD ? 2 : 1][2][FN], fa[AHEAD ? 2 : 1][2][FM];  // fragments, [parity of the step][half]
    uint32_t cb[2][FN], ca[2][FM];                             // scale words, by parity of the step
    const int wn = wave % WN * FN * 32, wm = wave / WN * FM * 32;
    // fragment i of half h of step sp of a pair: A's first, which every row of matrix instructions needs
    auto read_frag = [&](int set, int pair, int sp, int h, int i) {
        const int pos = ((4 * sp + 2 * h + half) ^ ((l32 >> 1) & 7)) * 16;
        const uint8_t* slot = lds + (set * 2 + pair) * kSlotBytes + pos + l32 * 128;
        if (i < FM) fa[AHEAD ? sp : 0][h][i] = *reinterpret_cast<const u32x4*>(slot + (BN + wm + i * 32) * 128);
        else fb[AHEAD ? sp : 0][h][i - FM] = *reinterpret_cast<const u32x4*>(slot + (wn + (i - FM) * 32) * 128);
    };
    auto read_scale = [&](int slot, int u, int i) {
        const uint8_t* at = lds + PAIRS * kSlotBytes + slot * kScaleBytes + u * 4 + l32 * 16;
        if (i < FM) ca[u & 1][i] = *reinterpret_cast<const uint32_t*>(at + (BN + wm + i * 32) * 16);
        else cb[u & 1][i - FM] = *reinterpret_cast<const uint32_t*>(at + (wn + (i - FM) * 32) * 16);
    };
    // Moves this half's scale bytes into place. A step past the end of k (its
    // codes are those of another one) gets scale bytes 0 instead: every product
    // is at most 36 * 2^-254 then, and adds nothing to an fp32 sum.
    auto shift_scales = [&](int p, bool work) {
        const uint32_t width = work ? 24u : 0u;
        // not before here: the words are still on their way while matrix instructions can be issued
#pragma unroll
        for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(ca[p][i]));
#pragma unroll
        for (int i = 0; i < FN; ++i) asm volatile("" : "+v"(cb[p][i]));
#pragma unroll
        for (int i = 0; i < FM; ++i) ca[p][i] = __builtin_amdgcn_ubfe(ca[p][i], 8 * half, width);
#pragma unroll
        for (int i = 0; i < FN; ++i) cb[p][i] = __builtin_amdgcn_ubfe(cb[p][i], 8 * half, width);
    };

    // consecutive workgroups run on different XCDs: each XCD takes consecutive items of a round
    const uint32_t first = gridDim.x % 8 == 0 ? (blockIdx.x & 7) * (gridDim.x / 8) + (blockIdx.x >> 3) : blockIdx.x;
    if (first >= items) return;
    // the group that is fetched next, SETS groups before it is used: group fg of item ft
    uint32_t ft = first, fg = first / tiles * per_split;
    int64_t m0, n0;
    place(ft % tiles, m0, n0);
    offsets(m0, n0);
    Stream next = stream_of(m0, n0, fg);
    uint32_t group_end = fg + per_split < groups ? fg + per_split : groups;  // of item ft
    auto advance = [&] {
        if (++fg < group_end) {
            next.bq += 256;
            next.aq += 256;
            next.bs += 16;
            next.as += 16;
            next.left -= 4;
            settle(next);
            return;
        }
        if (ft + gridDim.x < items) {  // behind the last item its groups are fetched once more and not used
            ft += gridDim.x;
            place(ft % tiles, m0, n0);
            offsets(m0, n0);
        }
        fg = ft / tiles * per_split;
        group_end = fg + per_split < groups ? fg + per_split : groups;
        next = stream_of(m0, n0, fg);
    };
    using zero = std::integral_constant<int, 0>;
    using one = std::integral_constant<int, 1>;
    // With two slots the last pair's later loads follow before the first phase.
    constexpr int kLast = PAIRS > 2 ? L / 2 : L;
    each<SETS>([&](auto set) {
        if constexpr (set > 0) advance();
        fetch_scales(next, set);
        each<L>([&](auto i) { fetch_part(next, set, zero{}, i); });
        each<(set + 1 < SETS ? L : kLast)>([&](auto i) { fetch_part(next, set, one{}, i); });
    });
    wait_vm_and_lds_then_barrier<0>();
#pragma unroll
    for (int i = 0; i < D; ++i) {
        read_frag(0, 0, 0, 0, i);
        if constexpr (AHEAD) read_frag(0, 0, 0, 1, i);
        read_scale(0, 0, i);
    }
    shift_scales(0, true);
    // Set of slots and scale slot of the group in work, and of the next one; scales are
    // fetched into the one scale slot that neither these nor the groups between hold.
    int set = 0, sslot = 0;
    auto next_set = [&] { return SETS == 1 ? 0 : (set + 1 < SETS ? set + 1 : 0); };
    auto next_sslot = [&] { return sslot < SETS ? sslot + 1 : 0; };
    auto free_sslot = [&] { return sslot > 0 ? sslot - 1 : SETS; };
    uint32_t t = first, g = 0;
    const bool lines = FN * FM <= 4 || (((uintptr_t)y | ((uint64_t)ld * sizeof(T))) & 127) == 0;  // a piece fills lines of y

    f32x16 acc[FN][FM];
    // A phase. A wavefront issues in order, and a matrix instruction occupies its
    // unit for 32 cycles: the few other instructions that the phase needs are dealt
    // out between them, first the reads of the next phase's fragments (and scale
    // words, if that begins a step), then loads into LDS: half of a pair's in its
    // predecessor's last phase, the others (carry) in the phase behind that.
    auto phase = [&](auto pair, auto f, uint32_t carry) {
        constexpr int kInstr = AHEAD ? 2 * FN * FM : FN * FM;
        constexpr bool last = f == PHASES - 1, new_step = AHEAD || f % 2 == 1;
        constexpr int kReads = AHEAD ? 2 * D : D, kItems = kReads + (last || f == 0 ? L / 2 : 0);
        constexpr int u = 2 * pair + (AHEAD ? f : f / 2), p = u & 1;  // step of the group
        each<kInstr>([&](auto q) {
            each<(q + 1) * kItems / kInstr - q * kItems / kInstr>([&](auto r) {
                constexpr int item = q * kItems / kInstr + r;
                if constexpr (item < kReads) {
                    constexpr int nf = (f + 1) % PHASES;  // the phase that is read for
                    constexpr int sp = AHEAD ? nf : nf / 2, h = AHEAD ? item / D : nf % 2;
                    if constexpr (new_step && item < D)
                        read_scale(u == 3 ? next_sslot() : sslot, (u + 1) & 3, item);
                    read_frag(last && pair == 1 ? next_set() : set, last ? 1 - pair : pair, sp, h, item % D);
                } else if constexpr (last) {
                    fetch_part(next, set, pair, std::integral_constant<int, item - kReads>{});
                } else {
                    fetch_part(next, pair == 1 ? set : (set > 0 ? set - 1 : SETS - 1), std::integral_constant<int, 1 - pair>{},
                               std::integral_constant<int, item - kReads + L / 2>{}, PAIRS > 2 || pair == 1 ? 1 : carry);
                }
            });
            __builtin_amdgcn_sched_barrier(0);
            constexpr int h = AHEAD ? q / (FN * FM) : f % 2, i = q / FM % FN, j = q % FM;
            constexpr int r = AHEAD ? p : 0;
            acc[i][j] = mfma_fp4<2 * h>(fb[r][h][i], fa[r][h][j], acc[i][j], cb[p][i], ca[p][j]);
            asm volatile("" : "+a"(acc[i][j]));  // keeps the order
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (new_step) shift_scales(p ^ 1, u == 3 || 4 * g + u + 1 < steps);
    };
    // A pair. `after_stores`: the loads of the next one were all issued before the
    // last item's stores, which may still run when it is needed.
    auto pair_of_steps = [&](auto pair, uint32_t carry, uint32_t after_stores) {
        each<PHASES - 1>([&](auto f) { phase(pair, f, carry); });
        // still running at most: the loads of the pairs behind the next one, one group's scale bytes among them
        constexpr int kAllow = (PAIRS - 2) * L + (PAIRS > 2 ? SC : 0);
        constexpr int kLate = kAllow + kStores < 63 ? kAllow + kStores : 63;  // the counter's end
        if (after_stores) wait_vm_and_lds_then_barrier<kLate>();
        else wait_vm_and_lds_then_barrier<kAllow>();
        if constexpr (pair == 0) {
            advance();
            fetch_scales(next, free_sslot());
        }
        phase(pair, std::integral_constant<int, PHASES - 1>{}, 0);
    };
    for (; t < items; t += gridDim.x) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        int64_t cm0, cn0;
        place(t % tiles, cm0, cn0);
        T* const yc = y + t / tiles * part;
        const uint32_t g0 = t / tiles * per_split, g1 = g0 + per_split < groups ? g0 + per_split : groups;
#pragma nounroll
        for (g = g0; g < g1; ++g) {
            uint32_t carry = __builtin_amdgcn_readfirstlane(g != g0 ? 1 : 0);
            uint32_t after_stores = __builtin_amdgcn_readfirstlane(g == g0 && t != first ? 1 : 0);
            asm volatile("" : "+s"(after_stores), "+s"(carry));  // the loop stays one loop
            pair_of_steps(zero{}, carry, after_stores);
            pair_of_steps(one{}, 1, PAIRS > 2 ? after_stores : 0u);
            set = next_set();
            sslot = next_sslot();
        }
        if constexpr (PAIRS == 2) each<L / 2>([&](auto i) { fetch_part(next, 0, one{}, std::integral_constant<int, i + L / 2>{}); });
        // Out through LDS of this wavefront's own, 32 rows of PIECE bytes at a
        // time, so that each store writes long runs of a row: chunk c of row r
        // lies at position c ^ (r % chunks).
        const bool whole = cm0 + BM <= m && cn0 + BN <= n;
        uint8_t* out = lds + PAIRS * kSlotBytes + (SETS + 1) * kScaleBytes + wave * 32 * PIECE;
        constexpr int kChunks = PIECE / 16, kPer = 16 / sizeof(T);  // chunks of a row, elements of a chunk
        constexpr int kBlocks = PIECE / (int)sizeof(T) / 16;        // blocks of 16 columns of a piece
#pragma unroll
        for (int j = 0; j < FM; ++j) {
#pragma unroll
            for (int pc = 0; pc < 2 * FN / kBlocks; ++pc) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const f32x16& v = acc[(pc * kBlocks + b) / 2][j];
                    const int e = (pc * kBlocks + b) % 2 * 8;
                    auto put = [&](int c, const u32x4& w) {
                        *reinterpret_cast<u32x4*>(out + l32 * PIECE + ((c ^ (l32 & (kChunks - 1))) * 16)) = w;
                    };
                    if constexpr (sizeof(T) == 4) {
                        put(4 * b + half, u32x4{float_bits(v[e]), float_bits(v[e + 1]), float_bits(v[e + 2]), float_bits(v[e + 3])});
                        put(4 * b + 2 + half,
                            u32x4{float_bits(v[e + 4]), float_bits(v[e + 5]), float_bits(v[e + 6]), float_bits(v[e + 7])});
                    } else {
                        // lanes l and l + 32 exchange so that each holds 8 consecutive columns
                        const u32x2 w0 = __builtin_amdgcn_permlane32_swap(bf16_pair(v[e], v[e + 1]),
                                                                          bf16_pair(v[e + 4], v[e + 5]), false, false);
                        const u32x2 w1 = __builtin_amdgcn_permlane32_swap(bf16_pair(v[e + 2], v[e + 3]),
                                                                          bf16_pair(v[e + 6], v[e + 7]), false, false);
                        put(2 * b + half, u32x4{w0[0], w1[0], w0[1], w1[1]});
                    }
                }
                const int lr = lane / kChunks, lc = lane % kChunks;
                const int64_t row0 = cm0 + wm + j * 32, col0 = cn0 + wn + pc * kBlocks * 16;
                auto store_rows = [&](auto past) {
                    T* to = yc + (row0 + lr) * ld + col0 + lc * kPer;
#pragma unroll
                    for (int r = 0; r < 32; r += kWave / kChunks) {
                        const u32x4 w = *reinterpret_cast<const u32x4*>(out + (r + lr) * PIECE + ((lc ^ (lr & (kChunks - 1))) * 16));
                        store_chunk<past.value>(to + r * ld, w);
                    }
                };
                if (whole && lines) {
                    asm volatile("; whole lines" ::: "memory");  // around the branch, which otherwise becomes
                    store_rows(std::bool_constant<(FN * FM > 4)>{});
                    asm volatile("; of y" ::: "memory");  // one with the next, and its stores plain ones
                } else if (whole) {
                    store_rows(std::false_type{});
                } else {  // what exists of each chunk
                    const int64_t left = n - (col0 + lc * kPer);
#pragma nounroll
                    for (int r = lr; r < 32 && row0 + r < m; r += kWave / kChunks) {
                        const uint8_t* from = out + r * PIECE + ((lc ^ (r & (kChunks - 1))) * 16);
                        T* to = yc + (row0 + r) * ld + col0 + lc * kPer;
                        if (left >= kPer) {
                            store_chunk<false>(to, *reinterpret_cast<const u32x4*>(from));
                        } else {
#pragma nounroll
                            for (int e = 0; e < (int)left; ++e) gp(to)[e] = reinterpret_cast<const T*>(from)[e];
                        }
                    }
                }
            }
        }
        if (!whole) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    // nothing may still be on its way into LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Adds the partial sums of the splits, in their order: four columns a thread.
template <class T>
__global__ __launch_bounds__(kBlock) void mx4_matmul_join_kernel(const float* __restrict__ ws, int64_t part, int64_t lw,
                                                                 uint32_t splits, int64_t m, int64_t n,
                                                                 T* __restrict__ y, int64_t ld) {
    const int64_t quads = lw / 4, total = m * quads;
    for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < total; i += (int64_t)gridDim.x * kBlock) {
        const int64_t row = i / quads, col = (i - row * quads) * 4;
        const float* p = ws + row * lw + col;
        f32x4 sum = *reinterpret_cast<const gf32x4*>(gp(p));
        for (uint32_t s = 1; s < splits; ++s) {
            const f32x4 v = *reinterpret_cast<const gf32x4*>(gp(p + s * part));
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += v[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (col + j >= n) break;
            if constexpr (sizeof(T) == 4) gp(y)[row * ld + col + j] = sum[j];
            else gp(y)[row * ld + col + j] = (uint16_t)bf16_bits(sum[j]);
        }
    }
}

// ------------------------------------------------------------------ few rows of A
//
// Bound by reading B once, and by its launch where B is small: 1 x 13824 x 5120 (38
// MB) takes 9.0 us, 4.2 TB/s. A workgroup takes 16 rows of B; its wavefronts take a
// part of k each, straight from global memory into registers, and add their
// sums through LDS in order. Up to 16 FM rows of A; rows past the end are read
// as the last one and not stored.
//
// The matrix instruction here takes 16 rows of each operand over 128 values of
// k: lane l holds the 32 codes of row l % 16 in block l / 16, and their scale
// byte; accumulator r of lane l is y[l % 16][4 (l / 16) + r]. A load covers 64
// consecutive bytes of each row (a 32-row form of the instruction would make it
// 32), and a row's scale bytes of four steps come in one.
constexpr int kFewWaves = 8;
// Groups of four steps in a turn of the loop. The compiler deals a turn's loads out
// between its matrix instructions (59 registers, where all of them at once would take
// over 80), so that the loads of one or two steps are in flight at a time.
constexpr int kFewAhead = 2;

template <int FM, class T>
__global__ __launch_bounds__(kFewWaves* kWave) void mx4_matmul_few_kernel(const uint8_t* __restrict__ aq,
                                                                         const uint8_t* __restrict__ as, int64_t m,
                                                                         const uint8_t* __restrict__ bq,
                                                                         const uint8_t* __restrict__ bs, int64_t n,
                                                                         int64_t k, int per, T* __restrict__ y, int64_t ld) {
    __shared__ float sums[kFewWaves][4 * FM][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int block = lane >> 4, l16 = lane & 15;
    const int64_t n0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 16;
    if (n0 >= n) return;
    const int64_t qb = mx4_code_bytes(k), sb = mx4_scale_bytes(k);
    const int steps = (int)(qb / 64), groups = (steps + 3) / 4;  // groups of four steps
    const int g0 = wave * per, g1 = g0 + per < groups ? g0 + per : groups;
    const int64_t rb = n0 + l16 < n ? n0 + l16 : n - 1;
    const uint8_t *pb = bq + rb * qb + block * 16, *psb = bs + rb * sb;
    const uint8_t *pa[FM], *psa[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t ra = j * 16 + l16 < m ? j * 16 + l16 : m - 1;
        pa[j] = aq + ra * qb + block * 16;
        psa[j] = as + ra * sb;
    }
    f32x4 acc[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = g0; g < g1; g += kFewAhead) {
        u32x4 b[kFewAhead][4], a[kFewAhead][FM][4], cb[kFewAhead], ca[kFewAhead][FM];
#pragma unroll
        for (int v = 0; v < kFewAhead; ++v) {
            const int gv = g + v < g1 ? g + v : g1 - 1;
            cb[v] = *reinterpret_cast<const gu32x4*>(gp(psb) + gv * 16);
#pragma unroll
            for (int j = 0; j < FM; ++j) ca[v][j] = *reinterpret_cast<const gu32x4*>(gp(psa[j]) + gv * 16);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = 4 * gv + u < steps ? 4 * gv + u : steps - 1;
                b[v][u] = *reinterpret_cast<const gu32x4*>(gp(pb) + at * 64);
#pragma unroll
                for (int j = 0; j < FM; ++j) a[v][j][u] = *reinterpret_cast<const gu32x4*>(gp(pa[j]) + at * 64);
            }
        }
#pragma unroll
        for (int v = 0; v < kFewAhead; ++v)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // a step past this wavefront's part gets scale bytes 0, and adds nothing
                const uint32_t width = g + v < g1 && 4 * (g + v) + u < steps ? 8u : 0u;
                const uint32_t sbw = __builtin_amdgcn_ubfe(cb[v][u], 8 * block, width);
                const i32x8 vb{(int)b[v][u].x, (int)b[v][u].y, (int)b[v][u].z, (int)b[v][u].w, 0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const uint32_t sa = __builtin_amdgcn_ubfe(ca[v][j][u], 8 * block, width);
                    const u32x4 w = a[v][j][u];
                    const i32x8 va{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
                    acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[j], 4, 4, 0, (int)sbw, 0, (int)sa);
                }
            }
    }
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) sums[wave][j * 4 + r][lane] = acc[j][r];
    __syncthreads();
    const int rows = (int)(m < 16 * FM ? m : 16 * FM), waves = blockDim.x / kWave;
    for (int i = threadIdx.x; i < rows * 16; i += blockDim.x) {
        const int row = i / 16, col = i % 16;
        const int r = row / 16 * 4 + col % 4, at = col / 4 * 16 + row % 16;
        float sum = sums[0][r][at];
        for (int w = 1; w < waves; ++w) sum += sums[w][r][at];
        if (n0 + col < n) {
            if constexpr (sizeof(T) == 4) gp(y)[row * ld + n0 + col] = sum;
            else gp(y)[row * ld + n0 + col] = (uint16_t)bf16_bits(sum);
        }
    }
}

template <int FM, class T>
int launch_few(const uint8_t* aq, const uint8_t* as, int64_t m, const uint8_t* bq, const uint8_t* bs, int64_t n, int64_t k,
               T* y, int64_t ld, hipStream_t st) {
    // whole turns of the loop: 1 x 32000 x 4096 (8 groups) takes 14 us with 4
    // wavefronts of two groups and 25 with 8 of one
    const int64_t groups = div_up(k, 512), per = div_up(groups, kFewWaves * kFewAhead) * kFewAhead;
    const unsigned threads = (unsigned)div_up(groups, per) * kWave;
    const Grid g = grid_xy(div_up(n, 16), threads);
    hipLaunchKernelGGL((mx4_matmul_few_kernel<FM, T>), dim3(g.x, g.y), dim3(threads), 0, st, aq, as, m, bq, bs, n, k, (int)per, y,
                       ld);
    return launch_status();
}

template <class T>
int launch_matmul(const uint8_t* aq, const uint8_t* as, int64_t m, const uint8_t* bq, const uint8_t* bs, int64_t n,
                  int64_t k, T* y, int64_t ld, float* ws, hipStream_t st) {
    const Product p = product_of(m, n, k);
    if (p.way == Way::kFew) {
        return m <= 16 ? launch_few<1>(aq, as, m, bq, bs, n, k, y, ld, st) : launch_few<2>(aq, as, m, bq, bs, n, k, y, ld, st);
    }
    if (p.way == Way::kSmall) {
        const int64_t tn = div_up(n, 64), tiles = tn * div_up(m, 64);
        if (tiles > 0x7FFFFFFFll) return COAT_EINVAL;
        const Grid g = grid_xy(tiles, kBlock);
        hipLaunchKernelGGL(mx4_matmul_small_kernel<T>, dim3(g.x, g.y), dim3(kBlock), 0, st, aq, as, m, bq, bs, n, k, (uint32_t)tn,
                           y, ld);
        return launch_status();
    }
    auto grid_of = [](int64_t items) { return dim3((unsigned)(items < kCUs ? items : kCUs)); };
    auto small_tiles = [&](int64_t m0, int64_t n0) {  // rows of y from m0 and columns from n0
        const int64_t tm = div_up(m - m0, 128), tn = div_up(n - n0, 128), qb = mx4_code_bytes(k), sb = mx4_scale_bytes(k);
        hipLaunchKernelGGL((mx4_matmul_tile_kernel<2, 2, 2, 2, 4, 128, T>), grid_of(tm * tn), dim3(kBlock), 0, st, aq + m0 * qb,
                           as + m0 * sb, m - m0, bq + n0 * qb, bs + n0 * sb, n - n0, k, (uint32_t)tm, (uint32_t)tn, 1u,
                           p.per_split, y + m0 * ld + n0, ld, (int64_t)0);
    };
    if (p.way == Way::kTile256) {
        const int64_t tm = div_up(p.head_m, 256), tn = div_up(p.head_n, 256);
        hipLaunchKernelGGL((mx4_matmul_tile_kernel<2, 2, 4, 4, 2, 128, T>), grid_of(tm * tn), dim3(kBlock), 0, st, aq, as,
                           p.head_m, bq, bs, p.head_n, k, (uint32_t)tm, (uint32_t)tn, 1u, p.per_split, y, ld, (int64_t)0);
        if (p.head_m < m) small_tiles(p.head_m, 0);
        else if (p.head_n < n) small_tiles(0, p.head_n);
        return launch_status();
    }
    if (p.splits == 1) {
        small_tiles(0, 0);
        return launch_status();
    }
    const dim3 grid = grid_of((int64_t)p.tiles_m * p.tiles_n * p.splits);
    // Bound by latency (LDS reads active in 0.46 of the cycles, matrix units in 0.28,
    // wavefronts waiting in 0.35): eight wavefronts of 32 x 64 read half as much again from
    // LDS as four of 64 x 64, but hide more of it. One round of split tiles gains (64 x
    // 5120 x 13824 22 -> 20 us, 700 x 1000 x 8192 23 -> 20), whole ones lose (1500 x
    // 5120 x 13824 79 -> 86).
    hipLaunchKernelGGL((mx4_matmul_tile_kernel<4, 2, 1, 2, 4, 64, float>), grid, dim3(2 * kBlock), 0, st, aq, as, m, bq, bs, n,
                       k, p.tiles_m, p.tiles_n, p.splits, p.per_split, ws, p.lw, p.part);
    hipLaunchKernelGGL(mx4_matmul_join_kernel<T>, dim3((unsigned)(div_up(m * p.lw / 4, kBlock) < 8 * kCUs ? div_up(m * p.lw / 4, kBlock) : 8 * kCUs)),
                       dim3(kBlock), 0, st, (const float*)ws, p.part, p.lw, p.splits, m, n, y, ld);
    return launch_status();
}

}  // namespace

extern "C" {

size_t coat_mx4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) { return product_workspace_bytes(m, n, k); }

int coat_mx4_matmul(const uint8_t* a_q, const uint8_t* a_s, int64_t m, const uint8_t* b_q, const uint8_t* b_s,
                    int64_t n, int64_t k, void* y, int64_t ld, int32_t dtype, void* workspace, size_t workspace_bytes,
                    coat_stream_t stream) {
    const int rc = check_mx4_matmul(a_q, a_s, m, b_q, b_s, n, k, y, ld, dtype);
    if (rc || m == 0 || n == 0) return rc;
    const size_t need = product_workspace_bytes(m, n, k);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return COAT_EINVAL;
        if (!aligned(workspace, 256)) return COAT_EALIGN;
    }
    float* ws = static_cast<float*>(workspace);
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (dtype == COAT_FP32)
        return launch_matmul(a_q, a_s, m, b_q, b_s, n, k, static_cast<float*>(y), ld, ws, st);
    return launch_matmul(a_q, a_s, m, b_q, b_s, n, k, static_cast<uint16_t*>(y), ld, ws, st);
}

}  // extern "C"

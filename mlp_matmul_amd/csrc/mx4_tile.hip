// Many rows per expert (or a large batch) against 4-bit weights: the matrix
// units bound the product.
//
// A workgroup multiplies MT weight rows (of the pair: MT/2 of each matrix) with NT
// input rows in steps of 128 columns (bf16 rows) or 256 (4-bit rows): 64 or 128
// bytes of a weight row, 256 or 128 of an input row.
//   bf16 rows: the codes become bf16 with their block's scale in one instruction
//   for two of them, exactly, and go to the 16x16x32 bf16 MFMA; a lane's half block
//   of codes is its 16 columns of two of those.
//   4-bit rows: codes and scales go to the scaled 16x16x128 MFMA as they are, a
//   block a lane; the instruction takes the scale's byte for the half of the step.
// Sums in fp32.  LDS is filled from memory directly, S buffers deep, chunks of 16
// bytes exchanged within a row so that the fragments' reads meet no bank twice;
// a load to LDS costs by the 128-byte lines that it touches (17.5 cycles a KB for
// whole lines, 32 for half ones, 88 for 16 bytes a row), so the scales come for 512
// columns at a time, 16 bytes of a row.  Eight bands of weight rows are walked
// together, so that the workgroups of an XCD share both operands (3-10 %).
//
// Measured on MI355X, 8192 x 8192 weights and as many rows, us by tile:
//   bf16 rows:   64x64 1270,  128x64 1064,  256x128 842 (1.31 PFLOP/s)
//   4-bit rows:  64x64 536,   128x128 356,  256x256 287 (3.8 PFLOP/s)
// (the matrix units alone, from registers: 1.9 and 7.2 PFLOP/s).  Small ones for few
// rows: 777 rows of 14336 x 4096 in bf16 take 125, 106 and 108; pairs of 32 experts of
// 1024 x 2048 with 75 rows on average 47, 39 and 62, some with more than 128 (with
// 75 each 52, 41 and 36).
// Of the 256x256 tile's 726 thousand cycles the matrix units work 262, the LDS 213
// on fragments and 65 on what arrives, and its loads take 143 to issue: two
// waves a SIMD between barriers hide only part of these behind each other.  Without
// the loads of its loop it takes 237 us, not 295 (bf16 rows: 736, not 850).  Four
// waves of 128x128 each, with twice the registers, take 345 us; reading a step or
// more ahead into L2, loads spread among the products and priorities of waves
// change nothing.  A tile's first loads and its epilogue overlap no other tile's work:
// with one workgroup a compute unit they cost eight steps (mx4_matmul.hip), a third
// of the time at 4096 columns.
#include <type_traits>

#include "kernels.h"
#include "mx4_common.h"

namespace uwk {

namespace {

// How rows of RB bytes lie in LDS: 16-byte chunk c of row r at position c ^ swizzle(r), so that 16 rows' chunks of one
// column meet no bank twice (256 bytes of banks).
template <int RB>
__device__ __forceinline__ uint32_t swizzle(uint32_t r) {
    return RB == 64 ? (r >> 2) & 3u : RB == 128 ? (r & 7u) ^ ((r >> 3) & 1u) : r & 15u;
}

template <bool X4, bool PAIR, bool TAIL, int MT, int NT, int WM, int WN, int S, int G>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_tile_kernel(Mx4Args a, uint32_t bands) {
    constexpr int NW = WM * WN;
    constexpr int FM = MT / 16 / WM, FN = NT / 16 / WN;  // 16-row blocks of a wave's output
    constexpr int KB = X4 ? 8 : 4;                       // blocks of 32 columns of a step
    constexpr int WB = KB * 16, XB = X4 ? WB : KB * 64;  // bytes of a row of W and X
    constexpr int WC = WB / 16, XC = XB / 16;            // their chunks
    constexpr int WD = MT * WC / 64 / NW, XD = NT * XC / 64 / NW;   // loads of a wave and step
    constexpr int SR = MT + (X4 ? NT : 0);               // rows with scales
    constexpr int SS = 16 / KB;                          // steps whose scales are loaded together: 16 bytes of a row, a lane
    constexpr int SL = SR / 64;                          // those loads
    constexpr int SD = (SL + NW - 1) / NW;
    constexpr int U = S == 2 ? 2 : 3 * SS;               // steps after which all buffers come round
    constexpr int XG = XD / G;                           // loads of the rows of one of the G parts of X
    constexpr int kLoads = WD + XD, kMain = WD + XG;
    constexpr int kRows = PAIR ? MT / 2 : MT;            // rows of a matrix in a tile
    static_assert(WD * NW * 64 == MT * WC && XG * G * NW * 64 == NT * XC && SL * 64 == SR && (S == 2 || S == 3), "whole loads");
    static_assert(G == 1 || (G == 2 && S == 2), "the loads that a step waits for");
    constexpr int kX = MT * WB, kPart = NT / G * XB, kBuf = kX + kPart;
    __shared__ __align__(16) uint8_t buf0[kBuf], buf1[kBuf], buf2[S > 2 ? kBuf : 16];
    __shared__ __align__(16) uint8_t rest0[G > 1 ? kPart : 16], rest1[G > 1 ? kPart : 16];   // X's second part
    // Two buffers of scales in one array where the waits drain all loads to LDS anyway (behind them room for loads that
    // nobody reads), else three of their own: a read waits for the loads to its array.
    constexpr int kScales = SR * 16;
    __shared__ __align__(16) uint8_t scale0[S == 2 ? 2 * kScales + 1024 : kScales], scale1[S == 2 ? 16 : kScales],
        scale2[S == 2 ? 16 : kScales];
    constexpr int ES = kRows + 4;
    static_assert(16 * WN * ES * 4 <= kBuf, "a part of the outputs fits a buffer");
    static_assert((S - 1) * kLoads < 64, "loads in flight");

    GroupTile t;
    if (!group_tile<NT, 8>(a.g, bands, t)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const uint32_t R = uint32_t(a.g.R), blocks = uint32_t(a.g.C) / kMx4Block;
    const uint32_t row0 = uint32_t(t.band) * kRows;
    const uint32_t steps = blocks / KB;                  // whole ones; with TAIL the rest follows alone
    const int64_t first = int64_t(t.e) * R;

    // sources: the lane's chunk of its row in load j, as bytes from the row's start
    const uint8_t* wb[PAIR ? 2 : 1];
    uint32_t woff[WD];
    const uint8_t* xp[XD];
#pragma unroll
    for (int m = 0; m < (PAIR ? 2 : 1); ++m) wb[m] = a.w[m].codes + first * a.w[m].ldc;
    auto matrix = [&](int j) { return PAIR ? (wave * WD + j) * (64 / WC) / kRows : 0; };    // uniform
    auto w_chunk = [&](int j) { return (lane % WC) ^ swizzle<WB>(uint32_t(wave * WD + j) * (64 / WC) + lane / WC); };
    auto x_row = [&](int j) { return uint32_t(wave * XG + j % XG) * (64 / XC) + lane / XC; };   // in its part
    auto x_chunk = [&](int j) { return (lane % XC) ^ swizzle<XB>(x_row(j)); };
#pragma unroll
    for (int j = 0; j < WD; ++j) {
        const uint32_t r = uint32_t(wave * WD + j) * (64 / WC) + lane / WC;
        woff[j] = min(row0 + r % uint32_t(kRows), R - 1u) * uint32_t(a.w[matrix(j)].ldc) + w_chunk(j) * 16u;
    }
#pragma unroll
    for (int j = 0; j < XD; ++j) {
        const uint32_t r = uint32_t(j / XG) * (NT / G) + x_row(j);
        const int64_t x = group_x_index(a.g, t.row0 + min(r, uint32_t(t.rows) - 1u));
        xp[j] = (X4 ? a.x.codes + x * a.x.ldc : reinterpret_cast<const uint8_t*>(a.g.X + x * a.g.ldx)) + x_chunk(j) * 16u;
    }
    // scales: a row a lane, 64 rows a load
    const uint8_t* sp[SD];
#pragma unroll
    for (int j = 0; j < SD; ++j) {
        const uint32_t r = uint32_t(min(wave + j * NW, SL - 1)) * 64u + lane;
        if (r < uint32_t(MT)) {
            const Mx4Mat& w = a.w[PAIR && r >= uint32_t(kRows) ? 1 : 0];
            sp[j] = w.scales + (first + min(row0 + r % uint32_t(kRows), R - 1u)) * w.lds;
        } else {
            sp[j] = a.x.scales + group_x_index(a.g, t.row0 + min(r - MT, uint32_t(t.rows) - 1u)) * a.x.lds;
        }
    }
    auto buffer = [&](int i) -> uint8_t* { return i == 0 ? buf0 : i == 1 ? buf1 : buf2; };
    // The scales of steps SS u .. SS u + SS - 1 (past the end: the last ones again); i: the first of them, modulo U.
    auto scales_of = [&](int i) -> uint8_t* { return S == 2 || i / SS == 0 ? scale0 : i / SS == 1 ? scale1 : scale2; };
    auto load_scales = [&](uint32_t u, int i, bool now) {
        const uint64_t o = 16u * min(u, (blocks - 1u) / 16u);
#pragma unroll
        for (int j = 0; j < SD; ++j) {
            const bool mine = now && wave + j * NW < SL;
            if (S == 2) {
                // waves without a part in them, and steps that are not their turn, load one line to a place that nobody
                // reads: a branch in every step would cost the loop registers
                uint32_t to = mine ? (u & 1u) * kScales + uint32_t(wave + j * NW) * 1024u : 2u * kScales;
                asm("" : "+s"(to));                      // (as in read_scales)
                dma16(mine ? sp[j] + o : a.w[0].scales, scales_of(i) + to);
            } else if (mine) {
                dma16(sp[j] + o, scales_of(i) + (wave + j * NW) * 1024);
            }
        }
    };
    auto rest = [&](int i) -> uint8_t* { return i == 0 ? rest0 : rest1; };
    // steps past the end load the last one again: the waits count the same loads in every step
    // loads j0 .. j1 - 1: W's, those of X's first part, of its second
    auto load = [&](uint32_t s, int i, int j0, int j1) {
        uint8_t* const b = buffer(i);
        s = min(s, steps - 1u);
#pragma unroll
        for (int j = j0; j < j1; ++j) {
            if (j < WD) dma16(wb[matrix(j)] + uint64_t(s) * WB + woff[j < WD ? j : 0], b + (wave * WD + j) * 1024);
            else dma16(xp[j < WD ? 0 : j - WD] + uint64_t(s) * XB, (j < kMain ? b + kX : rest(i)) + (wave * XG + (j - WD) % XG) * 1024);
        }
    };

    // fragments of half h of a step: 4-bit rows' 8 blocks, lane q's block 2q + h; bf16 rows' half h of each of 4 blocks,
    // lane q's block q, and the weights' codes of that half.  The scales of both halves come with one read.
    const int wm = wave / WN, wn = wave % WN;
    constexpr int P = 2 * G, FG = FN / G, BK = X4 ? 1 : 2;
    struct FragsA {
        u32x4_t A[X4 ? FM : 1];
        u32x2_t a[X4 ? 1 : FM];
    };
    struct FragsB {
        u32x4_t B[FG][BK];
    };
    // 4-bit rows: two 16-row blocks' in a register, two bytes each (one in each, the 256x256 tile with columns behind the
    // last step would spill 62 registers, not 34: 14336 x 4000 with 4096 rows 199 us, not 182)
    struct Scales {
        uint32_t a[X4 ? FM / 2 : FM], b[X4 ? FN / 2 : 1];
    };
    auto a_block = [&](int i) { return PAIR ? (i < FM / 2 ? wm * FM / 2 + i : MT / 32 + wm * FM / 2 + i - FM / 2) : wm * FM + i; };
    // One variable index and one constant each: behind a longer chain of sums the compiler no longer knows the array,
    // and waits for every load to LDS.
    uint32_t ia[2], ib[2][BK];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        ia[h] = (uint32_t(a_block(0)) * 16u + rl) * WB + ((X4 ? 2u * q + uint32_t(h) : q) ^ swizzle<WB>(rl)) * 16u;
#pragma unroll
        for (int k = 0; k < BK; ++k)
            ib[h][k] = (uint32_t(wn * FG) * 16u + rl) * XB + ((X4 ? 2u * q + uint32_t(h) : 4u * q + uint32_t(2 * h + k)) ^ swizzle<XB>(rl)) * 16u;
    }
    auto read_a = [&](const uint8_t* b, int h, FragsA& f) {
        const uint8_t* const p = b + ia[h];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int o = (PAIR && i >= FM / 2 ? MT / 32 + i - FM / 2 : i) * 16 * WB;
            if (X4) f.A[i] = *reinterpret_cast<const u32x4_t*>(p + o);
            else f.a[i] = *reinterpret_cast<const u32x2_t*>(p + (o + 8 * h));
        }
    };
    auto read_b = [&](const uint8_t* b, int h, FragsB& f) {
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const uint8_t* const p = b + ib[h][k];
#pragma unroll
            for (int i = 0; i < FG; ++i) f.B[i][k] = *reinterpret_cast<const u32x4_t*>(p + i * 16 * XB);
        }
    };
    // of step s
    const uint32_t so = rl * 16u + (X4 ? 2u * q : q);
    auto read_scales = [&](uint32_t s, int i, Scales& f) {
        // indexes that the compiler can't take apart, as those of the fragments
        const uint32_t o = so + (S == 2 ? (s / SS & 1u) * kScales + s % SS * KB : uint32_t(i % SS * KB));
        uint32_t a0 = o + uint32_t(wm * (PAIR ? FM / 2 : FM)) * 256u, b0 = o + uint32_t(MT / 16 + wn * FG) * 256u;
        asm("" : "+v"(a0));
        if (X4) asm("" : "+v"(b0));
        const uint8_t* const b = scales_of(i);
        auto at_a = [&](int k) { return b + a0 + (PAIR && k >= FM / 2 ? MT / 32 + k - FM / 2 : k) * 256; };
        auto at_b = [&](int k) { return b + b0 + (k / FG * (NT / 16 / G) + k % FG) * 256; };
        auto two = [](const uint8_t* p, const uint8_t* q) {
            const s16x2_t v{*reinterpret_cast<const int16_t*>(p), *reinterpret_cast<const int16_t*>(q)};
            return __builtin_bit_cast(uint32_t, v);
        };
        if constexpr (X4) {
#pragma unroll
            for (int k = 0; k < FM / 2; ++k) f.a[k] = two(at_a(2 * k), at_a(2 * k + 1));
#pragma unroll
            for (int k = 0; k < FN / 2; ++k) f.b[k] = two(at_b(2 * k), at_b(2 * k + 1));
        } else {
#pragma unroll
            for (int k = 0; k < FM; ++k) f.a[k] = *at_a(k);
        }
    };
    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](auto h, int g, const FragsA& fa, const FragsB& fb, const Scales& sc, auto behind) {
        constexpr int H = decltype(h)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if constexpr (X4) {
#pragma unroll
                for (int j = 0; j < FG; ++j) {
                    const uint32_t sa = sc.a[i / 2], sb = sc.b[(g * FG + j) / 2];
                    f32x4_t& d = acc[i][g * FG + j];
                    if (i % 2) d = j % 2 ? mfma_mx4<2 + H, 2 + H>(fa.A[i], sa, fb.B[j][0], sb, d) : mfma_mx4<2 + H, H>(fa.A[i], sa, fb.B[j][0], sb, d);
                    else d = j % 2 ? mfma_mx4<H, 2 + H>(fa.A[i], sa, fb.B[j][0], sb, d) : mfma_mx4<H, H>(fa.A[i], sa, fb.B[j][0], sb, d);
                }
            } else {
#pragma unroll
                for (int k = 0; k < BK; ++k) {
                    const bf16x8_t w = mx4_to_bf16(fa.a[i][k], sc.a[i]);
#pragma unroll
                    for (int j = 0; j < FG; ++j)
                        acc[i][g * FG + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, fb.B[j][k]), acc[i][g * FG + j], 0, 0, 0);
                }
            }
            behind(i);
        }
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;

    // Step s, i modulo U, in P phases of one part of the input rows and one half of
    // the columns: each reads the next one's fragments.  After the first one a
    // step's buffer is free but for X's second part, which is free before the last
    // one; then come the barriers and the loads S steps ahead.  The scales of a step
    // are read in the one before it, so that their buffer is free in the last of
    // its steps.
    FragsA fa[2];
    FragsB fb[2];
    Scales sc;
    auto read_phase = [&](int i, int p) {
        if (p < 2) read_a(buffer(i), p, fa[p]);
        read_b(p < 2 ? buffer(i) + kX : rest(i), p % 2, fb[p % 2]);
    };
    auto mma_phase = [&](int p, auto behind) {
        if (p % 2) mma(H1{}, p / 2, fa[1], fb[1], sc, behind);
        else mma(H0{}, p / 2, fa[0], fb[0], sc, behind);
    };
    auto step = [&](uint32_t s, int i) {
#pragma unroll
        for (int p = 0; p + 1 < P; ++p) {
            read_phase(i % S, p + 1);
            mma_phase(p, [](int) {});
            __builtin_amdgcn_sched_barrier(0);
            if (G > 1 && p == 0) {
                wait_vm<63, true>();                     // this wave's fragments are here
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                load(s + S, i % S, 0, kMain);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // the next step's loads and this step's fragments are here
        wait_vm<(G > 1 ? kMain : (S - 2) * kLoads), true>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        Scales next;
        read_scales(s + 1, (i + 1) % U, next);
        __builtin_amdgcn_sched_barrier(0);
        if (S == 2) load_scales(s / SS + 2, 0, s % SS == SS - 1);
        else if (i % SS == SS - 1) load_scales(s / SS + 3, i, true);   // before the columns': the waits count those alone
        if (G > 1) load(s + S, i % S, kMain, kLoads);
        __builtin_amdgcn_sched_barrier(0);
        read_phase((i + 1) % S, 0);
        if (G > 1) {
            mma_phase(P - 1, [](int) {});
        } else {
            // the loads among the products (2 % faster than before them; with two parts 2 % slower)
            __builtin_amdgcn_sched_barrier(0);
            mma_phase(P - 1, [&](int k) {
                __builtin_amdgcn_sched_barrier(0);
                load(s + S, i % S, kLoads * k / FM, kLoads * (k + 1) / FM);
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        sc = next;
        __builtin_amdgcn_sched_barrier(0);
    };
    if (!TAIL || steps) {
        load_scales(0, 0, true);
        load_scales(1, SS, true);
        if (S == 3) load_scales(2, 2 * SS, true);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < S; ++i) {
            load(uint32_t(i), i, 0, kLoads);
            __builtin_amdgcn_sched_barrier(0);           // in this order: the waits count them
        }
        wait_vm<(S - 1) * kLoads, true>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read_scales(0, 0, sc);
        read_phase(0, 0);
        uint32_t s = 0;
        for (; s + U <= steps; s += U) {
#pragma unroll
            for (int i = 0; i < U; ++i) step(s + uint32_t(i), i);
        }
#pragma unroll
        for (int i = 0; i < U - 1; ++i)
            if (s + uint32_t(i) < steps) step(s + uint32_t(i), i);
        __builtin_amdgcn_s_waitcnt(0);                   // no load is on its way to LDS that is used again
        if (TAIL) __syncthreads();
    }
    if constexpr (TAIL) {
        // blocks behind the last whole step: lanes of those that are not there multiply zeros
        const uint32_t left = blocks % KB;
#pragma unroll
        for (int j = 0; j < WD; ++j) {
            const uint32_t c = w_chunk(j) < left ? 0u : w_chunk(j) * 16u;      // chunks behind the last read the first one
            dma16(wb[matrix(j)] + uint64_t(steps) * WB + woff[j] - c, buf0 + (wave * WD + j) * 1024);
        }
#pragma unroll
        for (int j = 0; j < XD; ++j) {
            const uint32_t c = x_chunk(j) < left * (XC / KB) ? 0u : x_chunk(j) * 16u;
            dma16(xp[j] + uint64_t(steps) * XB - c, (j < XG ? buf0 + kX : rest0) + (wave * XG + j % XG) * 1024);
        }
        load_scales(steps / SS, 0, true);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        read_scales(steps, int(steps % SS), sc);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            read_phase(0, p);
            const int h = p % 2;
            if ((X4 ? 2u * q + uint32_t(h) : q) >= left) {
                FragsA& f = fa[h];
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    if (X4) f.A[X4 ? i : 0] = u32x4_t{0u, 0u, 0u, 0u};
                    else f.a[X4 ? 0 : i] = u32x2_t{0u, 0u};
                }
                const uint32_t keep = X4 && h ? 0x00FF00FFu : 0u, one = (X4 ? 0x7F7F7F7Fu : 0x7Fu) & ~keep;
#pragma unroll
                for (int i = 0; i < (X4 ? FM / 2 : FM); ++i) sc.a[i] = (sc.a[i] & keep) | one;
#pragma unroll
                for (int i = 0; i < (X4 ? FN / 2 : 0); ++i) sc.b[i] = (sc.b[i] & keep) | one;
#pragma unroll
                for (int i = 0; i < (X4 ? 0 : FG); ++i)
#pragma unroll
                    for (int k = 0; k < BK; ++k) fb[p % 2].B[i][k] = u32x4_t{0u, 0u, 0u, 0u};
            }
            mma_phase(p, [](int) {});
        }
        __syncthreads();
    }

    // The epilogue in parts of a 16-row block of each wave column's inputs:
    // through LDS, so that a row of the output is written in one run and the
    // code is there once.  D layout: lane l holds input row l%16, weight rows
    // 4*(l/16)..+3 of a block.
    constexpr int OM = PAIR ? FM / 2 : FM;
    float* const part = reinterpret_cast<float*>(buf0);
    PartEpilogue<kRows, 16 * WN, 64 * NW, ES> out(a.g.ep, part, t, row0, a.g.R, tid);
    auto rows_of = [](int p) { return [p](int n) { return p / FG * (NT / G) + ((n / 16) * FG + p % FG) * 16 + n % 16; }; };
    out.load(rows_of(0));
#pragma unroll 1
    for (int p = 0; p < FN; ++p) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if (p != j) continue;
#pragma unroll
            for (int i = 0; i < OM; ++i) {
                f32x4_t v = acc[i][j];
                if (PAIR) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * acc[FM - OM + i][j][c];
                }
                *reinterpret_cast<f32x4_t*>(part + (wn * 16 + int(rl)) * ES + (wm * OM + i) * 16 + 4 * int(q)) = v;
            }
        }
        __syncthreads();
        out.store(rows_of(p), p + 1 < FN, rows_of(p + 1));
    }
}

template <bool X4, bool PAIR, int MT, int NT, int WM, int WN, int S, int G>
hipError_t launch(const Mx4Args& a, hipStream_t s) {
    const int64_t rows = PAIR ? MT / 2 : MT, bands = (a.g.R + rows - 1) / rows;
    const int64_t units = group_units(a.g, NT, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 grid{unsigned(units)}, block{64 * WM * WN};
    if (a.g.C % (X4 ? 256 : 128)) launch_timed(mx4_tile_kernel<X4, PAIR, true, MT, NT, WM, WN, S, G>, grid, block, 0, s, a, uint32_t(bands));
    else launch_timed(mx4_tile_kernel<X4, PAIR, false, MT, NT, WM, WN, S, G>, grid, block, 0, s, a, uint32_t(bands));
    return hipGetLastError();
}

template <bool X4, bool PAIR>
hipError_t launch_shape(const Mx4Args& a, Mx4TileShape shape, hipStream_t s) {
    switch (shape) {
        case MX4_TILE_SMALL: return launch<X4, PAIR, 64, 64, 2, 2, X4 ? 2 : 3, 1>(a, s);
        case MX4_TILE_MIDDLE:
            if constexpr (X4) return launch<X4, PAIR, 128, 128, 2, 2, 2, 1>(a, s);
            else return launch<X4, PAIR, 128, 64, 4, 2, 3, 1>(a, s);
        default:
            if constexpr (X4) return launch<X4, PAIR, 256, 256, 4, 2, 2, 2>(a, s);
            else return launch<X4, PAIR, 256, 128, 4, 2, 3, 1>(a, s);
    }
}

}  // namespace

hipError_t launch_mx4_tile(bool x4, bool pair, const Mx4Args& a, Mx4TileShape shape, hipStream_t s) {
    if (x4) return pair ? launch_shape<true, true>(a, shape, s) : launch_shape<true, false>(a, shape, s);
    return pair ? launch_shape<false, true>(a, shape, s) : launch_shape<false, false>(a, shape, s);
}

}  // namespace uwk

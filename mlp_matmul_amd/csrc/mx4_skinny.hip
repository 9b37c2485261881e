// Few rows per expert (or a small batch) against 4-bit weights: the product is
// bound by the weight stream, every weight is read once and used for up to NT
// input rows.
//
// A wave owns 16-row blocks of weights (the pair: the same rows of gate and up)
// and one K-slice, in steps of 128 columns.  Each step's operands go from memory
// to the wave's own LDS ring by global_load_lds, D steps in flight; the read-back
// in the MFMA operand layout is free of bank conflicts.  Scales come for 2048
// columns at a time, in one load a block.  Lane q of a row holds block q of the
// step: with bf16 rows its 32 weights become bf16 in registers, 8 an MFMA; with
// 4-bit rows they are multiplied as they are.  The KW waves of a workgroup split K
// and add their partial sums in wave order through LDS, then the epilogue
// runs on the sum: results do not depend on scheduling.
//
// Measured on MI355X, weights from memory: 16 rows with 4096 x 14336 12.6 us (32
// MB of weights; they alone take 6.6 at the rate of a copy, the rest is the
// start, two steps deep, the sums' end, and X: every workgroup brings all rows to
// LDS, four loads in five), one row with 1024 x 4096 4.2, pairs of 63 experts of
// 1408 x 2048 with one row each 43 (4.5 TB/s), with four 53 and with sixteen 65 on
// 16-row tiles, 47 and 110 on 4-row ones.
#include <algorithm>

#include "kernels.h"
#include "mx4_common.h"

namespace uwk {

namespace {

constexpr int kStepB = 4;            // blocks of 32 columns of a step
constexpr int kSegment = 16;         // steps whose scales are in LDS

// The place of 16-byte chunk c of row r of four chunks, so that 16 rows' chunks of one column meet no bank twice.
__device__ __forceinline__ uint32_t place4(uint32_t r, uint32_t c) { return r * 4u + (c ^ ((r >> 2) & 3u)); }

template <bool X4, bool PAIR, int NRB, int NT, int KW, int D>
__global__ __launch_bounds__(64 * KW) void mx4_skinny_kernel(Mx4Args a, uint32_t bands) {
    static_assert(!PAIR || NRB == 2, "the pair: one block of each matrix");
    constexpr int NB = (NT + 15) / 16;                   // 16-row tiles of the input rows
    constexpr int XL = X4 ? NB : NT / 4;                 // loads of their step
    constexpr int SB = NRB + (X4 ? NB : 0);              // 16-row blocks with scales
    constexpr int kX = NRB * 1024, kSlot = kX + XL * 1024;
    constexpr int kPer = NRB + XL;                       // loads of a step
    constexpr int TL = PAIR ? NB : NRB * NB;             // 16x16 tiles of outputs
    static_assert((D - 1) * kPer + SB < 64 && D >= 2 && D <= 4, "loads in flight");
    static_assert(NRB * NB * 1024 <= kSlot, "partial sums fit the first slots");
    // an array per slot: the compiler can tell them apart
    constexpr int kRing = KW * kSlot;
    static_assert(D == mx4_skinny_depth(NT, KW) && D * kRing + KW * SB * 1024 == mx4_skinny_lds(X4, PAIR, NT, KW) * 1024,
                  "what the choice of a kernel counts with");
    __shared__ __align__(16) uint8_t ring0[kRing], ring1[kRing], ring2[D > 2 ? kRing : 16], ring3[D > 3 ? kRing : 16];
    __shared__ __align__(16) uint8_t scale_buf[KW * SB * 1024];

    GroupTile t;
    if (!group_tile<NT>(a.g, bands, t)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const uint32_t R = uint32_t(a.g.R), blocks = uint32_t(a.g.C) / kMx4Block;
    constexpr uint32_t kRows = PAIR ? 16u : 16u * NRB;
    const uint32_t row0 = uint32_t(t.band) * kRows;
    const uint32_t steps = blocks / kStepB;              // whole ones; what is left goes to the last wave
    const uint32_t s_lo = steps * uint32_t(wave) / KW, s_hi = steps * uint32_t(wave + 1) / KW;

    const int64_t first = int64_t(t.e) * R;
    auto mat = [&](int r) -> const Mx4Mat& { return a.w[PAIR ? r : 0]; };
    // row i of block r; rows past the expert's read its last one and are not stored
    auto row_at = [&](int r, uint32_t i) -> uint32_t { return min(row0 + (PAIR ? 0u : 16u * uint32_t(r)) + i, R - 1u); };
    auto x_index = [&](uint32_t i) { return group_x_index(a.g, t.row0 + min(i, uint32_t(t.rows) - 1u)); };

    // a lane's chunk of a row is the one that lands where the lane's bytes do
    const uint32_t wr = lane >> 2, wc = (lane & 3u) ^ ((wr >> 2) & 3u);
    uint32_t woff[NRB];
#pragma unroll
    for (int r = 0; r < NRB; ++r) woff[r] = row_at(r, wr) * uint32_t(mat(r).ldc) + wc * 16u;
    const uint8_t* xp[XL];
    uint32_t xc[XL];
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const uint32_t i = X4 ? 16u * uint32_t(j) + wr : 4u * uint32_t(j) + q;
        xc[j] = X4 ? wc : rl ^ (i & 15u);
        xp[j] = (X4 ? a.x.codes + x_index(i) * a.x.ldc : reinterpret_cast<const uint8_t*>(a.g.X + x_index(i) * a.g.ldx)) + xc[j] * 16u;
    }
    // scales: lane l loads 16 bytes of row l % 16, unit l / 16 of the segment
    const uint8_t* sp[SB];
#pragma unroll
    for (int r = 0; r < SB; ++r)
        sp[r] = r < NRB ? mat(r).scales + (first + row_at(r, rl)) * mat(r).lds : a.x.scales + x_index(16u * uint32_t(r - NRB) + rl) * a.x.lds;
    const uint32_t last_unit = (blocks - 1u) / 16u;

    auto slot_base = [&](int i) -> uint8_t* { return i == 0 ? ring0 : i == 1 ? ring1 : i == 2 ? ring2 : ring3; };
    // (LDS is read at one index: behind a longer chain of sums the compiler waits for every load to LDS)
    const uint32_t mine = uint32_t(wave) * kSlot;
    auto load_scales = [&](uint32_t unit) {              // of 2048 columns
#pragma unroll
        for (int r = 0; r < SB; ++r) dma16(sp[r] + 16u * min(unit + q, last_unit), scale_buf + (wave * SB + r) * 1024);
        __builtin_amdgcn_sched_barrier(0);
    };
    const uint8_t* wb[PAIR ? 2 : 1];
#pragma unroll
    for (int r = 0; r < (PAIR ? 2 : 1); ++r) wb[r] = mat(r).codes + first * mat(r).ldc;
    auto issue = [&](uint32_t s, int slot) {
        uint8_t* const b = slot_base(slot);
#pragma unroll
        for (int r = 0; r < NRB; ++r) dma16(wb[PAIR ? r : 0] + uint64_t(s) * 64u + woff[r], b + (mine + r * 1024));
#pragma unroll
        for (int j = 0; j < XL; ++j) dma16(xp[j] + uint64_t(s) * (X4 ? 64u : 256u), b + (mine + kX + j * 1024));
        __builtin_amdgcn_sched_barrier(0);               // in this order: the waits count them
    };

    f32x4_t acc[NRB][NB];
#pragma unroll
    for (int r = 0; r < NRB; ++r)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[r][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // the step in `slot`, its scales at byte `at` of their rows' 16-byte units; zero: lanes of blocks that are not there
    auto compute = [&](int slot, uint32_t unit, uint32_t at, bool zero) {
        const uint8_t* const b = slot_base(slot);
        // one index that the compiler can't take apart: behind a chain of sums it no longer knows the array, and waits for
        // every load to LDS
        uint32_t so = uint32_t(wave * SB) * 1024u + unit * 256u + rl * 16u + at + q;
        asm("" : "+v"(so));
        const uint8_t* const sb = scale_buf + so;
        const uint8_t* const mine_w = b + (mine + place4(rl, q) * 16u);
        u32x4_t wf[NRB];
        uint32_t ws[NRB], xs[X4 ? NB : 1];
#pragma unroll
        for (int r = 0; r < NRB; ++r) {
            wf[r] = *reinterpret_cast<const u32x4_t*>(mine_w + r * 1024);
            ws[r] = sb[r * 1024];
        }
        u32x4_t xf[X4 ? 1 : 4][NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (X4) {
                xf[0][n] = *reinterpret_cast<const u32x4_t*>(mine_w + (kX + n * 1024));
                xs[X4 ? n : 0] = sb[(NRB + n) * 1024];
            } else {
                const uint32_t br = rl % uint32_t(NT);   // of 16-row tile n
#pragma unroll
                for (int k = 0; k < (X4 ? 1 : 4); ++k)
                    xf[k][n] = *reinterpret_cast<const u32x4_t*>(b + (mine + (br * 16u + ((4u * q + uint32_t(k)) ^ br)) * 16u) + (kX + n * 4096));
            }
        }
        if (zero) {
#pragma unroll
            for (int r = 0; r < NRB; ++r) {
                wf[r] = u32x4_t{0u, 0u, 0u, 0u};
                ws[r] = 127u;
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if (X4) xs[X4 ? n : 0] = 127u;
#pragma unroll
                for (int k = 0; k < (X4 ? 1 : 4); ++k) xf[k][n] = u32x4_t{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int r = 0; r < NRB; ++r) {
            if constexpr (X4) {
#pragma unroll
                for (int n = 0; n < NB; ++n) acc[r][n] = mfma_mx4<0, 0>(wf[r], ws[r], xf[0][n], xs[n], acc[r][n]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bf16x8_t w = mx4_to_bf16(wf[r][k], ws[r]);
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, xf[k][n]), acc[r][n], 0, 0, 0);
                }
            }
        }
        // every read of this slot has returned before it is refilled
        __builtin_amdgcn_sched_barrier(0);
    };

    // what the epilogue adds, for the wave's first output tile
    auto tile_row = [&](int i) { return row0 + 16u * uint32_t(PAIR ? 0 : i / NB) + 4u * q; };
    auto tile_b = [&](int i) { return 16u * uint32_t(i % NB) + rl; };
    EpilogueIn in{};
    for (uint32_t lo = s_lo; lo < s_hi;) {
        // a segment: the steps whose scales are loaded together
        const uint32_t unit = lo / 4u, hi = min(s_hi, 4u * unit + kSegment), last = hi - 1u;
        load_scales(unit);
#pragma unroll
        for (int d = 0; d < D; ++d) issue(min(lo + uint32_t(d), last), d);
        if (lo == s_lo && wave < TL && tile_b(wave) < uint32_t(t.rows) && tile_row(wave) < R)
            in = epilogue_load(a.g.ep, t.row0 + tile_b(wave), int(tile_row(wave)), a.g.R);
        __builtin_amdgcn_sched_barrier(0);
        // steps past the segment issue its last step again, so that the waits
        // are compile-time constants
        uint32_t s = lo;
        for (; s + D <= hi; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                wait_vm<(D - 1) * kPer, false>();
                const uint32_t i = s + uint32_t(d);
                compute(d, i / 4u - unit, i % 4u * 4u, false);
                issue(min(i + D, last), d);
            }
        }
#pragma unroll
        for (int d = 0; d < D - 1; ++d) {
            if (s + uint32_t(d) < hi) {
                wait_vm<(D - 1) * kPer, false>();
                const uint32_t i = s + uint32_t(d);
                compute(d, i / 4u - unit, i % 4u * 4u, false);
                issue(last, d);
            }
        }
        wait_vm<0, false>();                             // no load lands after its slot is used again
        lo = hi;
    }
    const uint32_t left = blocks % kStepB;
    if (left && wave == KW - 1) {                        // lanes behind the last block multiply zeros
        uint8_t* const b = slot_base(0);
        load_scales(steps / 4u);
#pragma unroll
        for (int r = 0; r < NRB; ++r) dma16(wb[PAIR ? r : 0] + uint64_t(steps) * 64u + woff[r] - (wc < left ? 0u : wc * 16u), b + (mine + r * 1024));
#pragma unroll
        for (int j = 0; j < XL; ++j)
            dma16(xp[j] + uint64_t(steps) * (X4 ? 64u : 256u) - (xc[j] < left * (X4 ? 1u : 4u) ? 0u : xc[j] * 16u), b + (mine + kX + j * 1024));
        wait_vm<0, false>();
        compute(0, 0u, steps % 4u * 4u, q >= left);
    }

    // D layout: lane l holds input row l%16 of its tile, weight rows 4*(l/16)..+3
    // of a block.  Wave w adds output tile w's (w + KW's ..) partial sums in wave order.
    __syncthreads();
    f32x4_t* const part = reinterpret_cast<f32x4_t*>(ring0);   // [KW][NRB][NB][64]
#pragma unroll
    for (int r = 0; r < NRB; ++r)
#pragma unroll
        for (int n = 0; n < NB; ++n) part[((wave * NRB + r) * NB + n) * 64 + int(lane)] = acc[r][n];
    __syncthreads();
    for (int i = wave; i < TL; i += KW) {
        const uint32_t b = tile_b(i), row = tile_row(i);
        f32x4_t y = part[i * 64 + int(lane)], u = PAIR ? part[(NB + i) * 64 + int(lane)] : y;
#pragma unroll
        for (int w = 1; w < KW; ++w) {
            y += part[(w * NRB * NB + i) * 64 + int(lane)];
            if (PAIR) u += part[(w * NRB * NB + NB + i) * 64 + int(lane)];
        }
        if (b >= uint32_t(t.rows) || row >= R) continue;
        if (PAIR) {
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = silu(y[c]) * u[c];
        }
        if (i != wave || s_lo == s_hi) in = epilogue_load(a.g.ep, t.row0 + b, int(row), a.g.R);
        epilogue_store(a.g.ep, in, t.row0 + b, int(row), a.g.R, y);
    }
}

template <bool X4, bool PAIR, int NRB, int NT, int KW, int D>
hipError_t launch(const Mx4Args& a, hipStream_t s) {
    const int64_t rows = PAIR ? 16 : 16 * NRB, bands = (a.g.R + rows - 1) / rows;
    const int64_t units = group_units(a.g, NT, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    launch_timed(mx4_skinny_kernel<X4, PAIR, NRB, NT, KW, D>, dim3(unsigned(units)), dim3(64 * KW), 0, s, a, uint32_t(bands));
    return hipGetLastError();
}

template <bool X4, bool PAIR, int NT>
hipError_t launch_nt(const Mx4Args& a, hipStream_t s) {
    constexpr int R = PAIR ? 2 : 1;
    constexpr int most = NT > 16 ? 4 : 8;
    switch (mx4_skinny_waves(NT, a)) {
        case 2: return launch<X4, PAIR, R, NT, 2, mx4_skinny_depth(NT, 2)>(a, s);
        case 4: return launch<X4, PAIR, R, NT, 4, mx4_skinny_depth(NT, 4)>(a, s);
        default: return launch<X4, PAIR, R, NT, most, mx4_skinny_depth(NT, most)>(a, s);
    }
}

template <bool X4, bool PAIR>
hipError_t launch_rows(const Mx4Args& a, int rows, hipStream_t s) {
    if constexpr (!X4)
        if (rows <= 4) return launch_nt<X4, PAIR, 4>(a, s);
    return rows <= 16 ? launch_nt<X4, PAIR, 16>(a, s) : launch_nt<X4, PAIR, 32>(a, s);
}

}  // namespace

// Waves that split K: the fewest (2, 4 or 8; 4 with 32 input rows) that give about six waves a compute unit.  With 16
// rows 4096 x 14336 takes 14.8 us on 4 waves and 12.7 on 8, 14336 x 4096 10.7, 14.1 and 18.6 on 2, 4 and 8, pairs of 64
// experts of 1408 x 2048 with four rows each 53.5, 68 and 104; one row with 1024 x 4096 5.7, 4.8 and 4.2.
int mx4_skinny_waves(int rows, const Mx4Args& a) {
    const int64_t bands = (int64_t(a.g.R) + 15) / 16, groups = a.g.offsets || a.g.E > 1 ? std::min<int64_t>(a.g.n, a.g.E) : 1;
    const int64_t units = bands * std::max<int64_t>(groups, a.g.offsets ? 1 : (a.g.n + rows - 1) / rows), want = 6 * int64_t(a.g.cus);
    return 2 * units >= want ? 2 : rows > 16 || 4 * units >= want ? 4 : 8;
}

hipError_t launch_mx4_skinny(bool x4, bool pair, const Mx4Args& a, int rows, hipStream_t s) {
    if (x4) return pair ? launch_rows<true, true>(a, rows, s) : launch_rows<true, false>(a, rows, s);
    return pair ? launch_rows<false, true>(a, rows, s) : launch_rows<false, false>(a, rows, s);
}

}  // namespace uwk

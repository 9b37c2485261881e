// Many rows per expert (or a large batch of the epilogue matmul): the matrix
// units bound the product.  bf16 weights.
//
// A workgroup multiplies MT weight rows with NT input rows in steps of 64
// columns.  Both tiles go from memory to LDS by global_load_lds, S steps of
// them there or on their way.  A wave owns a (MT/WM) x (NT/2) block of the
// output: 64 x 64 with 256 x 128 tiles and eight waves, 16 fragments of 1 KB
// from LDS for 32 MFMAs of 16 cycles a step; 64 x 128 with 256 x 256, 24 for 64:
// three quarters of the LDS reads an MFMA.  Fragments
// of the next 32 columns are read into a second register set while the MFMAs
// of these run.  One barrier a step, in its middle: by then every wave has the
// step's last fragments in registers and its own loads of the next step have
// landed, so the step's buffers can be refilled.
//   8192 x 8192 x 8192: 916 us with 256 x 256 (1200 TFLOP/s), 984 with
// 256 x 128, 1362 with 128 x 64, 2424 with 64 x 64; small products have too few
// of the large ones for every compute unit, and waste less of the small ones
// behind an expert's last row.  128 x 128 tiles, one or two a compute unit, were
// no better than 256 x 128 (4000 tokens of 8 experts: 101 against 96 us; 3000 of
// 64: 190 and 184).
//   Rows of a tile are 128 bytes in LDS; 16-byte chunk c of row r sits at
// position c ^ (r & 7) ^ (r >> 3 & 1), which makes the fragment reads (16 rows,
// one chunk column) free of bank conflicts while four lanes of a load still
// take 64 contiguous bytes of one row.
//   The gate/up pair: half of a tile's rows are gate's and half up's, each wave
// owns the same rows of both, so the SiLU product needs no exchange.
#include "grouped_common.h"
#include "kernels.h"

namespace uwk {

namespace {

constexpr int kStep = 64;

template <bool PAIR, int MT, int NT, int WM, int S>
__global__ __launch_bounds__(128 * WM, 1) void tile_kernel(GroupArgs a, uint32_t bands) {
    constexpr int WN = 2, NW = WM * WN;                  // waves across the input rows, in all
    constexpr int FM = MT / 16 / WM, FN = NT / 16 / WN;  // 16-row blocks of a wave's output
    constexpr int WD = MT / 8 / NW, XD = NT / 8 / NW;    // loads of a wave and step
    constexpr int kRows = PAIR ? MT / 2 : MT;            // rows of a matrix in a tile
    // a step's two tiles, an array per buffer (the compiler can tell them apart)
    constexpr int kBuf = (MT + NT) * kStep;
    __shared__ __align__(16) uint16_t buf0[kBuf], buf1[kBuf], buf2[S > 2 ? kBuf : 8], buf3[S > 3 ? kBuf : 8];
    // floats between the input rows of the part of the outputs that the epilogue
    // has in the first buffer: spread over the banks
    constexpr int ES = kRows + 4;
    static_assert(16 * WN * ES * 4 <= kBuf * 2, "a part of the outputs fits a buffer");
    static_assert((S - 2) * (WD + XD) < 64, "loads in flight");

    GroupTile t;
    if (!group_tile<NT>(a, bands, t)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const uint32_t R = uint32_t(a.R), C = uint32_t(a.C);
    const uint32_t row0 = uint32_t(t.band) * kRows;
    // the slice's steps (all of them without a split)
    const uint32_t s_lo = uint32_t(uint64_t(C / kStep) * uint32_t(t.slice) / uint32_t(a.split));
    const uint32_t steps = uint32_t(uint64_t(C / kStep) * uint32_t(t.slice + 1) / uint32_t(a.split)) - s_lo;
    const int64_t first = int64_t(t.e) * R * C;

    // sources: load j of this wave covers 8 rows of the tile
    const uint32_t lr = lane >> 3;
    uint32_t woff[WD];
    const uint8_t* wb[PAIR ? 2 : 1];
#pragma unroll
    for (int m = 0; m < (PAIR ? 2 : 1); ++m)
        wb[m] = static_cast<const uint8_t*>(a.w[m].w) + first * 2;
#pragma unroll
    for (int j = 0; j < WD; ++j) {
        const uint32_t blk = uint32_t(wave * WD + j);                      // of 8 rows
        const uint32_t row = row0 + (blk * 8u + lr) % uint32_t(kRows);     // pair: the second half is up's
        woff[j] = min(row, R - 1u) * C * 2u + (((lane & 7u) ^ lr ^ (blk & 1u)) * 16u);
    }
    const uint8_t* xp[XD];
#pragma unroll
    for (int j = 0; j < XD; ++j) {
        const uint32_t blk = uint32_t(wave * XD + j);
        xp[j] = reinterpret_cast<const uint8_t*>(group_x_row(a, t.row0 + min(blk * 8u + lr, uint32_t(t.rows) - 1u))) +
                (((lane & 7u) ^ lr ^ (blk & 1u)) * 16u);
    }
    auto buffer = [&](int i) -> uint16_t* { return i == 0 ? buf0 : i == 1 ? buf1 : i == 2 ? buf2 : buf3; };
    // steps past the end load the last one again: the waits count the same loads in every step
    auto load = [&](uint32_t s, int i) {
        uint16_t* const w = buffer(i), * const x = w + MT * kStep;
        s = s_lo + min(s, steps - 1u);
#pragma unroll
        for (int j = 0; j < WD; ++j) {
            const int m = PAIR ? (wave * WD + j) * 8 / kRows : 0;          // uniform
            dma16(wb[m] + uint64_t(s) * 128u + woff[j], w + (wave * WD + j) * 512);
        }
#pragma unroll
        for (int j = 0; j < XD; ++j) dma16(xp[j] + uint64_t(s) * 128u, x + (wave * XD + j) * 512);
    };

    // fragments: row block i of the wave, half h of the step
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t sw = (rl & 7u) ^ (rl >> 3);
    const uint32_t ro = rl * 64u;
    struct Frags {
        bf16x8_t A[FM], B[FN];
    };
    auto read = [&](int b, int h, Frags& f) {
        const uint16_t* const w = buffer(b), * const x = w + MT * kStep;
        const uint32_t o = ro + (((4u * uint32_t(h) + q) ^ sw) * 8u);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int blk = PAIR ? (i < FM / 2 ? wm * FM / 2 + i : MT / 32 + wm * FM / 2 + i - FM / 2) : wm * FM + i;
            f.A[i] = *reinterpret_cast<const bf16x8_t*>(w + blk * 1024 + o);
        }
#pragma unroll
        for (int i = 0; i < FN; ++i) f.B[i] = *reinterpret_cast<const bf16x8_t*>(x + (wn * FN + i) * 1024 + o);
    };
    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](const Frags& f) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.A[i], f.B[j], acc[i][j], 0, 0, 0);
    };
    // a half: fragment reads spread among the MFMAs
    auto mixed = [&]() {
#pragma unroll
        for (int i = 0; i < FM + FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, FM * FN / (FM + FN), 0);
        }
    };

    // one step in buffer i: half 0 on f0, then the barrier, the loads S steps
    // ahead, half 1 on f1
    Frags f0, f1;
    auto step = [&](uint32_t s, int i) {
        read(i, 1, f1);
        mma(f0);
        mixed();
        __builtin_amdgcn_sched_barrier(0);
        // the next step's loads and this step's fragments are here
        wait_vm<(S - 2) * (WD + XD), true>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load(s + S, i);
        read((i + 1) % S, 0, f0);
        mma(f1);
        mixed();
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int i = 0; i < S; ++i) {
        load(uint32_t(i), i);
        __builtin_amdgcn_sched_barrier(0);               // in this order: the waits count them
    }
    wait_vm<(S - 1) * (WD + XD), true>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(0, 0, f0);
    uint32_t s = 0;
    for (; s + S <= steps; s += S) {
#pragma unroll
        for (int i = 0; i < S; ++i) step(s + uint32_t(i), i);
    }
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (s + uint32_t(i) < steps) step(s + uint32_t(i), i);
    __builtin_amdgcn_s_waitcnt(0);                       // no load is on its way to LDS that the epilogue uses

    // The epilogue in parts of a 16-row block of each wave column's inputs:
    // through LDS, so that a row of the output is written in one run and the
    // code is there once.  D layout: lane l holds input row l%16, weight rows
    // 4*(l/16)..+3 of a block.
    constexpr int OM = PAIR ? FM / 2 : FM;
    float* const part = reinterpret_cast<float*>(buf0);
    Epilogue ep = a.ep;
    if (!PAIR && a.split > 1)
        ep = Epilogue{nullptr, nullptr, a.sums + int64_t(t.slice) * a.n * a.R, 0, a.R, VT_F32, VT_F32, VT_F32, ACT_NONE};
    PartEpilogue<kRows, 16 * WN, 64 * NW, ES> out(ep, part, t, row0, a.R, tid);
    auto rows_of = [](int p) { return [p](int n) { return ((n / 16) * FN + p) * 16 + n % 16; }; };
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

template <bool PAIR, int MT, int NT, int WM, int S>
hipError_t launch(const GroupArgs& a, hipStream_t s) {
    const int64_t rows = PAIR ? MT / 2 : MT, bands = (a.R + rows - 1) / rows;
    const int64_t units = group_units(a, NT, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    launch_timed(tile_kernel<PAIR, MT, NT, WM, S>, dim3(unsigned(units)), dim3(128 * WM), 0, s, a, uint32_t(bands));
    return hipGetLastError();
}

template <bool PAIR>
hipError_t launch_shape(const GroupArgs& a, TileShape shape, hipStream_t s) {
    switch (shape) {
        case TILE_64x64: return launch<PAIR, 64, 64, 2, 4>(a, s);
        case TILE_128x64: return launch<PAIR, 128, 64, 4, 3>(a, s);
        case TILE_256x128: return launch<PAIR, 256, 128, 4, 3>(a, s);
        // the pair's registers do not fit: 316 us against 280 (3000 tokens of 64 experts)
        default: return PAIR ? hipErrorInvalidValue : launch<false, 256, 256, 4, 2>(a, s);
    }
}

}  // namespace

hipError_t launch_tile(bool pair, const GroupArgs& a, TileShape shape, hipStream_t s) {
    return pair ? launch_shape<true>(a, shape, s) : launch_shape<false>(a, shape, s);
}

}  // namespace uwk

// Many rows per expert, direct-palette weights without scratch to expand them
// in: as the bf16 tile kernel, with the weight tile rebuilt on its way to LDS.
//
// A weight's indices, sign/mantissa byte and (in verbatim groups) raw exponent
// come to registers P + 1 steps ahead, input rows go to LDS by global_load_lds.
// A lane rebuilds 16 weights of a row a step, eight at a time: the 4-bit
// indices pick their exponents by byte permutes of the 16 palette bytes held
// in scalar registers (an LDS table, as the weight-bound kernels use it, would
// take the LDS's time from the fragments), a verbatim lane selects the raw
// bytes instead, and sign, mantissa and exponent are joined two weights at a
// time.  One half of a step's rebuild runs under the MFMAs of each half step.
//   Bound by the vector instructions of the rebuild and the LDS traffic next to
// the MFMAs: 8192 x 8192 x 8192 in 1.60 ms (690 TFLOP/s) with 128 x 128 tiles;
// 192 or 256 weight rows, 12 waves or a deeper ring were no faster: none of them
// changes the rebuild's share of an MFMA, which more input rows a tile would.
#include "grouped_common.h"
#include "kernels.h"

namespace uwk {

namespace {

constexpr int kStep = 64;            // columns of a step: one group of every row

// Exponents of the four 4-bit indices in the bytes of n by byte permutes: both
// 8-entry halves of the palette are looked up, the index's top bit selects.
__device__ __forceinline__ uint32_t look4(uint32_t n, const uint32_t (&pal)[4]) {
    const uint32_t sel = n & 0x07070707u, top = n & 0x08080808u;
    const uint32_t lo = __builtin_amdgcn_perm(pal[1], pal[0], sel), hi = __builtin_amdgcn_perm(pal[3], pal[2], sel);
    const uint32_t mask = (top << 5) - (top >> 3);       // 0xFF where the top bit is set
    return (lo & ~mask) | (hi & mask);
}

template <bool PAIR, int MT, int NT, int WM, int WN, int P>
__global__ __launch_bounds__(64 * WM * WN, 1) void tile_pal_kernel(GroupArgs a, uint32_t bands) {
    constexpr int NW = WM * WN;
    constexpr int FM = MT / 16 / WM, FN = NT / 16 / WN;
    constexpr int IT = MT / 16 / NW;                     // 16-weight items of a lane and step
    constexpr int XD = (NT / 8 + NW - 1) / NW;           // input loads of a wave and step
    constexpr int kRows = PAIR ? MT / 2 : MT;
    static_assert(IT >= 1, "whole items");
    // (1 KB more than the tile: the part of the outputs that the epilogue has there)
    __shared__ __align__(16) uint16_t wb0[MT * kStep + 512], wb1[MT * kStep];
    __shared__ __align__(16) uint16_t xb0[NT * kStep], xb1[NT * kStep], xb2[P > 1 ? NT * kStep : 8], xb3[P > 2 ? NT * kStep : 8];
    constexpr int ES = kRows + 4;
    constexpr int EC = WN < 2 ? WN : 2;                  // wave columns of a part
    static_assert(16 * EC * ES * 4 <= (MT * kStep + 512) * 2, "a part of the outputs fits a buffer");
    float* const part = reinterpret_cast<float*>(wb0);

    GroupTile t;
    if (!group_tile<NT>(a, bands, t)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const uint32_t R = uint32_t(a.R), C = uint32_t(a.C);
    const uint32_t row0 = uint32_t(t.band) * kRows, steps = C / kStep;
    const int64_t first = int64_t(t.e) * R * C;
    // items: row block wave + NW*it, row lane/4, columns 16*(lane%4)
    // (pair) a matrix's blocks are whole rounds of the waves, or the waves are split between the two
    auto item_m = [&](int it) -> int { return !PAIR ? 0 : MT / 32 >= NW ? it * NW / (MT / 32) : wave / (MT / 32); };
    auto item_blk = [&](int it) -> uint32_t { return uint32_t(wave + NW * it); };
    const uint32_t ir = lane >> 2, ic = (lane & 3u) * 16u;
    uint32_t wrow[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) wrow[it] = min(row0 + (item_blk(it) * 16u + ir) % uint32_t(kRows), R - 1u);
    struct Set {
        u32x2_t nib[IT];
        u32x4_t sm[IT], vx[IT];
        uint32_t flag[IT];
    };
    // flags of the row's groups from the next step on, slots before it (relative to the expert's first tile)
    uint32_t fl[IT][4], slot[IT], base[IT];
    auto tables = [&](uint32_t s0) {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const Weight& w = a.w[item_m(it)];
            const int64_t g0 = (first + int64_t(wrow[it]) * C) >> 6, g = g0 + min(s0, steps - 1u);
            const int64_t end = g0 + min(s0 + 64u, steps) - 1;
            const uint64_t w0 = w.bitmap[g >> 6], w1 = w.bitmap[max(g, end) >> 6];
            base[it] = min(w.tile_vbase[first >> 12], w.last_slot);
            const uint32_t bit = uint32_t(g) & 63u;
            slot[it] = w.tile_vbase[g >> 6] - base[it] + uint32_t(__popcll(w0 & ((uint64_t(1) << bit) - 1)));
            uint64_t lo = bit ? (w0 >> bit) | (w1 << (64u - bit)) : w0;
            const int64_t left = end - g + 1;            // steps past the segment find no flag
            if (left < 64) lo &= (uint64_t(1) << left) - 1;
            fl[it][0] = uint32_t(lo);
            fl[it][1] = uint32_t(lo >> 32);
        }
    };
    auto load_w = [&](uint32_t s, Set& st) {
        const uint32_t k = min(s, steps - 1u) * kStep + ic;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const Weight& w = a.w[item_m(it)];
            const uint32_t o = wrow[it] * C + k;
            st.nib[it] = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(w.w) + first / 2 + o / 2);
            st.sm[it] = load16(w.sm + first + o);
            st.flag[it] = fl[it][0] & 1u;
            const uint32_t off = st.flag[it] ? slot[it] * 64u + ic : 0u;
            st.vx[it] = load16(w.vexp + uint64_t(base[it]) * 64u + off);
            slot[it] += fl[it][0] & 1u;
            fl[it][0] = __builtin_amdgcn_alignbit(fl[it][1], fl[it][0], 1);
            fl[it][1] >>= 1;
        }
    };
    // rebuilds item it of a set into weight buffer b
    const uint32_t isw = (ir & 7u) ^ (ir >> 3);
    auto wbuf = [&](int b) -> uint16_t* { return b ? wb1 : wb0; };
    auto xbuf = [&](int b) -> uint16_t* { return b == 0 ? xb0 : b == 1 ? xb1 : b == 2 ? xb2 : xb3; };
    auto rebuild = [&](const Set& st, int it, int b) {
        uint32_t pal[4], w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) pal[i] = a.w[item_m(it)].pal[i];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t n = st.nib[it][h], v0 = st.vx[it][2 * h], v1 = st.vx[it][2 * h + 1];
            uint32_t ev = look4(n & 0x0F0F0F0Fu, pal), od = look4((n >> 4) & 0x0F0F0F0Fu, pal);
            // a verbatim lane takes its raw exponents (a select: no branch splits the MFMAs' schedule)
            ev = st.flag[it] ? __builtin_amdgcn_perm(v1, v0, 0x06040200u) : ev;
            od = st.flag[it] ? __builtin_amdgcn_perm(v1, v0, 0x07050301u) : od;
#pragma unroll
            for (int p = 0; p < 4; ++p) {                                  // [0, even, 0, odd] >> 1
                const uint32_t e7 = __builtin_amdgcn_perm(od, ev, 0x040C000Cu + 0x01000100u * uint32_t(p)) >> 1;
                w[4 * h + p] = (p & 1) ? join_pair<1>(st.sm[it][2 * h + (p >> 1)], e7)
                                       : join_pair<0>(st.sm[it][2 * h + (p >> 1)], e7);
            }
        }
        uint16_t* const d = wbuf(b) + (item_blk(it) * 16u + ir) * 64u;
        const uint32_t c = (lane & 3u) * 2u;
        store16(d + ((c ^ isw) * 8u), u32x4_t{w[0], w[1], w[2], w[3]});
        store16(d + (((c + 1u) ^ isw) * 8u), u32x4_t{w[4], w[5], w[6], w[7]});
    };

    const uint32_t lr = lane >> 3;
    const uint8_t* xp[XD];
#pragma unroll
    for (int j = 0; j < XD; ++j) {
        const uint32_t blk = min(uint32_t(wave * XD + j), NT / 8u - 1u);   // past the tile: its last again
        xp[j] = reinterpret_cast<const uint8_t*>(group_x_row(a, t.row0 + min(blk * 8u + lr, uint32_t(t.rows) - 1u))) +
                (((lane & 7u) ^ lr ^ (blk & 1u)) * 16u);
    }
    auto load_x = [&](uint32_t s, int b) {
        s = min(s, steps - 1u);
#pragma unroll
        for (int j = 0; j < XD; ++j) dma16(xp[j] + uint64_t(s) * 128u, xbuf(b) + min(wave * XD + j, NT / 8 - 1) * 512);
    };

    const int wm = wave / WN, wn = wave % WN;
    const uint32_t sw = (rl & 7u) ^ (rl >> 3);
    struct Frags {
        bf16x8_t A[FM], B[FN];
    };
    auto read = [&](int b, int xb, int h, Frags& f) {
        const uint32_t o = rl * 64u + (((4u * uint32_t(h) + q) ^ sw) * 8u);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int blk = PAIR ? (i < FM / 2 ? wm * FM / 2 + i : MT / 32 + wm * FM / 2 + i - FM / 2) : wm * FM + i;
            f.A[i] = *reinterpret_cast<const bf16x8_t*>(wbuf(b) + blk * 1024 + o);
        }
#pragma unroll
        for (int i = 0; i < FN; ++i) f.B[i] = *reinterpret_cast<const bf16x8_t*>(xbuf(xb) + (wn * FN + i) * 1024 + o);
    };
    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](const Frags& f) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < FM; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.A[i], f.B[j], acc[i][j], 0, 0, 0);
    };

    constexpr int NS = P + 1, U = NS % 2 ? 2 * NS : NS;  // sets and input buffers; steps of an unrolled pass
    constexpr int kWait = 3 * IT + (P - 1) * (XD + 3 * IT);
    Set st[NS];
    Frags f0;
    // step s = i mod U: the set of step s+2 is rebuilt into the weight buffer
    // that the step frees, in its second half and the next step's first
    auto step = [&](uint32_t s, int i) {
        mma(f0);
        if (IT > 1) {
#pragma unroll
            for (int it = 1; it < IT; ++it) rebuild(st[(i + 1) % NS], it, (i + 1) % 2);
        }
        read(i % 2, i % NS, 1, f0);
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<kWait, true>();                                   // the next step's input rows have landed
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load_x(s + P + 1, i % NS);
        __builtin_amdgcn_sched_barrier(0x40F);           // before the loads of weights: the wait counts on it
        if (((s + P + 2) & 63u) == 0 && s + P + 2 < steps) tables(s + P + 2);
        load_w(s + P + 2, st[(i + 1) % NS]);
        mma(f0);
        rebuild(st[(i + 2) % NS], 0, i % 2);
        read((i + 1) % 2, (i + 1) % NS, 0, f0);
        __builtin_amdgcn_sched_barrier(0);
    };
    tables(0);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        load_x(uint32_t(i), i);
        __builtin_amdgcn_sched_barrier(0);
        load_w(uint32_t(i), st[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();                                     // everything has landed
#pragma unroll
    for (int it = 0; it < IT; ++it) rebuild(st[0], it, 0);
    load_w(NS, st[0]);
    rebuild(st[1], 0, 1);
    __builtin_amdgcn_s_waitcnt(0xC07F);                  // LDS only
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(0, 0, 0, f0);
    uint32_t s = 0;
    for (; s + U <= steps; s += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) step(s + uint32_t(i), i);
    }
#pragma unroll
    for (int i = 0; i < U - 1; ++i)
        if (s + uint32_t(i) < steps) step(s + uint32_t(i), i);
    __builtin_amdgcn_s_waitcnt(0);

    constexpr int OM = PAIR ? FM / 2 : FM;
    PartEpilogue<kRows, 16 * EC, 64 * NW, ES> out(a.ep, part, t, row0, a.R, tid);
    auto rows_of = [](int p) { return [p](int n) { return ((p / FN * EC + n / 16) * FN + p % FN) * 16 + n % 16; }; };
    out.load(rows_of(0));
#pragma unroll 1
    for (int p = 0; p < FN * (WN / EC); ++p) {
        __syncthreads();
        const int c0 = p / FN * EC;                      // first wave column of the part
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if (p % FN != j || wn < c0 || wn >= c0 + EC) continue;
#pragma unroll
            for (int i = 0; i < OM; ++i) {
                f32x4_t v = acc[i][j];
                if (PAIR) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = silu(v[c]) * acc[FM - OM + i][j][c];
                }
                *reinterpret_cast<f32x4_t*>(part + ((wn - c0) * 16 + int(rl)) * ES + (wm * OM + i) * 16 + 4 * int(q)) = v;
            }
        }
        __syncthreads();
        out.store(rows_of(p), p + 1 < FN * (WN / EC), rows_of(p + 1));
    }
}

template <bool PAIR, int MT, int NT, int WM, int WN, int P>
hipError_t launch(const GroupArgs& a, hipStream_t s) {
    const int64_t rows = PAIR ? MT / 2 : MT, bands = (a.R + rows - 1) / rows;
    const int64_t units = group_units(a, NT, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    launch_timed(tile_pal_kernel<PAIR, MT, NT, WM, WN, P>, dim3(unsigned(units)), dim3(64 * WM * WN), 0, s, a,
                 uint32_t(bands));
    return hipGetLastError();
}

template <bool PAIR>
hipError_t launch_shape(const GroupArgs& a, PalTileShape shape, hipStream_t s) {
    switch (shape) {
        case PAL_TILE_64x64: return launch<PAIR, 64, 64, 2, 2, 2>(a, s);
        case PAL_TILE_128x64: return launch<PAIR, 128, 64, 4, 2, 2>(a, s);
        default: return launch<PAIR, 128, 128, 4, 2, 1>(a, s);
    }
}

}  // namespace

hipError_t launch_tile_pal(bool pair, const GroupArgs& a, PalTileShape shape, hipStream_t s) {
    return pair ? launch_shape<true>(a, shape, s) : launch_shape<false>(a, shape, s);
}

}  // namespace uwk

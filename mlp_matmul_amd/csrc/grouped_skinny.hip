// Few rows per expert (or a small batch of the epilogue matmul): the product
// is bound by the weight stream, every weight is read once and used for up to
// 4*XQ input rows.
//
// A wave owns a 16-row block of weights (the pair: the same rows of gate and
// up) and one K-slice, in steps of 128 columns.  Each step's operands go from
// memory to the wave's own LDS ring by global_load_lds (16 bytes a lane, a
// row's bytes side by side), two steps in flight: the loads in flight cost LDS
// and no registers, and the read-back in the MFMA operand layout (16 rows side
// by side) is a conflict-free LDS read, where loading that layout from memory
// would cost the vector cache one access per row.  The KW waves of a workgroup split K
// and add their partial sums in wave order through LDS, then the epilogue
// runs on the sum: results do not depend on scheduling.
//   bf16 weights: 16 rows x 256 bytes a step and block, four loads.
//   direct palette: 16 x 64 bytes of 4-bit indices and 16 x 128 of
//     sign/mantissa bytes, three loads; rebuilt in registers through a
//     256-entry LDS table of exponent pairs; verbatim lanes take the raw
//     exponents, which come in registers with the step's loads.
// The verbatim tables of a row's columns are kept in registers for segments
// of 4096 columns (at most two tiles of 64 groups); longer K-slices run one
// segment after another.  A last step of 64 columns multiplies zeros by zeros
// in its upper half.
//   Measured: gate/up of 33 tokens, 16 experts of 1792 x 4096 in bf16, 87 us for
// 470 MB (5.4 TB/s); 16 rows of 4096 x 14336, palette, 22 us for 91 MB, 6 of
// them the launch, the first loads and the last sums.
#include <algorithm>

#include "grouped_common.h"
#include "kernels.h"

namespace uwk {

namespace {

constexpr int kStepK = 128;          // columns of a step
constexpr int kSegment = 4096;       // columns whose verbatim tables are in registers

__device__ __forceinline__ u32x4_t lds16(const uint8_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

template <bool PAL, bool PAIR, int NRB, int XQ, int KW>
__global__ __launch_bounds__(64 * KW) void skinny_kernel(GroupArgs a, uint32_t bands) {
    static_assert(!PAIR || NRB == 2, "the pair: one block of each matrix");
    constexpr int D = 2;                                 // steps in flight
    constexpr int NT = 4 * XQ, NB = (NT + 15) / 16;      // input rows, 16-row tiles of them
    constexpr int M = PAIR ? 2 : 1;
    constexpr int WL = PAL ? 3 : 4;                      // weight loads of a block's step
    constexpr int kBlock = 1024 * WL;                    // bytes of a row block's step
    constexpr int kXOff = NRB * kBlock, kSlot = kXOff + XQ * 1024;
    constexpr int kV = PAL ? 2 * NRB : 0;                // loads of verbatim exponents of a step
    constexpr int kPer = NRB * WL + XQ + kV;             // vector memory operations of a step
    constexpr int TL = PAIR ? NB : NRB * NB;             // 16x16 tiles of outputs
    static_assert(kPer < 64 && XQ + 2 * kV < 64, "loads in flight");
    static_assert(NRB * NB * 1024 <= kSlot, "partial sums fit the first slots");
    __shared__ uint32_t lut[PAL ? 256 * M : 1];
    __shared__ __align__(16) uint8_t ring0[KW * kSlot];  // an array per slot: the compiler can tell them apart
    __shared__ __align__(16) uint8_t ring1[KW * kSlot];

    GroupTile t;
    if (!group_tile<NT>(a, bands, t)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const uint32_t R = uint32_t(a.R), C = uint32_t(a.C);
    constexpr uint32_t kRows = PAIR ? 16u : 16u * NRB;
    const uint32_t row0 = uint32_t(t.band) * kRows;
    const uint32_t steps = C / kStepK;                   // whole ones; 64 columns may be left to the last wave
    const uint32_t s_lo = steps * uint32_t(wave) / KW, s_hi = steps * uint32_t(wave + 1) / KW;

    // the expert's matrices: uniform bases, offsets inside them fit 32 bits
    const int64_t first = int64_t(t.e) * R * C;
    auto mat = [&](int r) -> const Weight& { return a.w[PAIR ? r : 0]; };
    auto wbase = [&](int r) -> const uint8_t* {
        return static_cast<const uint8_t*>(mat(r).w) + (PAL ? first / 2 : first * 2);
    };
    // row i of block r; rows past the expert's read its last one and are not stored
    auto row_at = [&](int r, uint32_t i) -> uint32_t {
        return min(row0 + (PAIR ? 0u : 16u * uint32_t(r)) + i, R - 1u);
    };
    // a lane's 16-byte chunk c of a row is the one that lands at the chunk
    // position the swizzle gives it.  LAST: 64 columns are left, the upper
    // chunks read the lower ones' bytes again.
    auto chunk = [&](uint32_t c, uint32_t per, bool last) { return (last && c >= per / 2 ? c - per / 2 : c) * 16u; };
    auto woff = [&](int r, int j, bool last) -> uint32_t {
        if (!PAL) {
            const uint32_t n = 64u * uint32_t(j) + lane, i = n >> 4;
            return row_at(r, i) * C * 2u + chunk((n & 15u) ^ (i & 7u), 16, last);
        }
        if (j == 0) {
            const uint32_t i = lane >> 2;
            return row_at(r, i) * (C / 2u) + chunk((lane & 3u) ^ ((i >> 1) & 3u), 4, last);
        }
        const uint32_t n = 64u * uint32_t(j - 1) + lane, i = n >> 3;
        return row_at(r, i) * C + chunk((n & 7u) ^ (i & 7u), 8, last);
    };
    auto xoff = [&](int j, bool last) -> uint32_t {
        const uint32_t n = 64u * uint32_t(j) + lane, b = n >> 4;
        return chunk((n & 15u) ^ (b & 7u), 16, last);
    };
    const uint16_t* xrow[XQ];
#pragma unroll
    for (int j = 0; j < XQ; ++j) xrow[j] = group_x_row(a, t.row0 + min((64u * uint32_t(j) + lane) >> 4, uint32_t(t.rows) - 1u));

    // verbatim groups: the flags of the lane's row from its group of the next
    // step on (128 bits shifted along), and the number of verbatim groups of
    // the expert before it
    uint32_t fl[NRB][4], slot[NRB], base[NRB];
    auto load_tables = [&](uint32_t s0, uint32_t s1) {
        if (!PAL) return;
#pragma unroll
        for (int r = 0; r < NRB; ++r) {
            const int64_t g0 = (first + int64_t(row_at(r, rl)) * C) >> 6, g = g0 + 2 * s0;
            const int64_t end = g0 + min(2 * s1, C / 64u) - 1;         // the segment's last group
            const uint64_t w0 = mat(r).bitmap[g >> 6], w1 = mat(r).bitmap[max(g, end) >> 6];
            const uint32_t before = mat(r).tile_vbase[g >> 6];
            base[r] = min(mat(r).tile_vbase[first >> 12], mat(r).last_slot);   // uniform: slots below are the expert's own
            const uint32_t bit = (uint32_t(g) & 63u) + (q >> 1);       // may be 64: the next word's first
            slot[r] = before - base[r] + uint32_t(__popcll(bit > 63u ? w0 : w0 & ((uint64_t(1) << bit) - 1)));
            uint64_t lo = bit > 63u ? w1 : (bit ? (w0 >> bit) | (w1 << (64u - bit)) : w0);
            uint64_t hi = bit > 63u ? 0 : w1 >> bit;
            // steps issued past the segment find no flag: no slot behind the last is read
            const int64_t left = end - g - int64_t(q >> 1) + 1;
            if (left < 64) {
                lo &= left > 0 ? (uint64_t(1) << left) - 1 : 0;
                hi = 0;
            } else if (left < 128) {
                hi &= (uint64_t(1) << (left - 64)) - 1;
            }
            fl[r][0] = uint32_t(lo);
            fl[r][1] = uint32_t(lo >> 32);
            fl[r][2] = uint32_t(hi);
            fl[r][3] = uint32_t(hi >> 32);
        }
    };

    struct Verbatim {
        u32x4_t vx[NRB][2];
        uint32_t flag[NRB];
    };
    auto slot_base = [&](int j) -> uint8_t* { return (j ? ring1 : ring0) + wave * kSlot; };
    uint32_t wo[NRB][WL];
    const uint8_t* xp[XQ];
    auto set_offsets = [&](bool last) {
#pragma unroll
        for (int r = 0; r < NRB; ++r)
#pragma unroll
            for (int j = 0; j < WL; ++j) wo[r][j] = woff(r, j, last);
#pragma unroll
        for (int j = 0; j < XQ; ++j) xp[j] = reinterpret_cast<const uint8_t*>(xrow[j]) + xoff(j, last);
    };
    auto issue_w = [&](uint32_t s, int j) {
        uint8_t* const b = slot_base(j);
#pragma unroll
        for (int r = 0; r < NRB; ++r)
#pragma unroll
            for (int i = 0; i < WL; ++i) {
                const uint8_t* const src = !PAL ? wbase(r) + uint64_t(s) * 256u
                                         : i    ? mat(r).sm + first + uint64_t(s) * 128u
                                                : wbase(r) + uint64_t(s) * 64u;
                dma16(src + wo[r][i], b + r * kBlock + 1024 * i);
            }
    };
    auto issue_x = [&](uint32_t s, int j) {
        uint8_t* const b = slot_base(j) + kXOff;
#pragma unroll
        for (int i = 0; i < XQ; ++i) dma16(xp[i] + uint64_t(s) * 256u, b + 1024 * i);
    };
    // the raw exponents of the lane's 32 weights (other lanes: one shared line)
    auto issue_v = [&](Verbatim& v) {
        if (!PAL) return;
#pragma unroll
        for (int r = 0; r < NRB; ++r) {
            v.flag[r] = fl[r][0] & 1u;
            const uint32_t off = v.flag[r] ? slot[r] * 64u + 32u * (q & 1u) : 0u;
            const uint8_t* const p = mat(r).vexp + uint64_t(base[r]) * 64u;
            v.vx[r][0] = load16(p + off);
            v.vx[r][1] = load16(p + off + 16);
            slot[r] += uint32_t(__popc(fl[r][0] & 3u));
            fl[r][0] = __builtin_amdgcn_alignbit(fl[r][1], fl[r][0], 2);
            fl[r][1] = __builtin_amdgcn_alignbit(fl[r][2], fl[r][1], 2);
            fl[r][2] = __builtin_amdgcn_alignbit(fl[r][3], fl[r][2], 2);
            fl[r][3] >>= 2;
        }
    };
    auto issue = [&](uint32_t s, int j, Verbatim& v) {
        issue_w(s, j);
        issue_x(s, j);
        issue_v(v);
        // the step's loads stay together: the waits count them in issue order
        __builtin_amdgcn_sched_barrier(0);
    };

    f32x4_t acc[NRB][NB];
#pragma unroll
    for (int r = 0; r < NRB; ++r)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[r][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](int j, const Verbatim& v, bool zero) {
        const uint8_t* const b = slot_base(j);
        u32x4_t xf[4][NB], wf[NRB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const uint32_t br = (16u * uint32_t(n) + rl) % uint32_t(NT);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                xf[i][n] = lds16(b + kXOff + (br * 16u + ((4u * q + uint32_t(i)) ^ (br & 7u))) * 16u);
        }
        if (PAL) {
            u32x4_t nb[NRB], sm[NRB][2];
#pragma unroll
            for (int r = 0; r < NRB; ++r) {
                nb[r] = lds16(b + r * kBlock + (rl * 4u + (q ^ ((rl >> 1) & 3u))) * 16u);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sm[r][h] = lds16(b + r * kBlock + 1024 + (rl * 8u + ((2u * q + uint32_t(h)) ^ (rl & 7u))) * 16u);
            }
            uint32_t e7[NRB][16];
#pragma unroll
            for (int r = 0; r < NRB; ++r) {
                const char* const l = reinterpret_cast<const char*>(lut + (PAIR ? 256 * r : 0));
#pragma unroll
                for (int p = 0; p < 16; ++p)
                    e7[r][p] = *reinterpret_cast<const uint32_t*>(l + (((nb[r][p >> 2] >> (8 * (p & 3))) & 0xFFu) << 2));
            }
            // a lane's 32 weights of a block lie in one group
#pragma unroll
            for (int r = 0; r < NRB; ++r) {
                if (v.flag[r]) {
#pragma unroll
                    for (int p = 0; p < 16; ++p) {
                        const uint32_t d = v.vx[r][p >> 3][(p & 7) >> 1];
                        e7[r][p] = (p & 1) ? exp_pair<1>(d) : exp_pair<0>(d);
                    }
                }
#pragma unroll
                for (int p = 0; p < 16; ++p) {
                    const uint32_t smw = sm[r][p >> 3][(p & 7) >> 1];
                    wf[r][p >> 2][p & 3] = (p & 1) ? join_pair<1>(smw, e7[r][p]) : join_pair<0>(smw, e7[r][p]);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < NRB; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    wf[r][i] = lds16(b + r * kBlock + (rl * 16u + ((4u * q + uint32_t(i)) ^ (rl & 7u))) * 16u);
        }
        if (zero) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int n = 0; n < NB; ++n) xf[i][n] = q > 1 ? u32x4_t{0u, 0u, 0u, 0u} : xf[i][n];
#pragma unroll
                for (int r = 0; r < NRB; ++r) wf[r][i] = q > 1 ? u32x4_t{0u, 0u, 0u, 0u} : wf[r][i];
            }
        }
#pragma unroll
        for (int r = 0; r < NRB; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wf[r][i]),
                                                                        __builtin_bit_cast(bf16x8_t, xf[i][n]),
                                                                        acc[r][n], 0, 0, 0);
        // every read of this slot has returned before it is refilled
        __builtin_amdgcn_sched_barrier(0);
    };

    set_offsets(false);
    if (s_lo < s_hi) {                                   // the first steps' weights go out before anything is waited for
        load_tables(s_lo, min(s_hi, s_lo + kSegment / kStepK));
        issue_w(s_lo, 0);
        issue_w(min(s_lo + 1u, s_hi - 1u), 1);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (PAL) {
        for (int i = tid; i < 256; i += 64 * KW)
#pragma unroll
            for (int m = 0; m < M; ++m)
                lut[256 * m + i] = (pal_byte(a.w[m].pal, uint32_t(i) & 15u) << 7) |
                                   (pal_byte(a.w[m].pal, uint32_t(i) >> 4) << 23);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    }
    // what the epilogue adds, for the wave's first output tile
    auto tile_row = [&](int i) { return row0 + 16u * uint32_t(PAIR ? 0 : i / NB) + 4u * q; };
    auto tile_b = [&](int i) { return 16u * uint32_t(i % NB) + rl; };
    EpilogueIn in{};
    if (wave < TL && tile_b(wave) < uint32_t(t.rows) && tile_row(wave) < R)
        in = epilogue_load(a.ep, t.row0 + tile_b(wave), int(tile_row(wave)), a.R);
    for (uint32_t lo = s_lo; lo < s_hi;) {
        const uint32_t hi = PAL ? min(s_hi, lo + kSegment / kStepK) : s_hi;
        // two steps in flight; steps past the segment issue its last step again,
        // so that the waits are compile-time constants
        const uint32_t last = hi - 1u;
        Verbatim v[D];
        if (lo != s_lo) {
            load_tables(lo, hi);
            issue_w(lo, 0);
            issue_w(min(lo + 1u, last), 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        issue_x(lo, 0);
        __builtin_amdgcn_sched_barrier(0);               // first of these loads: the wait counts on it
        issue_v(v[0]);
        issue_x(min(lo + 1u, last), 1);
        issue_v(v[1]);
        __builtin_amdgcn_sched_barrier(0);
        wait_vm<XQ + 2 * kV, false>();                          // step 0 of the segment is in LDS
        uint32_t s = lo;
        for (; s + D <= hi; s += D) {
#pragma unroll
            for (int j = 0; j < D; ++j) {
                wait_vm<kPer, false>();
                compute(j, v[j], false);
                issue(min(s + uint32_t(j + D), last), j, v[j]);
            }
        }
        if (s < hi) {
            wait_vm<kPer, false>();
            compute(0, v[0], false);
        }
        wait_vm<0, false>();                                    // no load lands after its slot is used again
        lo = hi;
    }
    if (C % kStepK && wave == KW - 1) {                  // 64 columns left: the upper half multiplies zeros
        Verbatim v;
        set_offsets(true);
        load_tables(steps, steps + 1);
        if (PAL && q > 1) {
#pragma unroll
            for (int r = 0; r < NRB; ++r) fl[r][0] = 0u;
        }
        issue(steps, 0, v);
        wait_vm<0, false>();
        compute(0, v, true);
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
        if (i != wave) in = epilogue_load(a.ep, t.row0 + b, int(row), a.R);
        epilogue_store(a.ep, in, t.row0 + b, int(row), a.R, y);
    }
}

template <bool PAL, bool PAIR, int XQ, int KW>
hipError_t launch_kw(const GroupArgs& a, int64_t bands, hipStream_t s) {
    const int64_t units = group_units(a, 4 * XQ, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    launch_timed(skinny_kernel<PAL, PAIR, PAIR ? 2 : 1, XQ, KW>, dim3(unsigned(units)), dim3(64 * KW), 0, s, a,
                 uint32_t(bands));
    return hipGetLastError();
}

template <bool PAL, bool PAIR, int XQ>
hipError_t launch(const GroupArgs& a, hipStream_t s) {
    const int64_t bands = (a.R + 15) / 16;
    switch (skinny_waves(PAIR, 4 * XQ, a)) {
        case 2: return launch_kw<PAL, PAIR, XQ, 2>(a, bands, s);
        case 4: return launch_kw<PAL, PAIR, XQ, 4>(a, bands, s);
        default: return launch_kw<PAL, PAIR, XQ, (PAIR || XQ > 4 ? 4 : 8)>(a, bands, s);
    }
}

template <bool PAL, bool PAIR>
hipError_t launch_xq(const GroupArgs& a, int rows, hipStream_t s) {
    if (rows <= 4) return launch<PAL, PAIR, 1>(a, s);
    return rows <= 16 ? launch<PAL, PAIR, 4>(a, s) : launch<PAL, PAIR, 8>(a, s);
}

}  // namespace

// Waves that split K: the fewest (2, 4 or 8) that give about six waves a
// compute unit; more only add to the partial sums and to what starts and ends
// together (16 rows of 14336 x 4096, palette: 22.7 us with two, 25.8 with four;
// of 4096 x 14336: 36.2, 23.6, 23.4 with two, four, eight).  The rings of eight
// fit a compute unit's LDS through 16 input rows of a single matrix.
int skinny_waves(bool pair, int rows, const GroupArgs& a) {
    const int64_t bands = (a.R + 15) / 16, most = std::max<int64_t>(a.offsets || a.E > 1 ? std::min<int64_t>(a.n, a.E) : 1, 1);
    const int64_t want = 6 * int64_t(a.cus);
    return 2 * bands * most >= want ? 2 : pair || rows > 16 || 4 * bands * most >= want ? 4 : 8;
}

hipError_t launch_skinny_rows(bool pal, bool pair, const GroupArgs& a, int rows, hipStream_t s) {
    if (pal) return pair ? launch_xq<true, true>(a, rows, s) : launch_xq<true, false>(a, rows, s);
    return pair ? launch_xq<false, true>(a, rows, s) : launch_xq<false, false>(a, rows, s);
}

}  // namespace uwk

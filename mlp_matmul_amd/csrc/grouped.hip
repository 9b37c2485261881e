// Matmul with bias, activation and residual in its epilogue, and the products
// of a mixture-of-experts layer grouped by expert: which kernel runs a shape.
//
//   y_s = act(W_e(s) x_s + b) + r_s,   h_s = SiLU(G_e(s) x_s) * (U_e(s) x_s)
//
// with fp32 sums, one rounding at the end.  Expert e's matrix is rows
// e*R .. e*R+R-1 of the stacked weights; its input rows are those between
// offsets[e] and offsets[e+1], which only the device knows: the choice goes by
// the rows an expert has on average.
#include <algorithm>

#include "grouped_common.h"
#include "kernels.h"

namespace uwk {

namespace {

// A tile shape's time for one 64-column step of its workgroups, in us on
// MI355X: `full` with every compute unit taken (8192 x 8192 x 8192: 2424, 1362,
// 984, 916 us), `one` with a workgroup here and there (64 rows of 14336 x 4096:
// 23.5, 26.7, 47.7, 79 us, less 4 us for launch and epilogue).
struct TileCost {
    int mt, nt, per_cu;
    double full, one;
};
constexpr TileCost kTiles[TILE_SHAPES] = {
    {64, 64, 2, 0.59, 0.30}, {128, 64, 2, 0.665, 0.35}, {256, 128, 1, 0.96, 0.68}, {256, 256, 1, 1.79, 1.2}};

// Time of `groups` products of `rows` input rows each with [R, C]: the rounds
// of workgroups that the chip takes, the last one by how full it is.
double tile_us(const TileCost& c, bool pair, double groups, double rows, bool exact, const GroupArgs& a) {
    const int mt = pair ? c.mt / 2 : c.mt;
    // tiles of an expert: the rows are spread, half a tile is lost on average
    const double tiles = exact ? double((int64_t(rows) + c.nt - 1) / c.nt) : std::max(1.0, rows / c.nt + 0.5);
    const double units = groups * tiles * double((a.R + mt - 1) / mt), slots = double(a.cus) * c.per_cu;
    const double rounds = double(int64_t(units / slots)), rest = units / slots - rounds;
    return (rounds * c.full + (rest > 0 ? c.one + (c.full - c.one) * rest : 0)) * double(a.C / 64) + 4;
}

TileShape best_tile(bool pair, double groups, double rows, bool exact, const GroupArgs& a, double* us = nullptr) {
    int best = 0;
    double t = 1e30;
    for (int i = 0; i < TILE_SHAPES; ++i) {
        const double v = tile_us(kTiles[i], pair, groups, rows, exact, a);
        if (v < t) {
            t = v;
            best = i;
        }
    }
    if (us) *us = t;
    return TileShape(best);
}

// ------------------------------------------------------------ direct palette to bf16
// 16 weights a lane; a lane's 16 columns lie in one 64-weight group.  Memory
// bound: 1.53 bytes read and 2 written a weight.
__global__ __launch_bounds__(256) void expand_kernel(Weight w, int64_t n, uint16_t* out) {
    __shared__ uint32_t lut[256];
    lut[threadIdx.x] = (pal_byte(w.pal, threadIdx.x & 15) << 7) | (pal_byte(w.pal, threadIdx.x >> 4) << 23);
    __syncthreads();
    const int64_t pos = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 16;
    if (pos >= n) return;
    const u32x2_t nib = load_stream8(static_cast<const uint8_t*>(w.w) + pos / 2);
    const u32x4_t sm = load_stream16(w.sm + pos);
    const int64_t g = pos >> 6;
    const uint64_t word = w.bitmap[g >> 6];
    const uint32_t bit = uint32_t(g) & 63u;
    uint32_t e7[8], v[8];
    if ((word >> bit) & 1) {
        const u32x4_t vx = load16(w.vexp + int64_t(verbatim_slot(word, bit, w.tile_vbase[g >> 6])) * 64 + (pos & 63));
#pragma unroll
        for (int p = 0; p < 8; ++p) e7[p] = (p & 1) ? exp_pair<1>(vx[p >> 1]) : exp_pair<0>(vx[p >> 1]);
    } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) e7[p] = lut[(nib[p >> 2] >> (8 * (p & 3))) & 0xFFu];
    }
#pragma unroll
    for (int p = 0; p < 8; ++p)
        v[p] = (p & 1) ? join_pair<1>(sm[p >> 1], e7[p]) : join_pair<0>(sm[p >> 1], e7[p]);
    store16(out + pos, u32x4_t{v[0], v[1], v[2], v[3]});
    store16(out + pos + 8, u32x4_t{v[4], v[5], v[6], v[7]});
}

// out = epilogue of the sum of `split` arrays [B, R], in order.
__global__ __launch_bounds__(256) void sums_epilogue_kernel(const float* sums, int split, int64_t B, int R, Epilogue ep) {
    const int64_t quads = (R + 3) / 4, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= B * quads) return;
    const int64_t b = i / quads;
    const int r = int(i % quads) * 4;
    f32x4_t v = load4(sums, VT_F32, b * R + r, r, R, (R & 3) == 0);
    for (int z = 1; z < split; ++z) v += load4(sums, VT_F32, (z * B + b) * R + r, r, R, (R & 3) == 0);
    epilogue4(ep, b, r, R, v);
}

MatArgs mat_args(const GroupArgs& a) {
    MatArgs m{};
    m.w = a.w[0].w;
    m.sm = a.w[0].sm;
    m.vexp = a.w[0].vexp;
    m.bitmap = a.w[0].bitmap;
    m.tile_vbase = a.w[0].tile_vbase;
    m.X = a.X;
    m.R = a.R;
    m.C = a.C;
    m.B = a.n;
    m.cus = a.cus;
    for (int i = 0; i < 4; ++i) m.pal[i] = a.w[0].pal[i];
    m.split_k = 1;
    return m;
}

// What a large batch of palette weights does: nothing special, K-slices of the
// tiled matmul into scratch, or the weights expanded to bf16 there.
enum PalPlan { PLAN_TILES, PLAN_SUMS, PLAN_EXPAND };

// Through 512 rows the tiled matmuls of gemm_mfma.hip and gemm_lds.hip, which
// split K, with their sums in scratch and the epilogue in the kernel that adds
// them (14336 x 4096, 64 rows: 36 us against 45 for the 64 x 64 tiles); above,
// the weights are expanded once and the bf16 tiles run at twice the rate of
// the rebuilding ones (4096 x 4096 x 2049 rows: 14 + 72 us against 156).
PalPlan pal_plan(const GroupArgs& a) {
    if (a.n > 512) return PLAN_EXPAND;
    const MatArgs m = mat_args(a);
    return mfma_supported(m) && a.n * a.C < (int64_t(1) << 31) && a.n * a.R < (int64_t(1) << 31) ? PLAN_SUMS
                                                                                                 : PLAN_TILES;
}

uint64_t plan_bytes(PalPlan p, const GroupArgs& a, int* split = nullptr) {
    if (p == PLAN_TILES) return 0;
    if (p == PLAN_EXPAND) return uint64_t(a.R) * uint64_t(a.C) * 2;
    const int k = mfma_default_split(SRC_PAL, mat_args(a), a.cus);
    if (split) *split = k;
    return uint64_t(k) * uint64_t(a.n) * uint64_t(a.R) * 4;
}

// bf16 rows above the skinny kernel's; a few rows behind the last whole tile go
// to the skinny kernel where they would start another round of tiles (2049
// rows of 4096 x 4096: 61 + 9 us against 100).
hipError_t linear_tiles(const GroupArgs& a, hipStream_t s) {
    double whole_us = 0, us = 0;
    const TileShape shape = best_tile(false, 1, double(a.n), true, a, &us);
    const int64_t tail = a.n % 128;                      // 128 and 256 both divide what is left
    if (tail && tail <= 32 && a.n > 256) {
        const TileShape part = best_tile(false, 1, double(a.n - tail), true, a, &whole_us);
        // the weights once more, at 5 TB/s, and a launch
        if (whole_us + 4 + double(a.R) * double(a.C) * 2 / 5e6 < us) {
            GroupArgs head = a, rest = a;
            head.n = head.x_rows = a.n - tail;
            rest.n = rest.x_rows = tail;
            rest.X = a.X + head.n * a.ldx;
            const int64_t ob = a.ep.out_type == VT_BF16 ? 2 : 4, rb = a.ep.residual_type == VT_BF16 ? 2 : 4;
            rest.ep.out = static_cast<uint8_t*>(a.ep.out) + head.n * a.ep.ldo * ob;
            if (a.ep.residual) rest.ep.residual = static_cast<const uint8_t*>(a.ep.residual) + head.n * a.ep.ldr * rb;
            const hipError_t e = launch_tile(false, head, part, s);
            return e == hipSuccess ? launch_linear(false, rest, nullptr, 0, s) : e;
        }
    }
    return launch_tile(false, a, shape, s);
}

}  // namespace

uint64_t linear_scratch(bool pal, int64_t rows, int64_t cols, int64_t batch, int cus) {
    if (!pal || batch <= 32 || rows == 0) return 0;
    GroupArgs a{};
    a.R = int32_t(rows);
    a.C = int32_t(cols);
    a.n = batch;
    a.cus = cus;
    return plan_bytes(pal_plan(a), a);
}

hipError_t launch_linear(bool pal, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s) {
    if (a.n <= 0 || a.R <= 0) return hipSuccess;
    if (a.n <= 2 && gemv_rows_supported(a, int(a.n))) return launch_gemv_rows(pal, false, a, int(a.n), s);
    if (a.n <= 32) return launch_skinny_rows(pal, false, a, int(a.n), s);
    if (!pal) return linear_tiles(a, s);
    PalPlan plan = pal_plan(a);
    int split = 1;
    if (plan_bytes(plan, a, &split) > scratch_bytes || (plan == PLAN_SUMS && a.ldx != a.C)) plan = PLAN_TILES;
    if (plan == PLAN_EXPAND) {
        const int64_t n = int64_t(a.R) * a.C;
        uint16_t* const w = static_cast<uint16_t*>(scratch);
        expand_kernel<<<unsigned((n / 16 + 255) / 256), 256, 0, s>>>(a.w[0], n, w);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        GroupArgs b = a;
        b.w[0] = Weight{};
        b.w[0].w = w;
        return linear_tiles(b, s);
    }
    if (plan == PLAN_SUMS) {
        MatArgs m = mat_args(a);
        m.split_k = split;
        m.Y = m.partial = static_cast<float*>(scratch);
        const hipError_t e = launch_mfma_sums(SRC_PAL, m, s);
        if (e != hipSuccess) return e;
        const int64_t quads = a.n * ((a.R + 3) / 4);
        sums_epilogue_kernel<<<unsigned((quads + 255) / 256), 256, 0, s>>>(m.partial, split, a.n, a.R, a.ep);
        return hipGetLastError();
    }
    // 64 x 64 tiles until they take four rounds (14336 x 4096, 64 rows: 45 us
    // against 68), then 128 x 128 (8192 x 8192 x 8192: 1.60 against 2.9 ms)
    const int64_t units = (a.n + 63) / 64 * ((a.R + 63) / 64);
    return launch_tile_pal(false, a, units <= 8 * int64_t(a.cus) ? PAL_TILE_64x64 : PAL_TILE_128x128, s);
}

hipError_t launch_grouped(bool pal, bool pair, const GroupArgs& a, hipStream_t s) {
    if (a.n <= 0 || a.R <= 0) return hipSuccess;
    const int64_t groups = std::min<int64_t>(a.n, a.E);
    const double rows = double(a.n) / double(groups);
    // one token's slots (each its own expert), or as few as to make equal ones
    // rare: the weight stream at its best; two rows for about two tokens' worth
    // of many experts (gate/up of 4 tokens, 16 experts: 34 us against 37-40)
    const bool single = a.order ? a.n <= a.div : 4 * a.n <= a.E || a.n == 1;
    if (single && gemv_rows_supported(a, 1)) return launch_gemv_rows(pal, pair, a, 1, s);
    if (2 * a.n <= a.E && gemv_rows_supported(a, 2)) return launch_gemv_rows(pal, pair, a, 2, s);
    // gate/up of 16 experts, 2 rows each: 4-row tiles 68 (bf16) and 74 us
    // (palette), 16-row ones 79 and 67; 4 rows each: 16-row ones 79 against 86;
    // 12 rows of 32 experts: 16-row ones 62 (bf16), 72 us (palette, 63 with tiles)
    if (rows <= (pal ? 1.5 : 2.5)) return launch_skinny_rows(pal, pair, a, 4, s);
    if (rows <= (pal ? 11 : 14)) return launch_skinny_rows(pal, pair, a, 16, s);
    if (!pal) return launch_tile(pair, a, best_tile(pair, double(groups), rows, false, a), s);
    // 25 rows of 8 experts: 128 x 64 tiles 111 us, 128 x 128 123; 64 rows: 151
    // and 122
    return launch_tile_pal(pair, a, rows <= 40 ? PAL_TILE_128x64 : PAL_TILE_128x128, s);
}

}  // namespace uwk

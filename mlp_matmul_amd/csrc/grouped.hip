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

// A tile shape's time for one 64-column step of a round of workgroups, in us on
// MI355X: with a workgroup here and there, with one on each compute unit, and
// with `per_cu` on each.
struct TileCost {
    int mt, nt, per_cu;
    double few, one, full;
};
constexpr TileCost kTiles[TILE_SHAPES] = {{64, 64, 2, 0.16, 0.265, 0.51},
                                          {128, 64, 2, 0.34, 0.45, 0.86},
                                          {256, 128, 1, 0.65, 0.96, 0.96},
                                          {256, 256, 1, 1.2, 1.7, 1.7}};
// A launch with its first loads and its stores, bytes a us from memory and the
// share of them that a second reading of the weights or the rows costs, and the
// kernel that adds slices, with the bytes a us of writing and reading them.
constexpr double kLaunchUs = 6, kBytesUs = 7.8e6, kWeightsAgain = 0.45, kRowsAgain = 0.33, kSumsUs = 2, kSumsBytesUs = 3.9e6;

struct TilePlan {
    TileShape shape;
    int split;
    double us;
};

// The tile shape and number of K-slices for `groups` products of `rows` input
// rows each with [R, C]: the choice of the least estimated time, which is the
// rounds of workgroups that the chip takes or the bytes from memory, whichever
// is longer.  The constants are fitted to the 16 choices at 32 sizes (1000 x
// 2048 to 14336 x 4096 and 4096 x 14336, 33 to 2049 rows); what it picks there is
// the fastest choice or within 8% of it.  At 4096 x 14336, us, against 64 x 64
// tiles without slices: 64 rows 31 (128 x 64, 8 slices) and 73, 256 rows 48
// (256 x 128, 8) and 72, 800 rows 106 (256 x 128, 2) and 198.
TilePlan plan_tiles(bool pair, double groups, double rows, bool exact, bool may_split, const GroupArgs& a) {
    TilePlan best{TILE_64x64, 1, 1e30};
    const double weights = groups * double(a.R) * double(a.C) * (pair ? 4 : 2);
    for (int i = 0; i < TILE_SHAPES; ++i) {
        const TileCost& c = kTiles[i];
        const int mt = pair ? c.mt / 2 : c.mt;
        const double bands = groups * double((a.R + mt - 1) / mt);
        // tiles of an expert: the rows are spread, half a tile is lost on average
        const double tiles = exact ? double((int64_t(rows) + c.nt - 1) / c.nt) : std::max(1.0, rows / c.nt + 0.5);
        const double again = kWeightsAgain * weights * (tiles - 1) + kRowsAgain * bands * rows * double(a.C) * 2;
        for (int split = 1; split <= (may_split ? 8 : 1) && split * 2 <= std::max(2, a.C / 64); split *= 2) {
            const double per = bands * tiles * split / a.cus;          // workgroups a compute unit
            const double rounds = double(int64_t(per / c.per_cu)), rest = per - rounds * c.per_cu;
            double round = rounds * c.full;
            if (rest > 1) round += c.one + (c.full - c.one) * (rest - 1);
            else if (rest > 0) round += c.few + (c.one - c.few) * rest;
            double us = kLaunchUs + std::max(round * double(a.C / 64) / split, (weights + again) / kBytesUs);
            if (split > 1) us += kSumsUs + split * rows * double(a.R) * 8 / kSumsBytesUs;
            if (us < best.us) best = {TileShape(i), split, us};
        }
    }
    return best;
}

// ------------------------------------------------------------ direct palette to bf16
// n weights of each expert (blockIdx.y) that has rows, 16 a lane; a lane's 16
// columns lie in one 64-weight group.  Memory bound: 1.53 bytes read and 2
// written a weight.
__global__ __launch_bounds__(256) void expand_kernel(Weight w, int64_t n, const int32_t* offsets, uint16_t* out) {
    __shared__ uint32_t lut[256];
    if (offsets && offsets[blockIdx.y + 1] <= offsets[blockIdx.y]) return;
    lut[threadIdx.x] = (pal_byte(w.pal, threadIdx.x & 15) << 7) | (pal_byte(w.pal, threadIdx.x >> 4) << 23);
    __syncthreads();
    const int64_t in = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 16, pos = int64_t(blockIdx.y) * n + in;
    if (in >= n) return;
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

// The experts' weights (one matrix's) as bf16 at `out`.
uint64_t expanded_bytes(const GroupArgs& a) {
    return (uint64_t(a.E) * uint64_t(a.R) * uint64_t(a.C) * 2 + 255) & ~uint64_t(255);
}

hipError_t expand(const GroupArgs& a, Weight* w, uint16_t* out, hipStream_t s) {
    const int64_t n = int64_t(a.R) * a.C;
    expand_kernel<<<dim3(unsigned((n / 16 + 255) / 256), unsigned(a.E)), 256, 0, s>>>(*w, n, a.offsets, out);
    *w = Weight{};
    w->w = out;
    return hipGetLastError();
}

// What a large batch of palette weights does: nothing special, K-slices of the
// tiled matmul into scratch, or the weights expanded to bf16 there.
enum PalPlan { PLAN_TILES, PLAN_SUMS, PLAN_EXPAND };

// Through 512 rows the tiled matmul of gemm_lds.hip, which splits K, with its
// sums in scratch and the epilogue in the kernel that adds them (14336 x 4096,
// 64 rows: 33 us against 45 for the 64 x 64 tiles); above, the weights are
// expanded once and the bf16 tiles run at twice the rate of the rebuilding ones
// (4096 x 4096 x 2049 rows: 14 + 72 us against 156; at 400 rows of 4096 x 14336
// expanding costs 46 us of 112, the sums take 90).
PalPlan pal_plan(const GroupArgs& a) {
    if (a.n > 512) return PLAN_EXPAND;
    const MatArgs m = mat_args(a);
    return lds_gemm_supported(SRC_PAL, m) && a.n * a.C < (int64_t(1) << 31) && a.n * a.R < (int64_t(1) << 31) ? PLAN_SUMS
                                                                                                 : PLAN_TILES;
}

// Whether n rows are left to the skinny kernel: through 16, and through 32 on
// matrices below 2^25 weights (24 rows of 4096 x 4096: 10 us against 13; of
// 14336 x 4096: 34 against 29, palette 40 against 33).
bool few_rows(const GroupArgs& a) { return a.n <= 16 || (a.n <= 32 && int64_t(a.R) * a.C < (int64_t(1) << 25)); }

uint64_t sums_bytes(const GroupArgs& a, int split) { return uint64_t(split) * uint64_t(a.n) * uint64_t(a.R) * 4; }

hipError_t add_sums(const GroupArgs& a, const float* sums, int split, hipStream_t s) {
    const int64_t quads = a.n * ((a.R + 3) / 4);
    sums_epilogue_kernel<<<unsigned((quads + 255) / 256), 256, 0, s>>>(sums, split, a.n, a.R, a.ep);
    return hipGetLastError();
}

// bf16 tiles.  A few rows behind the last whole tile go to the skinny kernel
// where they would start another round of tiles (2049 rows of 4096 x 4096: 61 +
// 9 us against 95).
hipError_t linear_tiles(const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s) {
    TilePlan plan = plan_tiles(false, 1, double(a.n), true, true, a);
    if (plan.split > 1 && sums_bytes(a, plan.split) > scratch_bytes) plan = plan_tiles(false, 1, double(a.n), true, false, a);
    const int64_t tail = a.n % 128;                      // 128 and 256 both divide what is left
    if (tail && tail <= 32 && a.n > 256) {
        const TilePlan part = plan_tiles(false, 1, double(a.n - tail), true, false, a);
        // the weights once more, and a launch
        if (part.us + kLaunchUs + double(a.R) * double(a.C) * 2 / kBytesUs < plan.us) {
            GroupArgs head = a, rest = a;
            head.n = head.x_rows = a.n - tail;
            rest.n = rest.x_rows = tail;
            rest.X = a.X + head.n * a.ldx;
            const int64_t ob = a.ep.out_type == VT_BF16 ? 2 : 4, rb = a.ep.residual_type == VT_BF16 ? 2 : 4;
            rest.ep.out = static_cast<uint8_t*>(a.ep.out) + head.n * a.ep.ldo * ob;
            if (a.ep.residual) rest.ep.residual = static_cast<const uint8_t*>(a.ep.residual) + head.n * a.ep.ldr * rb;
            const hipError_t e = launch_tile(false, head, part.shape, s);
            if (e != hipSuccess) return e;
            if (tail <= 2 && gemv_rows_supported(rest, int(tail))) return launch_gemv_rows(false, false, rest, int(tail), s);
            return launch_skinny_rows(false, false, rest, int(tail), s);
        }
    }
    GroupArgs b = a;
    b.split = plan.split;
    b.sums = static_cast<float*>(scratch);
    const hipError_t e = launch_tile(false, b, plan.shape, s);
    return e != hipSuccess || plan.split == 1 ? e : add_sums(a, b.sums, plan.split, s);
}

// Whether palette weights of experts with so many rows on average are expanded
// (512 is where it pays):
// with 530 rows of 4 experts' 4096 x 4096 138 us against 169 rebuilding tile by
// tile, gate/up of 8 experts' 1024 x 2048 96 against 96; with 2000 rows 335
// against 484 and 201 against 276.
bool expand_groups(const GroupArgs& a) { return a.n > 512 * std::min<int64_t>(a.n, a.E); }

}  // namespace

uint64_t linear_scratch(bool pal, int64_t rows, int64_t cols, int64_t batch, int cus) {
    GroupArgs a{};
    a.R = int32_t(rows);
    a.C = int32_t(cols);
    a.n = batch;
    a.E = 1;
    a.cus = cus;
    if (rows == 0 || few_rows(a)) return 0;
    const PalPlan p = pal ? pal_plan(a) : PLAN_TILES;
    if (p == PLAN_SUMS) return sums_bytes(a, lds_gemm_default_split(SRC_PAL, mat_args(a), cus));
    if (pal && p == PLAN_TILES) return 0;
    const TilePlan t = plan_tiles(false, 1, double(a.n), true, true, a);
    return (p == PLAN_EXPAND ? expanded_bytes(a) : 0) + (t.split > 1 ? sums_bytes(a, t.split) : 0);
}

hipError_t launch_linear(bool pal, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s) {
    if (a.n <= 0 || a.R <= 0) return hipSuccess;
    if (a.n <= 2 && gemv_rows_supported(a, int(a.n))) return launch_gemv_rows(pal, false, a, int(a.n), s);
    if (few_rows(a)) return launch_skinny_rows(pal, false, a, int(a.n), s);
    if (!pal) return linear_tiles(a, scratch, scratch_bytes, s);
    const PalPlan plan = pal_plan(a);
    if (plan == PLAN_EXPAND && scratch_bytes >= expanded_bytes(a)) {
        GroupArgs b = a;
        const hipError_t e = expand(a, &b.w[0], static_cast<uint16_t*>(scratch), s);
        if (e != hipSuccess) return e;
        return linear_tiles(b, static_cast<uint8_t*>(scratch) + expanded_bytes(a), scratch_bytes - expanded_bytes(a), s);
    }
    if (plan == PLAN_SUMS && a.ldx == a.C) {
        MatArgs m = mat_args(a);
        m.split_k = lds_gemm_default_split(SRC_PAL, m, a.cus);
        if (sums_bytes(a, m.split_k) <= scratch_bytes) {
            m.Y = m.partial = static_cast<float*>(scratch);
            const hipError_t e = launch_lds_gemm(SRC_PAL, m, s);
            return e == hipSuccess ? add_sums(a, m.partial, m.split_k, s) : e;
        }
    }
    // 64 x 64 tiles until they take four rounds (14336 x 4096, 64 rows: 45 us
    // against 68), then 128 x 128 (8192 x 8192 x 8192: 1.60 against 2.9 ms)
    const int64_t units = (a.n + 63) / 64 * ((a.R + 63) / 64);
    return launch_tile_pal(false, a, units <= 8 * int64_t(a.cus) ? PAL_TILE_64x64 : PAL_TILE_128x128, s);
}

uint64_t grouped_scratch(bool pal, bool pair, int experts, int64_t rows, int64_t cols, int64_t n) {
    GroupArgs a{};
    a.R = int32_t(rows);
    a.C = int32_t(cols);
    a.E = experts;
    a.n = n;
    return pal && rows && n && expand_groups(a) ? expanded_bytes(a) * (pair ? 2 : 1) : 0;
}

hipError_t launch_grouped(bool pal, bool pair, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s) {
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
    if (!pal) return launch_tile(pair, a, plan_tiles(pair, double(groups), rows, false, false, a).shape, s);
    if (expand_groups(a) && scratch_bytes >= expanded_bytes(a) * (pair ? 2 : 1)) {
        GroupArgs b = a;
        for (int m = 0; m < (pair ? 2 : 1); ++m) {
            const hipError_t e = expand(a, &b.w[m], static_cast<uint16_t*>(scratch) + uint64_t(m) * (expanded_bytes(a) / 2), s);
            if (e != hipSuccess) return e;
        }
        return launch_tile(pair, b, plan_tiles(pair, double(groups), rows, false, false, b).shape, s);
    }
    // 25 rows of 8 experts: 128 x 64 tiles 111 us, 128 x 128 123; 64 rows: 151
    // and 122
    return launch_tile_pal(pair, a, rows <= 40 ? PAL_TILE_128x64 : PAL_TILE_128x128, s);
}

}  // namespace uwk

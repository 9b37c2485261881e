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
    f32x4_t v = load4(sums, VT_F32, b * R + r, r, R);
    for (int z = 1; z < split; ++z) v += load4(sums, VT_F32, (z * B + b) * R + r, r, R);
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

uint64_t sums_bytes(const GroupArgs& a, int split) { return uint64_t(split) * uint64_t(a.n) * uint64_t(a.R) * 4; }

hipError_t add_sums(const GroupArgs& a, const float* sums, int split, hipStream_t s) {
    const int64_t quads = a.n * ((a.R + 3) / 4);
    sums_epilogue_kernel<<<unsigned((quads + 255) / 256), 256, 0, s>>>(sums, split, a.n, a.R, a.ep);
    return hipGetLastError();
}

// ------------------------------------------------------------ which kernel
// The choice goes by estimated times.  The constants below are fitted to 746
// sizes of both weight forms (one matrix of 64 x 64 to 16000 x 14000 with 3 to
// 2500 rows, the pair and the single product of 2 to 64 experts with 3 to 900
// rows each, even and skewed), each timed on MI355X with every kernel; what the
// estimates choose there takes 1.02 to 1.04 times the fastest kernel's time in
// the geometric mean, by kind of product, and 1.7 times at worst.  Thresholds
// on the rows alone took 1.05 to 1.21 times.  A constant of 0 is a term that those
// sizes did not tell from its neighbours.

// Times in us: a 64-column step of a round of workgroups with one here and
// there, with one on each compute unit, with `per_cu` on each; the launch, and
// what a round needs before its first step and behind its last, in steps.  Bytes a us
// of the weight stream where that takes longer, and the share of it that a
// further tile of rows costs: tiles of one band run side by side and find part
// of its weights in a cache.
struct TileCost {
    int mt, nt, per_cu;
    double few, one, full, launch, around, stream, again;
};
constexpr TileCost kTiles[TILE_SHAPES] = {{64, 64, 2, 0.18, 0.28, 0.45, 4.7, 7.2, 4.8e6, 0.53},
                                          {128, 64, 2, 0.30, 0.48, 0.69, 4.6, 6.1, 5.0e6, 0.43},
                                          {256, 128, 1, 0.62, 0.93, 0.93, 4.9, 7.6, 4.8e6, 0.35},
                                          {256, 256, 1, 1.1, 1.5, 1.5, 5.8, 6.9, 5.7e6, 1.1}};
constexpr TileCost kPalTiles[PAL_TILE_SHAPES] = {{64, 64, 3, 0.52, 0.62, 0.97, 4.6, 5.3, 3.3e6, 0.73},
                                                 {128, 64, 2, 0.71, 0.90, 1.1, 3.1, 6.8, 3.1e6, 0.64},
                                                 {128, 128, 2, 0.93, 1.1, 1.7, 6.1, 3.2, 2.9e6, 0.80}};
constexpr double kFillUnits = 1.5;             // the stream is at its full rate from 1 / 1.5 workgroups a compute unit on
// The skinny kernel: a wave's step of 128 columns with few waves and with the
// chip full of them; the rest as above, in us.
struct SkinnyCost {
    double few, full, launch, around, stream, again;
};
constexpr int kSkinnyRows[3] = {4, 16, 32};
constexpr SkinnyCost kSkinny[2][2][3] = {      // palette, pair, rows
    {{{0.30, 0.30, 4.9, 0, 5.5e6, 0.34}, {0.43, 1.0, 3.8, 1.5, 4.3e6, 0}, {0.33, 0.80, 3.3, 2.1, 3.5e6, 0.40}},
     {{0, 1.2, 3.4, 2.9, 5.6e6, 0}, {0, 0.85, 4.6, 2.9, 5.0e6, 0.36}, {0, 1.0, 3.9, 4.6, 5.6e6, 0.24}}},
    {{{0.52, 2.2, 4.2, 2.1, 5.3e6, 0.14}, {0.66, 1.2, 3.8, 2.9, 3.9e6, 0.62}, {0.59, 1.0, 3.2, 3.4, 2.4e6, 0.30}},
     {{0.37, 1.7, 3.2, 5.2, 3.8e6, 0.20}, {0.52, 1.2, 4.6, 4.1, 3.1e6, 0.34}, {0.29, 1.5, 7.4, 3.9, 3.0e6, 0.32}}}};
// The tiled matmul of gemm_lds.hip into scratch: a step by its tiles' rows.
constexpr double kSums[3] = {0.64, 1.1, 1.9}, kSumsLaunch = 6.4, kSumsAround = 2.9, kSumsStream = 5.5e6;
// What expanding one matrix or a pair adds, and the bytes a us; the launch that
// adds slices, and the bytes a us of writing and reading them.
constexpr double kExpandLaunch[2] = {4.6, 6.3}, kExpandStream = 6.4e6, kAddLaunch = 3.1, kSliceStream = 7e6;

struct Choice {
    enum Kernel { SKINNY, TILE, PAL_TILE, SUMS, EXPAND } kernel;
    int shape, split;
    double us;
};

struct Problem {
    bool pal, pair, exact;       // exact: one group, `rows` is no average
    double groups, rows;
    const GroupArgs& a;

    double weights() const { return groups * double(a.R) * double(a.C) * (pair ? 2 : 1); }
    // tiles of a group: with rows spread over the groups half a tile is lost on average
    double tiles(int nt) const { return exact ? double((a.n + nt - 1) / nt) : std::max(1.0, rows / nt + 0.5); }
};

double slices_us(const GroupArgs& a, int split) { return split * double(a.n) * double(a.R) * 8 / kSliceStream; }

double tile_us(const Problem& p, const TileCost& c, bool pal, int split) {
    const int mt = p.pair ? c.mt / 2 : c.mt;
    const double tiles = p.tiles(c.nt), bands = p.groups * double((p.a.R + mt - 1) / mt);
    const double per = bands * tiles * split / p.a.cus;                // workgroups a compute unit
    const double rounds = double(int64_t(per / c.per_cu)), rest = per - rounds * c.per_cu;
    double step = rounds * c.full;
    if (rest > 1) step += c.one + (c.full - c.one) * (rest - 1) / (c.per_cu - 1);
    else if (rest > 0) step += c.few + (c.one - c.few) * rest;
    const double stream = p.weights() * (pal ? 1.53 : 2) * (1 + c.again * (tiles - 1)) / c.stream /
                          std::min(1.0, per * kFillUnits);
    const double us = c.launch + std::max(step * (double(p.a.C / 64) / split + c.around), stream);
    return split > 1 ? us + kAddLaunch + slices_us(p.a, split) : us;
}

double skinny_us(const Problem& p, int i) {
    const SkinnyCost& c = kSkinny[p.pal][p.pair][i];
    const int rows = kSkinnyRows[i], kw = skinny_waves(p.pair, rows, p.a);
    const int slot = (p.pal ? 3 : 4) * (p.pair ? 2 : 1) + rows / 4;    // KB of a wave's step; two of them, 160 KB in all
    const int per_cu = std::min(160 / (2 * kw * slot + 2), 32 / kw);
    const double tiles = p.tiles(rows), units = p.groups * double((p.a.R + 15) / 16) * tiles;
    const double rounds = units / p.a.cus / per_cu, steps = std::max(1.0, double(p.a.C / 64) / 2 / kw);
    const double step = c.few + (c.full - c.few) * std::min(1.0, rounds);
    return c.launch + std::max(std::max(1.0, rounds) * (steps * step + c.around),
                               p.weights() * (p.pal ? 1.53 : 2) * (1 + c.again * (tiles - 1)) / c.stream);
}

// The tiled matmul of gemm_lds.hip, with its sums in scratch.
bool sums_supported(const GroupArgs& a) {
    return a.ldx == a.C && lds_gemm_supported(SRC_PAL, mat_args(a)) && a.n * a.C < (int64_t(1) << 31) &&
           a.n * a.R < (int64_t(1) << 31);
}

int sums_split(const GroupArgs& a) { return lds_gemm_default_split(SRC_PAL, mat_args(a), a.cus); }

double sums_us(const Problem& p) {
    const int i = p.a.n <= 64 ? 0 : p.a.n <= 128 || p.a.R >= 8192 ? 1 : 2, nt = 64 << i, split = sums_split(p.a);
    const int64_t per = (int64_t((p.a.R + 127) / 128) * ((p.a.n + nt - 1) / nt) * split + p.a.cus - 1) / p.a.cus;
    return kSumsLaunch + std::max(double(per) * (kSums[i] * double(p.a.C / 64) / split + kSumsAround),
                                  p.weights() * 1.53 / kSumsStream) +
           slices_us(p.a, split);
}

// What a choice takes of the scratch.
uint64_t choice_bytes(const Choice& c, bool pair, const GroupArgs& a) {
    return (c.kernel == Choice::EXPAND ? expanded_bytes(a) * (pair ? 2 : 1) : 0) +
           (c.kernel == Choice::SUMS || c.split > 1 ? sums_bytes(a, c.split) : 0);
}

// The fastest choice that the scratch allows.
Choice choose(const Problem& p, uint64_t scratch_bytes) {
    Choice best{Choice::SKINNY, 16, 1, 1e30};
    auto offer = [&](Choice c) {
        if (c.us < best.us && choice_bytes(c, p.pair, p.a) <= scratch_bytes) best = c;
    };
    for (int i = 0; i < 3; ++i) offer({Choice::SKINNY, kSkinnyRows[i], 1, skinny_us(p, i)});
    for (int i = 0; i < (p.pair ? TILE_256x256 : TILE_SHAPES); ++i)
        for (int split = 1; split <= (p.exact ? 8 : 1) && (split == 1 || split * 2 <= p.a.C / 64); split *= 2) {
            const double us = tile_us(p, kTiles[i], false, split);
            if (!p.pal) offer({Choice::TILE, i, split, us});
            else offer({Choice::EXPAND, i, split, us + kExpandLaunch[p.pair] + p.weights() * 3.53 / kExpandStream});
        }
    if (p.pal)
        for (int i = 0; i < PAL_TILE_SHAPES; ++i) offer({Choice::PAL_TILE, i, 1, tile_us(p, kPalTiles[i], true, 1)});
    if (p.pal && p.exact && sums_supported(p.a)) offer({Choice::SUMS, 0, sums_split(p.a), sums_us(p)});
    return best;
}

// bf16 tiles of one matrix.  A few rows behind the last whole tile go to the
// skinny kernel where they would start another round of tiles (2049 rows of
// 4096 x 4096: 69 + 8 us against 95).
hipError_t linear_tiles(const GroupArgs& a, const Choice& c, void* sums, hipStream_t s) {
    const int64_t tail = a.n % 128;                      // 128 and 256 both divide what is left
    if (tail && tail <= 32 && a.n > 256) {
        GroupArgs head = a, rest = a;
        head.n = head.x_rows = a.n - tail;
        rest.n = rest.x_rows = tail;
        const Problem ph{false, false, true, 1, double(head.n), head}, pr{false, false, true, 1, double(tail), rest};
        const Choice part = choose(ph, 0), last = choose(pr, 0);
        const bool gemv = tail <= 2 && gemv_rows_supported(rest, int(tail));
        const double whole = tile_us({false, false, true, 1, double(a.n), a}, kTiles[c.shape], false, c.split);
        if (part.kernel == Choice::TILE && last.kernel == Choice::SKINNY && part.us + last.us < whole) {
            rest.X = a.X + head.n * a.ldx;
            const int64_t ob = a.ep.out_type == VT_BF16 ? 2 : 4, rb = a.ep.residual_type == VT_BF16 ? 2 : 4;
            rest.ep.out = static_cast<uint8_t*>(a.ep.out) + head.n * a.ep.ldo * ob;
            if (a.ep.residual) rest.ep.residual = static_cast<const uint8_t*>(a.ep.residual) + head.n * a.ep.ldr * rb;
            const hipError_t e = launch_tile(false, head, TileShape(part.shape), s);
            if (e != hipSuccess) return e;
            return gemv ? launch_gemv_rows(false, false, rest, int(tail), s) : launch_skinny_rows(false, false, rest, last.shape, s);
        }
    }
    GroupArgs b = a;
    b.split = c.split;
    b.sums = static_cast<float*>(sums);
    const hipError_t e = launch_tile(false, b, TileShape(c.shape), s);
    return e != hipSuccess || c.split == 1 ? e : add_sums(a, b.sums, c.split, s);
}

Problem linear_problem(bool pal, const GroupArgs& a) { return {pal, false, true, 1, double(a.n), a}; }

Problem grouped_problem(bool pal, bool pair, const GroupArgs& a) {
    const double groups = double(std::min<int64_t>(a.n, a.E));
    return {pal, pair, false, groups, double(a.n) / groups, a};
}

// Sizes alone, for the scratch that they ask for.
GroupArgs size_args(int experts, int64_t rows, int64_t cols, int64_t n, int cus) {
    GroupArgs a{};
    a.E = experts;
    a.R = int32_t(rows);
    a.C = int32_t(cols);
    a.ldx = cols;
    a.n = n;
    a.cus = cus;
    return a;
}

}  // namespace

uint64_t linear_scratch(bool pal, int64_t rows, int64_t cols, int64_t batch, int cus) {
    const GroupArgs a = size_args(1, rows, cols, batch, cus);
    if (rows == 0 || batch <= 2) return 0;
    return choice_bytes(choose(linear_problem(pal, a), UINT64_MAX), false, a);
}

hipError_t launch_linear(bool pal, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s) {
    if (a.n <= 0 || a.R <= 0) return hipSuccess;
    if (a.n <= 2 && gemv_rows_supported(a, int(a.n))) return launch_gemv_rows(pal, false, a, int(a.n), s);
    const Choice c = choose(linear_problem(pal, a), scratch_bytes);
    switch (c.kernel) {
        case Choice::SKINNY: return launch_skinny_rows(pal, false, a, c.shape, s);
        case Choice::TILE: return linear_tiles(a, c, scratch, s);
        case Choice::PAL_TILE: return launch_tile_pal(false, a, PalTileShape(c.shape), s);
        case Choice::SUMS: {
            MatArgs m = mat_args(a);
            m.split_k = c.split;
            m.Y = m.partial = static_cast<float*>(scratch);
            const hipError_t e = launch_lds_gemm(SRC_PAL, m, s);
            return e == hipSuccess ? add_sums(a, m.partial, c.split, s) : e;
        }
        default: {
            GroupArgs b = a;
            const hipError_t e = expand(a, &b.w[0], static_cast<uint16_t*>(scratch), s);
            return e == hipSuccess ? linear_tiles(b, c, static_cast<uint8_t*>(scratch) + expanded_bytes(a), s) : e;
        }
    }
}

uint64_t grouped_scratch(bool pal, bool pair, int experts, int64_t rows, int64_t cols, int64_t n, int cus) {
    const GroupArgs a = size_args(experts, rows, cols, n, cus);
    return pal && rows && n ? choice_bytes(choose(grouped_problem(pal, pair, a), UINT64_MAX), pair, a) : 0;
}

hipError_t launch_grouped(bool pal, bool pair, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s) {
    if (a.n <= 0 || a.R <= 0) return hipSuccess;
    // one token's slots (each its own expert), or as few as to make equal ones
    // rare: the weight stream at its best; two rows for about two tokens' worth
    // of many experts (gate/up of 4 tokens, 16 experts: 34 us against 37-40)
    const bool single = a.order ? a.n <= a.div : 4 * a.n <= a.E || a.n == 1;
    if (single && gemv_rows_supported(a, 1)) return launch_gemv_rows(pal, pair, a, 1, s);
    if (2 * a.n <= a.E && gemv_rows_supported(a, 2)) return launch_gemv_rows(pal, pair, a, 2, s);
    const Choice c = choose(grouped_problem(pal, pair, a), scratch_bytes);
    switch (c.kernel) {
        case Choice::SKINNY: return launch_skinny_rows(pal, pair, a, c.shape, s);
        case Choice::PAL_TILE: return launch_tile_pal(pair, a, PalTileShape(c.shape), s);
        case Choice::TILE: return launch_tile(pair, a, TileShape(c.shape), s);
        default: {                                       // expanded
            GroupArgs b = a;
            for (int m = 0; m < (pair ? 2 : 1); ++m) {
                uint16_t* const out = static_cast<uint16_t*>(scratch) + uint64_t(m) * (expanded_bytes(a) / 2);
                const hipError_t e = expand(a, &b.w[m], out, s);
                if (e != hipSuccess) return e;
            }
            return launch_tile(pair, b, TileShape(c.shape), s);
        }
    }
}

}  // namespace uwk

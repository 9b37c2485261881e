// Products with microscaled 4-bit weights, alone or grouped by expert: which
// kernel runs a shape.
//
//   y_s = act(W_e(s) x_s + b) + r_s,   h_s = SiLU(G_e(s) x_s) * (U_e(s) x_s)
//
// with fp32 sums, one rounding at the end.  A weight is 2^(s-127) c with c of
// two significant bits: a product with a bf16 number is exact in fp32, as it is
// with another 4-bit one.
#include <algorithm>
#include <cmath>

#include "mx4.h"

namespace uwk {

namespace {

// The choice goes by estimated times, in us.  The constants are fitted to 1121
// sizes (one matrix of 64 x 256 to 16000 x 14336 with 1 to 9000 rows, the pair
// and the single product of 2 to 64 experts), each timed on MI355X with every
// kernel, so that the sum of the squared logarithms of estimate over time is least;
// what the estimates chose there took 1.01 times the fastest kernel's time in the
// geometric mean and 1.34 times at worst.  At 600 other sizes, drawn alike and with
// the kernels as they are, it takes 1.034 times in the geometric mean (1.10 at the
// 90th percentile, where two runs differ by 5 %).  The estimates are furthest
// off for thousands of rows with a matrix of under 200 (5457 bf16 rows of 144 x
// 1216: 26 us, 13 on 64x64 tiles) and, elsewhere, for 840 rows of pairs of five
// experts of 3232 x 3840 (106 us, 67 on 128x64 tiles).
//
// Tiles: a step of a round of workgroups with one here and there, with one on
// each compute unit, with `per_cu` on each; the launch, and what a round needs
// before its first step and behind its last, in steps, and for columns behind the
// last whole step.
struct TileCost {
    int mt, nt, per_cu;
    double few, one, full, launch, around, tail;
};
constexpr TileCost kTiles[2][MX4_TILE_SHAPES] = {      // bf16 rows, 4-bit rows
    {{64, 64, 2, 0.27, 0.48, 0.60, 4.8, 6.1, 2.5},
     {128, 64, 2, 0.35, 0.70, 0.99, 5.7, 4.1, 2.0},
     {256, 128, 1, 1.34, 1.62, 1.52, 5.6, 5.5, 1.5}},
    {{64, 64, 4, 0.30, 0.55, 1.01, 5.0, 3.3, 1.1},
     {128, 128, 2, 0.69, 1.08, 1.24, 5.4, 4.9, 0.8},
     {256, 256, 1, 1.25, 1.72, 1.68, 7.8, 8.0, 3.6}}};
constexpr int kStepCols[2] = {128, 256};
// The skinny kernel: a wave's step of 128 columns with few waves and with the
// chip full of them; the launch, and what a workgroup needs around its steps.
struct SkinnyCost {
    double few, full, launch, around;
};
constexpr int kSkinnyRows[3] = {4, 16, 32};
constexpr SkinnyCost kSkinny[2][2][3] = {              // 4-bit rows, pair, rows
    {{{0.060, 1.05, 2.5, 2.7}, {0.17, 0.82, 2.9, 2.4}, {0.20, 0.86, 3.3, 2.5}},
     {{0.21, 1.27, 3.1, 2.4}, {0.10, 0.81, 3.3, 3.4}, {0.09, 0.68, 3.6, 4.1}}},
    {{{}, {0.044, 0.92, 3.2, 1.9}, {0.054, 0.84, 3.1, 2.0}}, {{}, {0.15, 1.08, 4.5, 1.4}, {0.05, 0.84, 4.0, 2.6}}}};
// Bytes a us of the weights, and the share of them that a further tile of rows reads again: tiles of one band run side
// by side and find part of them in a cache.
constexpr double kStream = 5e6, kAgain = 0.3;

struct Problem {
    bool x4, pair, exact;        // exact: one group, `rows` is no average
    double groups, rows;
    const Mx4Args& a;

    // tiles of a group: with rows spread over the groups half a tile is lost on average
    double tiles(int nt) const { return exact ? double((a.g.n + nt - 1) / nt) : std::max(1.0, rows / nt + 0.5); }
    double stream_us(double t) const {
        return groups * double(a.g.R) * double(a.g.C) * (pair ? 2 : 1) * 0.53125 * (1 + kAgain * (t - 1)) / kStream;
    }
};

double tile_us(const Problem& p, int i) {
    const TileCost& c = kTiles[p.x4][i];
    const int mt = p.pair ? c.mt / 2 : c.mt;
    const double tiles = p.tiles(c.nt), per = p.groups * double((p.a.g.R + mt - 1) / mt) * tiles / p.a.g.cus;
    const double rounds = double(int64_t(per / c.per_cu)), rest = per - rounds * c.per_cu;
    double step = rounds * c.full;
    if (rest > 1) step += c.one + (c.full - c.one) * (rest - 1) / (c.per_cu - 1);
    else if (rest > 0) step += c.few + (c.one - c.few) * rest;
    const double around = c.around + (p.a.g.C % kStepCols[p.x4] ? c.tail : 0);
    return c.launch + std::max(step * (double(p.a.g.C) / kStepCols[p.x4] + around), p.stream_us(tiles) / std::min(1.0, per * 1.5));
}

double skinny_us(const Problem& p, int i) {
    const SkinnyCost& c = kSkinny[p.x4][p.pair][i];
    const int rows = kSkinnyRows[i], kw = mx4_skinny_waves(rows, p.a);
    const int per_cu = std::max(1, std::min(160 / mx4_skinny_lds(p.x4, p.pair, rows, kw), 32 / kw));
    const double tiles = p.tiles(rows), rounds = p.groups * double((p.a.g.R + 15) / 16) * tiles / p.a.g.cus / per_cu;
    const double step = c.few + (c.full - c.few) * std::min(1.0, rounds);
    return c.launch + std::max(std::max(1.0, rounds) * (std::max(1.0, double(p.a.g.C) / 128 / kw) * step + c.around), p.stream_us(tiles));
}

struct Choice {
    bool skinny;
    int i;
    double us;
};

Choice choose(const Problem& p) {
    Choice best{true, 1, 1e30};
    auto offer = [&](Choice c) {
        if (c.us < best.us) best = c;
    };
    for (int i = p.x4 ? 1 : 0; i < 3; ++i) offer({true, i, skinny_us(p, i)});
    for (int i = 0; i < MX4_TILE_SHAPES; ++i) offer({false, i, tile_us(p, i)});
    return best;
}

hipError_t run(bool x4, bool pair, const Mx4Args& a, const Choice& c, hipStream_t s) {
    return c.skinny ? launch_mx4_skinny(x4, pair, a, kSkinnyRows[c.i], s) : launch_mx4_tile(x4, pair, a, Mx4TileShape(c.i), s);
}

}  // namespace

hipError_t launch_mx4(bool x4, bool pair, const Mx4Args& a, hipStream_t s) {
    if (a.g.n <= 0 || a.g.R <= 0) return hipSuccess;
    const bool exact = !a.g.offsets;
    const double groups = exact ? 1 : double(std::min<int64_t>(a.g.n, a.g.E));
    const Choice c = choose({x4, pair, exact, groups, double(a.g.n) / groups, a});
    if (!exact || c.skinny) return run(x4, pair, a, c, s);
    // A few rows behind the last whole tile go to the skinny kernel where another
    // round of tiles would take longer (4097 4-bit rows with 4096 x 4096 take 48 us
    // so, 65 on 128x128 tiles; 8193 with 8192 x 8192 299, 336 on 256x256 ones).
    const int64_t tail = a.g.n % kTiles[x4][c.i].nt;
    if (tail == 0 || tail > 32 || tail == a.g.n) return run(x4, pair, a, c, s);
    Mx4Args head = a, rest = a;
    head.g.n = head.g.x_rows = a.g.n - tail;
    rest.g.n = rest.g.x_rows = tail;
    const Choice ch = choose({x4, pair, true, 1, double(head.g.n), head}), cr = choose({x4, pair, true, 1, double(tail), rest});
    if (ch.us + cr.us >= c.us) return run(x4, pair, a, c, s);
    if (x4) {
        rest.x.codes += head.g.n * a.x.ldc;
        rest.x.scales += head.g.n * a.x.lds;
    } else {
        rest.g.X += head.g.n * a.g.ldx;
    }
    const int64_t ob = a.g.ep.out_type == VT_BF16 ? 2 : 4, rb = a.g.ep.residual_type == VT_BF16 ? 2 : 4;
    rest.g.ep.out = static_cast<uint8_t*>(a.g.ep.out) + head.g.n * a.g.ep.ldo * ob;
    if (a.g.ep.residual) rest.g.ep.residual = static_cast<const uint8_t*>(a.g.ep.residual) + head.g.n * a.g.ep.ldr * rb;
    const hipError_t e = run(x4, pair, head, ch, s);
    return e == hipSuccess ? run(x4, pair, rest, cr, s) : e;
}

}  // namespace uwk

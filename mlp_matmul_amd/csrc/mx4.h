// Argument blocks and launchers of the microscaled 4-bit operators.
//
// The format: the 32 numbers of columns 32b .. 32b+31 of a row share the power
// of two 2^(s - 127), s an unsigned byte (255: no number), each is one of
// +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it, held in four bits, sign first; the
// even column's lie in the low half of their byte.
#pragma once

#include "experts.h"

namespace uwk {

constexpr int kMx4Block = 32;        // numbers that share a scale

struct Mx4Mat {
    const uint8_t* codes;       // rows of C/2 bytes, ldc apart
    const uint8_t* scales;      // rows of C/32 bytes, lds apart
    int64_t ldc, lds;           // multiples of 16
};

// One matmul (or the gate/up pair) with 4-bit weights over rows grouped by
// expert.  g.w is not read; the rows of X are bf16 (g.X, g.ldx) or 4-bit (x).
struct Mx4Args {
    GroupArgs g;
    Mx4Mat w[2];                // [1]: up of the pair
    Mx4Mat x;
};

hipError_t launch_mx4_quantize(const void* X, int type, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes,
                               int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s);
hipError_t launch_mx4_dequantize(const Mx4Mat& m, int64_t rows, int64_t cols, void* out, int type, int64_t ldo,
                                 hipStream_t s);

// The product of any shape (x4: the rows of X are 4-bit too).
hipError_t launch_mx4(bool x4, bool pair, const Mx4Args& a, hipStream_t s);

// A single token's down projection with the sum over its experts.
struct Mx4OneArgs {
    Mx4Mat w;                   // [E*R, C]
    const uint16_t* h;          // top_k rows of C, ldh apart
    int64_t ldh;
    const int32_t* offsets;
    const int32_t* place;
    const float* weights;
    int32_t E, top_k, R, C;
    Epilogue ep;
};
bool mx4_one_supported(const Mx4OneArgs& a);                  // and faster
hipError_t launch_mx4_one(const Mx4OneArgs& a, hipStream_t s);

// The kernels behind it.  Up to `rows` (4, 16 or 32; 16 or 32 4-bit ones) rows an expert before its weights are read
// again.
hipError_t launch_mx4_skinny(bool x4, bool pair, const Mx4Args& a, int rows, hipStream_t s);
int mx4_skinny_waves(int rows, const Mx4Args& a);             // of its workgroups
// Steps of a wave on their way: four where LDS has room (one row with 4096 x 14336 takes 8.8 us so, 9.5 with two); and the
// workgroup's LDS in KB, slots of a step of the weights and rows, and the scales.
constexpr int mx4_skinny_depth(int rows, int waves) { return rows == 4 && waves == 8 ? 4 : 2; }
constexpr int mx4_skinny_lds(bool x4, bool pair, int rows, int waves) {
    const int w = pair ? 2 : 1, x = x4 ? (rows + 15) / 16 : rows / 4;
    return waves * ((w + x) * mx4_skinny_depth(rows, waves) + w + (x4 ? x : 0));
}
// Tiles of weight rows x input rows.
enum Mx4TileShape { MX4_TILE_SMALL, MX4_TILE_MIDDLE, MX4_TILE_LARGE, MX4_TILE_SHAPES };
hipError_t launch_mx4_tile(bool x4, bool pair, const Mx4Args& a, Mx4TileShape shape, hipStream_t s);

}  // namespace uwk

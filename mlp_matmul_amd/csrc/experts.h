// Argument blocks and launchers of the epilogue matmul, the products grouped
// by expert, the router's selection and the weighted sum of the experts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace uwk {

enum ValueType { VT_F32 = 0, VT_BF16 = 1 };
enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_COUNT = 5 };

constexpr int kMaxExperts = 512;   // of one routed layer
constexpr int kMaxTopK = 16;       // experts of a token

// A weight: bf16 [experts, rows, cols], or the direct-palette form of
// [experts*rows, cols] (sm not NULL).
struct Weight {
    const void* w;              // bf16 or 4-bit indices
    const uint8_t* sm;
    const uint8_t* vexp;
    const uint64_t* bitmap;
    const uint32_t* tile_vbase;
    uint32_t pal[4];
    uint32_t last_slot;         // of the verbatim groups (0 without any): lanes without one read inside VEXP
};

// y = act(v + bias[r]) + residual[b][r], rounded once to the type of `out`.
struct Epilogue {
    const void* bias;
    const void* residual;
    void* out;
    int64_t ldr, ldo;           // elements between rows of residual and out
    int32_t bias_type, residual_type, out_type, act;
};

// One matmul (or the gate/up pair) over rows grouped by expert.
struct GroupArgs {
    Weight w[2];                // [1]: up of the pair
    const uint16_t* X;
    const int32_t* offsets;     // [E+1] first row of each expert; NULL: one group of n rows
    const int32_t* order;       // row s reads X row order[s]/div; NULL: row s
    int64_t ldx, x_rows, n;
    int32_t E, R, C, div;
    Epilogue ep;                // the pair: only out (bf16) and ldo
    int32_t cus;
    int32_t split;              // K-slices of the bf16 tile kernel without offsets (1: none)
    float* sums;                // [split, n, R] of them when split > 1: out is not written
};

struct CombineArgs {
    const float* Y;             // [n, cols]
    const int32_t* place;       // [tokens, top_k], -1: none
    const int32_t* ids;         // [tokens, top_k] (launch_gemv_combine)
    const float* weights;       // [tokens, top_k]
    int64_t n, cols, tokens;
    int32_t top_k;
    const void* residual;
    void* out;
    int64_t ldr, ldo;
    int32_t residual_type, out_type;
};

// Scratch of the epilogue matmul (0: none is used).
uint64_t linear_scratch(bool pal, int64_t rows, int64_t cols, int64_t batch, int cus);
// The epilogue matmul: a.n rows of X in order, no offsets.
hipError_t launch_linear(bool pal, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s);
// A product grouped by expert, or the gate/up pair.
hipError_t launch_grouped(bool pal, bool pair, const GroupArgs& a, void* scratch, uint64_t scratch_bytes, hipStream_t s);
uint64_t grouped_scratch(bool pal, bool pair, int experts, int64_t rows, int64_t cols, int64_t n, int cus);

// The kernels behind them.  One or two rows an expert, cols <= 24576 / rows:
bool gemv_rows_supported(const GroupArgs& a, int nb);
hipError_t launch_gemv_rows(bool pal, bool pair, const GroupArgs& a, int nb, hipStream_t s);
// One token's down projection and the weighted sum of its experts (c.Y is not
// read): a.X the rows that c.place names.
bool gemv_combine_supported(const GroupArgs& a, int top_k);
hipError_t launch_gemv_combine(bool pal, const GroupArgs& a, const CombineArgs& c, hipStream_t s);
// Up to `rows` (4, 16 or 32) rows an expert before its weights are read again.
hipError_t launch_skinny_rows(bool pal, bool pair, const GroupArgs& a, int rows, hipStream_t s);
int skinny_waves(bool pair, int rows, const GroupArgs& a);    // of its workgroups
// Tiles of weight rows x input rows, bf16 and palette.
enum TileShape { TILE_64x64, TILE_128x64, TILE_256x128, TILE_256x256, TILE_SHAPES };
hipError_t launch_tile(bool pair, const GroupArgs& a, TileShape shape, hipStream_t s);
enum PalTileShape { PAL_TILE_64x64, PAL_TILE_128x64, PAL_TILE_128x128, PAL_TILE_SHAPES };
hipError_t launch_tile_pal(bool pair, const GroupArgs& a, PalTileShape shape, hipStream_t s);

struct RouteArgs {
    const void* logits;
    int64_t ld, tokens;
    int32_t type, experts, top_k, renorm;
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* order;
    int32_t* place;
    uint16_t* counts;           // [blocks, experts up to 8s] of every block's slots, when blocks > 1
    int32_t blocks, per_block;  // tokens of a block: a multiple of 16
};

// Blocks of tokens of a routing call (1: a single launch, no counts).
void route_blocks(int64_t tokens, int32_t* blocks, int32_t* per_block);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

hipError_t launch_combine(const CombineArgs& a, hipStream_t s);

}  // namespace uwk

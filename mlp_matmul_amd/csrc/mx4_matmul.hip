// Products with microscaled 4-bit weights, alone or grouped by expert: which
// kernel runs a shape.
//
//   y_s = act(W_e(s) x_s + b) + r_s,   h_s = SiLU(G_e(s) x_s) * (U_e(s) x_s)
//
// with fp32 sums, one rounding at the end.  A weight is 2^(s-127) c with c of
// two significant bits: a product with a bf16 number is exact in fp32, as it is
// with another 4-bit one.
#include <algorithm>

#include "grouped_common.h"
#include "kernels.h"
#include "mx4.h"

namespace uwk {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// A 16 x 16 tile a wave straight from memory, 128 columns a step; four waves
// share 16 input rows.
template <bool X4, bool PAIR>
__global__ __launch_bounds__(256) void mx4_simple_kernel(Mx4Args a, uint32_t bands) {
    GroupTile t;
    if (!group_tile<16>(a.g, bands, t)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const int64_t R = a.g.R, row0 = int64_t(t.band) * 64 + wave * 16;
    if (row0 >= R) return;
    const int64_t wr = int64_t(t.e) * R + min(row0 + rl, R - 1);
    const int64_t xr = group_x_index(a.g, t.row0 + min(rl, uint32_t(t.rows) - 1u));
    const uint32_t blocks = uint32_t(a.g.C) / kMx4Block;
    constexpr int M = PAIR ? 2 : 1;
    f32x4_t acc[M] = {};
    for (uint32_t b0 = 0; b0 < blocks; b0 += 4) {
        const bool in = b0 + q < blocks;                 // a lane behind the last block multiplies zeros
        const uint32_t b = in ? b0 + q : 0u;
        i32x8_t xc{};
        uint32_t xs = 127;
        u32x4_t xv[4];
        if (X4) {
            const u32x4_t c = load16(a.x.codes + xr * a.x.ldc + b * 16u);
#pragma unroll
            for (int k = 0; k < 4; ++k) xc[k] = in ? int(c[k]) : 0;
            if (in) xs = a.x.scales[xr * a.x.lds + b];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                xv[k] = load16(a.g.X + xr * a.g.ldx + b * 32u + uint32_t(k) * 8u);
                if (!in) xv[k] = u32x4_t{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const u32x4_t c = load16(a.w[m].codes + wr * a.w[m].ldc + b * 16u);
            const uint32_t s = in ? a.w[m].scales[wr * a.w[m].lds + b] : 127u;
            if (X4) {
                i32x8_t wc{};
#pragma unroll
                for (int k = 0; k < 4; ++k) wc[k] = in ? int(c[k]) : 0;
                acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wc, xc, acc[m], 4, 4, 0, int(s), 0, int(xs));
            } else {
                const float scale = __uint_as_float(s << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t d = in ? c[k] : 0u;
                    const u32x4_t w{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0)),
                                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1)),
                                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2)),
                                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3))};
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                                     __builtin_bit_cast(bf16x8_t, xv[k]), acc[m], 0, 0, 0);
                }
            }
        }
    }
    const uint32_t row = uint32_t(row0) + 4u * q;
    if (rl >= uint32_t(t.rows) || row >= uint32_t(R)) return;
    f32x4_t y = acc[0];
    if (PAIR) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = silu(y[i]) * acc[M - 1][i];
    }
    epilogue4(a.g.ep, t.row0 + rl, int(row), a.g.R, y);
}

template <bool X4, bool PAIR>
hipError_t launch_simple(const Mx4Args& a, hipStream_t s) {
    const int64_t bands = (int64_t(a.g.R) + 63) / 64, units = group_units(a.g, 16, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    launch_timed(mx4_simple_kernel<X4, PAIR>, dim3(unsigned(units)), dim3(256), 0, s, a, uint32_t(bands));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4(bool x4, bool pair, const Mx4Args& a, hipStream_t s) {
    if (a.g.n <= 0 || a.g.R <= 0) return hipSuccess;
    if (x4) return pair ? launch_simple<true, true>(a, s) : launch_simple<true, false>(a, s);
    return pair ? launch_simple<false, true>(a, s) : launch_simple<false, false>(a, s);
}

}  // namespace uwk

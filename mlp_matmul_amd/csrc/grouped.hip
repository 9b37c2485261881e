// Matmul with bias, activation and residual in its epilogue, and the products
// of a mixture-of-experts layer grouped by expert: single matrices and the
// gate/up pair with the SiLU product, over bf16 weights or the direct-palette
// form.
//
//   y_s = act(W_e(s) x_s + b) + r_s,   h_s = SiLU(G_e(s) x_s) * (U_e(s) x_s)
//
// with fp32 sums, one rounding at the end.  Expert e's matrix is rows
// e*R .. e*R+R-1 of the stacked weights; its input rows are those between
// offsets[e] and offsets[e+1].
#include "grouped_common.h"

namespace uwk {

namespace {

constexpr int kMT = 64, kNT = 64, kKS = 64;    // weight rows, input rows, columns of a step
constexpr int kPad = 8;

// One lane's 16 weights at element pos of the stacked matrix.
template <bool PAL>
__device__ __forceinline__ void weights16(const Weight& w, int64_t pos, const uint32_t* lut, uint32_t out[8]) {
    if (!PAL) {
        const uint16_t* p = static_cast<const uint16_t*>(w.w) + pos;
        const u32x4_t a = load16(p), b = load16(p + 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[i] = a[i];
            out[4 + i] = b[i];
        }
        return;
    }
    const u32x2_t nib = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(w.w) + pos / 2);
    const u32x4_t sm = load16(w.sm + pos);
    const int64_t g = pos >> 6;
    const uint64_t word = w.bitmap[g >> 6];
    const uint32_t bit = uint32_t(g) & 63u;
    uint32_t e7[8];
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
        out[p] = (p & 1) ? join_pair<1>(sm[p >> 1], e7[p]) : join_pair<0>(sm[p >> 1], e7[p]);
}

template <bool PAL, bool PAIR>
__global__ __launch_bounds__(256) void grouped_kernel(GroupArgs a, uint32_t bands) {
    constexpr int M = PAIR ? 2 : 1;
    __shared__ __align__(16) uint16_t wl[M][kMT][kKS + kPad];
    __shared__ __align__(16) uint16_t xl[kNT][kKS + kPad];
    __shared__ uint32_t lut[M][256];
    GroupTile t;
    if (!group_tile<kNT>(a, bands, t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (PAL) {
#pragma unroll
        for (int m = 0; m < M; ++m)
            lut[m][tid] = (pal_byte(a.w[m].pal, tid & 15) << 7) | (pal_byte(a.w[m].pal, tid >> 4) << 23);
    }
    __syncthreads();
    const int r0 = t.band * kMT;
    // the thread's weights: row tid/4 of the band, columns 16*(tid%4).. of a
    // step; its input pieces: row tid/4, the same columns
    const int lr = tid >> 2, lc = (tid & 3) * 16;
    const int row = min(r0 + lr, a.R - 1);
    const int64_t wpos = (int64_t(t.e) * a.R + row) * a.C + lc;
    const uint16_t* const x = group_x_row(a, t.row0 + min(lr, t.rows - 1)) + lc;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32, q = lane >> 4, l16 = lane & 15;
    f32x4_t acc[M][2][2];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i >> 1][i & 1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < a.C; k += kKS) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            uint32_t w[8];
            weights16<PAL>(a.w[m], wpos + k, lut[m], w);
            store16(&wl[m][lr][lc], u32x4_t{w[0], w[1], w[2], w[3]});
            store16(&wl[m][lr][lc + 8], u32x4_t{w[4], w[5], w[6], w[7]});
        }
        store16(&xl[lr][lc], load16(x + k));
        store16(&xl[lr][lc + 8], load16(x + k + 8));
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8_t A[M][2], B[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                B[i] = *reinterpret_cast<const bf16x8_t*>(&xl[wn + 16 * i + l16][32 * h + 8 * q]);
#pragma unroll
                for (int m = 0; m < M; ++m)
                    A[m][i] = *reinterpret_cast<const bf16x8_t*>(&wl[m][wm + 16 * i + l16][32 * h + 8 * q]);
            }
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[m][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[m][i], B[j], acc[m][i][j], 0, 0, 0);
        }
        __syncthreads();
    }
    // D layout: lane l holds input row l%16, weight rows 4*(l/16) .. +3
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + wm + 16 * i + 4 * q;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int b = wn + 16 * j + l16;
            if (b >= t.rows || r >= a.R) continue;
            f32x4_t v = acc[0][i][j];
            if (PAIR) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = silu_mul1(v[c], acc[M - 1][i][j][c]);
            }
            epilogue4(a.ep, t.row0 + b, r, a.R, v);
        }
    }
}

template <bool PAL, bool PAIR>
hipError_t launch(const GroupArgs& a, hipStream_t s) {
    const int64_t bands = (a.R + kMT - 1) / kMT, units = group_units(a, kNT, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    grouped_kernel<PAL, PAIR><<<unsigned(units), 256, 0, s>>>(a, uint32_t(bands));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(bool pal, bool pair, const GroupArgs& a, hipStream_t s) {
    if (a.n <= 0 || a.R <= 0) return hipSuccess;
    if (pal) return pair ? launch<true, true>(a, s) : launch<true, false>(a, s);
    return pair ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace uwk

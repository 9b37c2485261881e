// Microscaled 4-bit numbers from bf16 or fp32 and back.
//
// Quantising a block of 32: with e the biased exponent of its largest
// magnitude, s = max(e - 2, 0) (the largest lands in [4, 8), in steps of 2),
// and x 2^(127-s) is rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6,
// ties to the even code, magnitudes above 5 to 6.  Every step is exact but the
// rounding, so the result does not depend on how it is computed.  A block with
// a NaN or an infinity is no number: s = 255, its codes 0.
//
// Four lanes share a block, eight numbers each: one 16-byte load of bf16 (two
// of fp32), the largest magnitude as an integer over the four lanes by DPP, and
// the hardware's conversion, two numbers an instruction, which rounds and
// saturates as above (v_cvt_scalef32_pk_fp4_*).  Memory bound: 14336 x 4096 in
// bf16 takes 26.3 us there and 22.0 back, 149 MB each (5.7 and 6.8 TB/s; a copy
// of 2 GiB runs at 4.85).
#include <algorithm>

#include "grouped_common.h"
#include "mx4.h"

namespace uwk {

namespace {

constexpr int kLoads = 4;            // eights of a lane, all on their way at once

// idx / d and the rest, d > 0 and m = min(2^32 / d, 2^32 - 1): the product is below the quotient by at most one.
__device__ __forceinline__ uint32_t divide(uint32_t idx, uint32_t d, uint32_t m, uint32_t& rest) {
    uint32_t q = __umulhi(idx, m);
    rest = idx - q * d;
    if (rest >= d) {
        ++q;
        rest -= d;
    }
    return q;
}

inline uint32_t divisor(uint32_t d) { return d > 1 ? uint32_t((uint64_t(1) << 32) / d) : 0xFFFFFFFFu; }

// the larger over the four lanes of a quad, in each of them
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));   // lanes 1 0 3 2
    return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));   // lanes 2 3 0 1
}

struct ConvertArgs {
    const void* in;
    void* out;
    uint8_t* codes;
    uint8_t* scales;
    int64_t ld, ldc, lds;       // of the numbers, the codes, the scales
    uint32_t eights, total, m;  // eights of numbers of a row and in all, divisor(eights)
};

template <bool F32>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(ConvertArgs a) {
    const uint64_t base = uint64_t(blockIdx.x) * (256 * kLoads) + threadIdx.x;
    u32x4_t v[kLoads][F32 ? 2 : 1];
    uint32_t row[kLoads], col[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const uint64_t i = min(base + uint64_t(k) * 256u, uint64_t(a.total) - 1u);
        row[k] = divide(uint32_t(i), a.eights, a.m, col[k]);
        const int64_t o = int64_t(row[k]) * a.ld + int64_t(col[k]) * 8;
        if (F32) {
            const float* const p = static_cast<const float*>(a.in) + o;
            v[k][0] = load_stream16(p);
            v[k][F32 ? 1 : 0] = load_stream16(p + 4);
        } else {
            v[k][0] = load_stream16(static_cast<const uint16_t*>(a.in) + o);
        }
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (F32) {
                top = max(top, max(v[k][0][j] & 0x7FFFFFFFu, v[k][F32 ? 1 : 0][j] & 0x7FFFFFFFu));
            } else {
                top = max(top, max((v[k][0][j] << 16) & 0x7FFFFFFFu, v[k][0][j] & 0x7FFF0000u));
            }
        }
        const uint32_t e = quad_max(top) >> 23, s = e == 255u ? 255u : max(e, 2u) - 2u;
        const float scale = __uint_as_float(s << 23);        // its exponent counts: 0 is 2^-127
        uint32_t c = 0;
        if (F32) {
            const f32x4_t x = __builtin_bit_cast(f32x4_t, v[k][0]), y = __builtin_bit_cast(f32x4_t, v[k][F32 ? 1 : 0]);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], scale, 3);
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, uint32_t(v[k][0][0])), scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, uint32_t(v[k][0][1])), scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, uint32_t(v[k][0][2])), scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, uint32_t(v[k][0][3])), scale, 3);
        }
        if (s == 255u) c = 0;
        if (base + uint64_t(k) * 256u >= a.total) continue;
        *reinterpret_cast<uint32_t*>(a.codes + int64_t(row[k]) * a.ldc + int64_t(col[k]) * 4) = c;
        if ((col[k] & 3u) == 0) a.scales[int64_t(row[k]) * a.lds + (col[k] >> 2)] = uint8_t(s);
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(ConvertArgs a) {
    const uint64_t base = uint64_t(blockIdx.x) * (256 * kLoads) + threadIdx.x;
    uint32_t row[kLoads], col[kLoads], c[kLoads], s[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const uint64_t i = min(base + uint64_t(k) * 256u, uint64_t(a.total) - 1u);
        row[k] = divide(uint32_t(i), a.eights, a.m, col[k]);
        c[k] = *reinterpret_cast<const uint32_t*>(a.codes + int64_t(row[k]) * a.ldc + int64_t(col[k]) * 4);
        s[k] = a.scales[int64_t(row[k]) * a.lds + (col[k] >> 2)];
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        if (base + uint64_t(k) * 256u >= a.total) continue;
        const float scale = __uint_as_float(s[k] << 23);
        const int64_t o = int64_t(row[k]) * a.ld + int64_t(col[k]) * 8;
        const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 0);
        const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 1);
        const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 2);
        const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 3);
        const u32x4_t h{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1), __builtin_bit_cast(uint32_t, p2),
                        __builtin_bit_cast(uint32_t, p3)};
        if (F32) {                                           // bf16 holds each of the values
            float* const d = static_cast<float*>(a.out) + o;
            *reinterpret_cast<u32x4_e4_t*>(d) = u32x4_t{h[0] << 16, h[0] & 0xFFFF0000u, h[1] << 16, h[1] & 0xFFFF0000u};
            *reinterpret_cast<u32x4_e4_t*>(d + 4) = u32x4_t{h[2] << 16, h[2] & 0xFFFF0000u, h[3] << 16, h[3] & 0xFFFF0000u};
        } else {
            *reinterpret_cast<u32x4_e2_t*>(static_cast<uint16_t*>(a.out) + o) = h;
        }
    }
}

// Eights of one launch: their numbers fit 32 bits.
constexpr int64_t kMostEights = (int64_t(1) << 32) - 1;

template <class K>
hipError_t launch_rows(K kernel, ConvertArgs a, int64_t rows, int64_t in_row, int64_t out_row, hipStream_t s) {
    const int64_t per = std::max<int64_t>(kMostEights / a.eights, 1);
    for (int64_t r = 0; r < rows; r += per) {                // more than 2^35 numbers: several launches
        const int64_t n = std::min(per, rows - r);
        ConvertArgs b = a;
        b.in = a.in ? static_cast<const uint8_t*>(a.in) + r * in_row : nullptr;
        b.out = a.out ? static_cast<uint8_t*>(a.out) + r * out_row : nullptr;
        b.codes = a.codes + r * a.ldc;
        b.scales = a.scales + r * a.lds;
        b.total = uint32_t(n * a.eights);
        b.m = divisor(a.eights);
        kernel<<<unsigned((int64_t(b.total) + 256 * kLoads - 1) / (256 * kLoads)), 256, 0, s>>>(b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_mx4_quantize(const void* X, int type, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes,
                               int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s) {
    if (rows <= 0 || cols <= 0) return hipSuccess;
    const ConvertArgs a{X, nullptr, codes, scales, ldx, ldc, lds, uint32_t(cols / 8), 0, 0};
    return type == VT_F32 ? launch_rows(mx4_quantize_kernel<true>, a, rows, ldx * 4, 0, s)
                          : launch_rows(mx4_quantize_kernel<false>, a, rows, ldx * 2, 0, s);
}

hipError_t launch_mx4_dequantize(const Mx4Mat& m, int64_t rows, int64_t cols, void* out, int type, int64_t ldo,
                                 hipStream_t s) {
    if (rows <= 0 || cols <= 0) return hipSuccess;
    const ConvertArgs a{nullptr, out, const_cast<uint8_t*>(m.codes), const_cast<uint8_t*>(m.scales), ldo, m.ldc, m.lds,
                        uint32_t(cols / 8), 0, 0};
    return type == VT_F32 ? launch_rows(mx4_dequantize_kernel<true>, a, rows, 0, ldo * 4, s)
                          : launch_rows(mx4_dequantize_kernel<false>, a, rows, 0, ldo * 2, s);
}

}  // namespace uwk

// Device helpers of the products with 4-bit weights.
#pragma once

#include "grouped_common.h"
#include "mx4.h"

namespace uwk {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));

// The 8 numbers of a dword of codes with scale byte s, exactly.
__device__ __forceinline__ bf16x8_t mx4_to_bf16(uint32_t codes, uint32_t s) {
    const float scale = __uint_as_float(s << 23);            // the instruction takes the exponent: 0 is 2^-127, 255 NaN
    const u32x4_t w{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3))};
    return __builtin_bit_cast(bf16x8_t, w);
}

// acc + A B over 128 columns: lane l has row l % 16 and its block l / 16 of A and of B, 32 codes and the scale, byte
// BA of sa and BB of sb.
template <int BA, int BB>
__device__ __forceinline__ f32x4_t mfma_mx4(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x4_t acc) {
    const i32x8_t A{int(a[0]), int(a[1]), int(a[2]), int(a[3]), 0, 0, 0, 0};
    const i32x8_t B{int(b[0]), int(b[1]), int(b[2]), int(b[3]), 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 4, BA, int(sa), BB, int(sb));
}

}  // namespace uwk

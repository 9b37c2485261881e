// A single token's down projection with 4-bit weights and the sum over its
// experts:  out = sum_j w_j D_e(j) h_j (+ residual).
//
// The rows of h are those that gate/up wrote, a slot each, at place[j]; the
// expert of a row is the one whose offsets hold it.  A workgroup owns 16 rows of
// every chosen expert's matrix.  Its eight waves share the slots' steps of 128 columns
// in contiguous runs: codes, scales and h go from memory to registers, D steps
// on their way, the weights become bf16 there and meet h on the matrix units.  At
// the end of a slot a wave adds w_j times its fp32 sum to its own, and the waves'
// sums are added in wave order: results do not depend on scheduling.
//
// Bound by the launch and the latency of a few loads.  With gate/up, 6 of 64 experts
// of 2048 x 1408 take 16.9 us, 18.1 with the grouped product and the sum in a
// launch each (and 3.3 more on the host); 2 of 8 of 4096 x 3584 17.6, not 19.4.  With
// 4 or 16 waves 0.5 us more, and with one lane in sixteen loading h no less.
#include "kernels.h"
#include "mx4_common.h"

namespace uwk {

namespace {

constexpr int KW = 8;                // waves of a workgroup

__global__ __launch_bounds__(64 * KW) void mx4_one_kernel(Mx4OneArgs a) {
    constexpr int D = 4;
    __shared__ f32x4_t part[KW][64];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, q = lane >> 4, rl = lane & 15u;
    const uint32_t R = uint32_t(a.R), blocks = uint32_t(a.C) / kMx4Block, steps = (blocks + 3u) / 4u;
    const uint32_t row0 = blockIdx.x * 16u;

    // lane j: row, weight and expert of slot j (-1: none)
    const int32_t place = int(lane) < a.top_k ? a.place[lane] : -1;
    const float weight = int(lane) < a.top_k ? a.weights[lane] : 0.f;
    int32_t expert = -1;
    for (int c = 0; c < a.E; c += 64) {
        const int32_t o0 = a.offsets[min(c + int(lane), a.E)], o1 = a.offsets[min(c + int(lane) + 1, a.E)];
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = __builtin_amdgcn_readlane(place, j);
            const uint64_t here = __builtin_amdgcn_ballot_w64(o0 <= r && r < o1 && c + int(lane) < a.E);
            if (here && int(lane) == j && expert < 0) expert = c + __builtin_ctzll(here);
        }
    }
    if (place < 0 || place >= a.top_k) expert = -1;          // h has top_k rows

    const uint32_t total = uint32_t(a.top_k) * steps, lo = total * uint32_t(wave) / KW, hi = total * uint32_t(wave + 1) / KW;
    f32x4_t sum{0.f, 0.f, 0.f, 0.f};
    for (uint32_t j = lo / steps; j * steps < hi; ++j) {
        const int32_t e = __builtin_amdgcn_readlane(expert, int(j));
        if (e < 0) continue;
        const uint32_t s0 = max(lo, j * steps) - j * steps, s1 = min(hi, (j + 1u) * steps) - j * steps;
        if (s0 >= s1) continue;
        // lane l has row l % 16 and block l / 16 of a step; blocks behind the last read it, and count as zeros
        const int64_t row = int64_t(e) * R + min(row0 + rl, R - 1u);
        const uint8_t* const codes = a.w.codes + row * a.w.ldc;
        const uint8_t* const scales = a.w.scales + row * a.w.lds;
        const uint16_t* const x = a.h + int64_t(__builtin_amdgcn_readlane(place, int(j))) * a.ldh;
        u32x4_t c[D], h[D][4];
        uint32_t s[D];
        auto load = [&](int d, uint32_t step) {
            const uint32_t b = min(4u * min(step, s1 - 1u) + q, blocks - 1u);
            c[d] = *reinterpret_cast<const u32x4_t*>(codes + b * 16u);
            s[d] = scales[b];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[d][k] = *reinterpret_cast<const u32x4_t*>(x + b * 32u + k * 8);
        };
        f32x4_t acc{0.f, 0.f, 0.f, 0.f};
        auto add = [&](int d, uint32_t step) {
            const bool gone = 4u * step + q >= blocks;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const u32x4_t none{0u, 0u, 0u, 0u};
                const bf16x8_t w = mx4_to_bf16(gone ? 0u : c[d][k], gone ? 127u : s[d]);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, gone ? none : h[d][k]), acc, 0, 0, 0);
            }
        };
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, s0 + uint32_t(d));
        for (uint32_t i = s0; i < s1; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i + uint32_t(d) < s1) add(d, i + uint32_t(d));
                if (i + uint32_t(d) + D < s1) load(d, i + uint32_t(d) + D);
            }
        }
        const float w = __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(weight)), int(j))));
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = fmaf(w, acc[k], sum[k]);
    }
    // D layout: weight rows 4 * (l / 16) .. + 3, alike for every l % 16
    part[wave][lane] = sum;
    __syncthreads();
    const uint32_t r = row0 + 4u * q;
    if (wave || rl || r >= R) return;
    f32x4_t y = part[0][lane];
#pragma unroll
    for (int w = 1; w < KW; ++w) y += part[w][lane];
    epilogue4(a.ep, 0, int(r), a.R, y);
}

}  // namespace

// Long sums over few rows keep too few compute units busy: with gate/up, 2 of 2 experts of 4096 x 14336 take 54.4 us,
// 51.7 with the product and the sum apart, 8 of 32 of 2048 x 2048 25.2 and 21.7; 3 of 8 of 4096 x 4096 26.0 and 26.4.
// At 300 drawn sizes (1 to 16 of 2 to 256 experts, 128 to 14336 columns, 512 to 8192 rows) the rule takes 1.011 times the
// faster one's time in the geometric mean, 1.03 at the 90th percentile and 1.32 at worst; with 3 or 10 in the place of 5
// it takes 1.017 and 1.013.
bool mx4_one_supported(const Mx4OneArgs& a) { return int64_t(a.top_k) * a.C <= 5 * int64_t(a.R); }

hipError_t launch_mx4_one(const Mx4OneArgs& a, hipStream_t s) {
    if (a.R <= 0) return hipSuccess;
    launch_timed(mx4_one_kernel, dim3(unsigned((int64_t(a.R) + 15) / 16)), dim3(64 * KW), 0, s, a);
    return hipGetLastError();
}

}  // namespace uwk

// The router of a mixture-of-experts layer and the weighted sum of a token's
// experts.
//
// Selection.  Of a token's E logits l the top_k largest are chosen, equal
// ones by the lowest index; the chosen experts' weights are
//   w_j = exp(l_j - max) / sum exp(l_i - max)
// over the chosen ones or over all E.  A -inf or NaN logit is never chosen
// (id -1, weight 0), +inf counts as the largest finite number.  Sums and
// exponentials are fp32 with the maximum taken off, so every exponent is <= 0.
//
// Mapping to CDNA4.  16 lanes (one DPP row) hold a token, E/16 logits each;
// four tokens a wave.  A round finds the largest remaining logit: a scan of
// the lane's own values, then four DPP row rotations for the value and four
// for the lowest index that holds it: no LDS traffic, no barrier.  A wave per
// token would spend as many instructions on a quarter of the tokens.
//
// Grouping.  A counting sort that keeps flat order t*top_k + j inside every
// expert, so results are deterministic: every wave owns a contiguous run of
// tokens, the slots before a slot are those of earlier blocks (counts summed
// from memory), of earlier waves (per-wave counts in LDS) and of lower lanes
// or earlier chunks of its wave (equal experts matched bit by bit with
// ballots).  Up to 64 tokens take one launch of one workgroup; more take a
// launch for the selection and the blocks' counts, and one for the places.
#include <float.h>

#include "grouped_common.h"

namespace uwk {

namespace {

constexpr int kRT = 1024;            // threads of a workgroup
constexpr int kRW = kRT / 64;        // its waves
constexpr int kMaxBlocks = 256;         // one a compute unit: 16384 tokens in blocks of 64

template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + N, 0xF, 0xF, false));
}

// over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, row_ror<8>(v));
    v = max(v, row_ror<4>(v));
    v = max(v, row_ror<2>(v));
    return max(v, row_ror<1>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
    v = min(v, row_ror<8>(v));
    v = min(v, row_ror<4>(v));
    v = min(v, row_ror<2>(v));
    return min(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
    v += dpp_ror(v, 8);
    v += dpp_ror(v, 4);
    v += dpp_ror(v, 2);
    return v + dpp_ror(v, 1);
}

// floats as unsigned numbers in the same order; 0 is below every float
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);          // -0 becomes +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t t, int e) {
    const int64_t i = t * a.ld + e;
    return a.type == VT_BF16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.logits)[i]) << 16)
                             : static_cast<const float*>(a.logits)[i];
}

// Selects the experts of tokens t (one per DPP row; t >= tokens: nothing) and
// counts them in cnt[expert].  V logits a lane: expert 16*c + lane.
template <int V>
__device__ void select(const RouteArgs& a, int64_t t, uint32_t sub, uint32_t* cnt) {
    const bool live = t < a.tokens;
    uint32_t key[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int e = 16 * c + int(sub);
        key[c] = 0;                                        // no such expert, -inf, NaN
        if (live && e < a.experts) {
            const float f = load_logit(a, t, e);
            if (f > -INFINITY) key[c] = order_key(fminf(f, FLT_MAX));
        }
    }
    uint32_t my_key = 0, my_id = ~0u, top = 0;
    float all = 0.f, chosen = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0, at = ~0u;
#pragma unroll
        for (int c = 0; c < V; ++c)
            if (key[c] > best) {
                best = key[c];
                at = 16u * c + sub;
            }
        const uint32_t m = row_max(best);
        const uint32_t e = row_min(best == m && m ? at : ~0u);
        if (j == 0) {
            top = m;
            if (!a.renorm) {
#pragma unroll
                for (int c = 0; c < V; ++c) all += key[c] ? expf(order_value(key[c]) - order_value(m)) : 0.f;
                all = row_sum(all);
            }
        }
#pragma unroll
        for (int c = 0; c < V; ++c)
            if (e == 16u * c + sub) key[c] = 0;
        if (m) chosen += expf(order_value(m) - order_value(top));
        if (uint32_t(j) == sub) {
            my_key = m;
            my_id = e;
        }
    }
    if (live && int(sub) < a.top_k) {
        const int64_t o = t * a.top_k + sub;
        const float w = my_key ? expf(order_value(my_key) - order_value(top)) / (a.renorm ? chosen : all) : 0.f;
        a.ids[o] = int32_t(my_id);
        a.weights[o] = w;
        if (my_key) atomicAdd(cnt + my_id, 1u);
    }
}

__device__ __forceinline__ void select_any(const RouteArgs& a, int64_t t, uint32_t sub, uint32_t* cnt) {
    if (a.experts <= 16) select<1>(a, t, sub, cnt);
    else if (a.experts <= 32) select<2>(a, t, sub, cnt);
    else if (a.experts <= 64) select<4>(a, t, sub, cnt);
    else if (a.experts <= 128) select<8>(a, t, sub, cnt);
    else if (a.experts <= 256) select<16>(a, t, sub, cnt);
    else select<32>(a, t, sub, cnt);
}

// PHASE 0: everything (one block); 1: selection and the block's counts; 2:
// offsets and places.
template <int PHASE>
__global__ __launch_bounds__(kRT) void route_kernel(RouteArgs a) {
    __shared__ uint32_t cnt[kRW][kMaxExperts];             // slots of each wave, then the next place of each
    __shared__ uint32_t wave_total[kMaxExperts / 64];
    __shared__ uint32_t part[2][PHASE == 2 ? kRT : 1];     // (before, in all) of each group of blocks
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, sub = lane & 15u;
    const int E = a.experts, K = a.top_k;
    const int64_t tb = int64_t(blockIdx.x) * a.per_block;  // the block's tokens, the wave's inside them
    const int64_t t_lo = tb + int64_t(wave) * (a.per_block / kRW), t_hi = min(t_lo + a.per_block / kRW, a.tokens);
    for (int i = tid; i < kRW * E; i += kRT) cnt[i / E][i % E] = 0;
    __syncthreads();
    if (PHASE != 2) {
        for (int64_t t = t_lo; t < t_hi; t += 4) {
            const int64_t mine = t + (lane >> 4);
            select_any(a, mine < t_hi ? mine : a.tokens, sub, cnt[wave]);
        }
    } else {
        for (int64_t i = t_lo * K + lane; i < t_hi * K; i += 64)
            if (a.ids[i] >= 0) atomicAdd(&cnt[wave][a.ids[i]], 1u);
    }
    __syncthreads();
    if (PHASE == 1) {
        if (tid < E) {
            uint32_t s = 0;
#pragma unroll
            for (int w = 0; w < kRW; ++w) s += cnt[w][tid];
            a.counts[int64_t(blockIdx.x) * E + tid] = int32_t(s);
        }
        return;
    }

    // slots of every expert, before this block and in all; then where each
    // expert starts: a scan over the experts.  The blocks' counts are summed by
    // as many groups of threads as fit, 16 loads on their way at a time.
    uint32_t before = 0, total = 0;
    if (PHASE == 2) {
        const int ep = (E + 63) & ~63, groups = kRT / ep, g = tid / ep, e = tid % ep;
        const int lo = a.blocks * g / groups, hi = a.blocks * (g + 1) / groups;
        uint32_t bef = 0, tot = 0;
        if (g < groups && e < E) {
#pragma unroll 16
            for (int b = lo; b < hi; ++b) {
                const uint32_t c = uint32_t(a.counts[int64_t(b) * E + e]);
                tot += c;
                bef += b < int(blockIdx.x) ? c : 0u;
            }
            part[0][tid] = bef;
            part[1][tid] = tot;
        }
        __syncthreads();
        if (tid < E)
            for (int i = 0; i < groups; ++i) {
                before += part[0][i * ep + tid];
                total += part[1][i * ep + tid];
            }
    } else if (tid < E) {
#pragma unroll
        for (int w = 0; w < kRW; ++w) total += cnt[w][tid];
    }
    uint32_t incl = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(incl, d, 64);
        if (int(lane) >= d) incl += o;
    }
    if (tid < kMaxExperts && lane == 63) wave_total[wave] = incl;
    __syncthreads();
    uint32_t all = 0, mine = 0;
#pragma unroll
    for (int w = 0; w < kMaxExperts / 64; ++w) {
        if (w < wave) mine += wave_total[w];
        all += wave_total[w];
    }
    if (tid < E) {
        uint32_t at = mine + incl - total;
        if (blockIdx.x == 0) {
            a.offsets[tid] = int32_t(at);
            if (tid == E - 1) a.offsets[E] = int32_t(at + total);
        }
        at += before;
#pragma unroll
        for (int w = 0; w < kRW; ++w) {
            const uint32_t c = cnt[w][tid];
            cnt[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i0 = t_lo * K; i0 < t_hi * K; i0 += 64) {
        const int64_t i = i0 + lane;
        const int32_t e = i < t_hi * K ? a.ids[i] : -1;
        uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
#pragma unroll
        for (int b = 0; (1 << b) < kMaxExperts; ++b) {
            const uint64_t set = __builtin_amdgcn_ballot_w64((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const uint32_t rank = uint32_t(__popcll(same & ((uint64_t(1) << lane) - 1)));
        uint32_t first = 0;
        if (e >= 0) first = cnt[wave][e];
        __builtin_amdgcn_wave_barrier();                   // every lane has read before one adds
        if (e >= 0 && rank == 0) cnt[wave][e] = first + uint32_t(__popcll(same));
        __builtin_amdgcn_wave_barrier();
        if (e >= 0) {
            a.order[first + rank] = int32_t(i);
            a.place[i] = int32_t(first + rank);
        } else if (i < t_hi * K) {
            a.place[i] = -1;
        }
    }
    // rows behind the last expert's
    const int64_t lo = tb * K, hi = min(tb + a.per_block, a.tokens) * K;
    for (int64_t i = lo + tid; i < hi; i += kRT)
        if (i >= int64_t(all)) a.order[i] = -1;
}

// out[t] = sum_j weights[t][j] * Y[place[t][j]] (+ residual[t]), j ascending.
// Memory bound: four columns a lane.
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    const int64_t quads = (a.cols + 3) / 4, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.tokens * quads) return;
    const int64_t t = i / quads;
    const int c = int(i % quads) * 4, C = int(a.cols);
    const bool aligned = (C & 3) == 0;
    f32x4_t v{0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.top_k; ++j) {
        const int32_t p = a.place[t * a.top_k + j];
        if (p < 0 || p >= a.n) continue;
        const f32x4_t y = load4(a.Y, VT_F32, int64_t(p) * C + c, c, C, aligned);
        const float w = a.weights[t * a.top_k + j];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = fmaf(w, y[k], v[k]);
    }
    epilogue4(Epilogue{nullptr, a.residual, a.out, a.ldr, a.ldo, VT_F32, a.residual_type, a.out_type, ACT_NONE}, t, c, C, v);
}

}  // namespace

void route_blocks(int64_t tokens, int32_t* blocks, int32_t* per_block) {
    const int64_t per = ((tokens + kMaxBlocks - 1) / kMaxBlocks + 63) / 64 * 64;
    *per_block = int32_t(per > 64 ? per : 64);
    const int64_t n = (tokens + *per_block - 1) / *per_block;
    *blocks = int32_t(n > 1 ? n : 1);                      // no tokens: one block writes the offsets
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    if (a.blocks == 1) {
        route_kernel<0><<<1, kRT, 0, s>>>(a);
        return hipGetLastError();
    }
    route_kernel<1><<<unsigned(a.blocks), kRT, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_kernel<2><<<unsigned(a.blocks), kRT, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
    if (a.tokens <= 0 || a.cols <= 0) return hipSuccess;
    const int64_t quads = a.tokens * ((a.cols + 3) / 4), blocks = (quads + 255) / 256;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    combine_kernel<<<unsigned(blocks), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace uwk

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
//
// Measured: 8 tokens of 64 experts 4.1 us, a launch; 16384 of 256 12 us for the
// selection, bound by vector instructions (85 a round of four tokens), and 8 for the
// places, bound by the latency of a chain of small steps.
#include <float.h>

#include <algorithm>

#include "grouped_common.h"

namespace uwk {

namespace {

constexpr int kRT = 1024;            // threads of a workgroup
constexpr int kRW = kRT / 64;        // its waves
constexpr int kMaxBlocks = 256;      // one a compute unit (16 to 64 tokens each through 16384), until 16 bits end

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

// Selects the experts of tokens t (one per DPP row; t >= tokens: nothing) and
// counts them in cnt[expert].  V logits a lane, in runs of four where V allows
// a wide load.
template <int V>
__device__ void select(const RouteArgs& a, int64_t t, uint32_t sub, uint32_t* cnt) {
    constexpr int W = V < 4 ? 1 : 4;
    const bool live = t < a.tokens;
    auto expert = [&](int c) { return uint32_t(16 * W * (c / W) + c % W) + W * sub; };
    uint32_t key[V];
    // every load stays inside the logits and none waits for another
    float f[V];
    const int E = a.experts;
    const int64_t row = min(t, a.tokens - 1) * a.ld;
    const float* const pf = static_cast<const float*>(a.logits) + row;
    const uint16_t* const ph = static_cast<const uint16_t*>(a.logits) + row;
    if (W == 4 && ((a.ld | E) & 3) == 0 && (reinterpret_cast<uint64_t>(a.logits) & 15) == 0) {
        if (a.type == VT_F32) {
#pragma unroll
            for (int c = 0; c + W <= V; c += W) {
                const f32x4_t q = *reinterpret_cast<const f32x4_t*>(pf + min(int(expert(c)), E - W));
#pragma unroll
                for (int k = 0; k < W; ++k) f[c + k] = q[k];
            }
        } else {
#pragma unroll
            for (int c = 0; c + W <= V; c += W) {
                const u32x2_t q = *reinterpret_cast<const u32x2_t*>(ph + min(int(expert(c)), E - W));
#pragma unroll
                for (int k = 0; k < W; ++k) f[c + k] = __uint_as_float(k & 1 ? q[k / 2] & 0xFFFF0000u : q[k / 2] << 16);
            }
        }
    } else if (a.type == VT_F32) {
#pragma unroll
        for (int c = 0; c < V; ++c) f[c] = pf[min(int(expert(c)), E - 1)];
    } else {
#pragma unroll
        for (int c = 0; c < V; ++c) f[c] = bf16_value(ph[min(int(expert(c)), E - 1)]);
    }
#pragma unroll
    for (int c = 0; c < V; ++c)
        key[c] = live && int(expert(c)) < E && f[c] > -INFINITY ? order_key(fminf(f[c], FLT_MAX)) : 0;
    auto largest = [&]() {
        uint32_t m = key[0];
#pragma unroll
        for (int c = 1; c < V; ++c) m = max(m, key[c]);
        return row_max(m);
    };
    float sum = 0.f;
    if (!a.renorm) {
        const float top = order_value(largest());
#pragma unroll
        for (int c = 0; c < V; ++c) sum += key[c] ? expf(order_value(key[c]) - top) : 0.f;
        sum = row_sum(sum);
    }
    uint32_t my_key = 0, my_id = ~0u, top = 0;
    for (int j = 0; j < a.top_k; ++j) {
        const uint32_t m = largest(), find = max(m, 1u);   // 1 is a NaN's key: with m = 0 nothing is found
        bool has[V];
        uint32_t at = ~0u;
#pragma unroll
        for (int c = V - 1; c >= 0; --c) {
            has[c] = key[c] == find;
            at = has[c] ? expert(c) : at;
        }
        const uint32_t e = row_min(at);
        bool open = m && at == e;                          // this lane has it: its lowest one goes
#pragma unroll
        for (int c = 0; c < V; ++c) {
            key[c] = has[c] && open ? 0 : key[c];
            open = open && !has[c];
        }
        top = j == 0 ? m : top;
        if (uint32_t(j) == sub) {
            my_key = m;
            my_id = e;
        }
    }
    float w = my_key ? expf(order_value(my_key) - order_value(top)) : 0.f;
    if (a.renorm) sum = row_sum(w);
    if (live && int(sub) < a.top_k) {
        const int64_t o = t * a.top_k + sub;
        a.ids[o] = int32_t(my_id);
        a.weights[o] = my_key ? w / sum : 0.f;
        if (my_key) atomicAdd(cnt + my_id, 1u);
    }
}

// PHASE 0: everything (one block); 1: selection and the block's counts; 2:
// offsets and places.  Every block of phase 2 adds up the counts of all: 16
// bits each, so that 16-byte loads bring eight experts' and all of a thread's
// loads are on their way at once, from the kernel's first instruction on.
// V: logits a lane.
template <int PHASE, int V>
__global__ __launch_bounds__(kRT) void route_kernel(RouteArgs a) {
    __shared__ uint32_t cnt[PHASE == 1 ? 1 : kRW][kMaxExperts];     // slots of each wave, then the next place of each
    __shared__ uint32_t wave_total[kMaxExperts / 64];
    __shared__ __align__(16) uint32_t part[2][PHASE == 2 ? kRT * 8 : 1];   // (before, in all) of each group of blocks
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lane = uint32_t(tid) & 63u, sub = lane & 15u;
    const int E = a.experts, K = a.top_k, vecs = (E + 7) / 8;
    const int64_t tb = int64_t(blockIdx.x) * a.per_block;  // the block's tokens, the wave's inside them
    const int waves = PHASE == 1 ? int(blockDim.x >> 6) : kRW;
    const int64_t t_lo = tb + int64_t(wave) * (a.per_block / waves), t_hi = min(t_lo + a.per_block / waves, a.tokens);
    auto slot_id = [&](int64_t i) { return i < t_hi * K ? a.ids[i] : -1; };

    const int groups = min(kRT / vecs, 32), g = tid / vecs;                // of blocks; this thread's
    const int lo = int(int64_t(a.blocks) * g / groups), hi = g < groups ? int(int64_t(a.blocks) * (g + 1) / groups) : 0;
    const u32x4_t* const counts = reinterpret_cast<const u32x4_t*>(a.counts) + tid % vecs;
    constexpr int kFly = 8;
    u32x4_t q[kFly];
    int32_t id = -1;
    if (PHASE == 2) {
        id = slot_id(t_lo * K + lane);
#pragma unroll
        for (int i = 0; i < kFly; ++i)
            if (lo + i < hi) q[i] = counts[int64_t(lo + i) * vecs];
    }
    if (PHASE == 1) {
        for (int e = tid; e < vecs * 8; e += int(blockDim.x)) cnt[0][e] = 0;
    } else {
        for (int e = int(lane); e < E; e += 64) cnt[wave][e] = 0;
    }
    __syncthreads();
    if (PHASE != 2) {
        for (int64_t t = t_lo; t < t_hi; t += 4) {
            const int64_t mine = t + (lane >> 4);
            select<V>(a, mine < t_hi ? mine : a.tokens, sub, cnt[PHASE == 1 ? 0 : wave]);
        }
    } else {
        if (id >= 0) atomicAdd(&cnt[wave][id], 1u);
        for (int64_t i = t_lo * K + 64 + lane; i < t_hi * K; i += 64)
            if (a.ids[i] >= 0) atomicAdd(&cnt[wave][a.ids[i]], 1u);
        uint32_t bef[8] = {}, tot[8] = {};
        for (int b = lo; b < hi; b += kFly) {
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                if (b + i >= hi) continue;
                const bool before = b + i < int(blockIdx.x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t l = q[i][k] & 0xFFFFu, h = q[i][k] >> 16;
                    tot[2 * k] += l;
                    tot[2 * k + 1] += h;
                    bef[2 * k] += before ? l : 0u;
                    bef[2 * k + 1] += before ? h : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < kFly; ++i)
                if (b + kFly + i < hi) q[i] = counts[int64_t(b + kFly + i) * vecs];
        }
        if (g < groups) {
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
                *reinterpret_cast<u32x4_t*>(&part[0][tid * 8 + k]) = u32x4_t{bef[k], bef[k + 1], bef[k + 2], bef[k + 3]};
                *reinterpret_cast<u32x4_t*>(&part[1][tid * 8 + k]) = u32x4_t{tot[k], tot[k + 1], tot[k + 2], tot[k + 3]};
            }
        }
    }
    __syncthreads();
    if (PHASE == 1) {
        uint32_t* const out = reinterpret_cast<uint32_t*>(a.counts) + int64_t(blockIdx.x) * vecs * 4;
        if (tid < vecs * 4) out[tid] = cnt[0][2 * tid] | (cnt[0][2 * tid + 1] << 16);
        return;
    }

    // slots of every expert, before this block and in all; then where each
    // expert starts: a scan over the experts
    uint32_t before = 0, total = 0;
    if (PHASE == 2) {
        if (tid < E) {
#pragma unroll 8
            for (int i = 0; i < groups; ++i) {
                before += part[0][i * vecs * 8 + tid];
                total += part[1][i * vecs * 8 + tid];
            }
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
        const int32_t e = PHASE == 2 && i0 == t_lo * K ? id : slot_id(i);
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
    const int64_t end = min(tb + a.per_block, a.tokens) * K;
    for (int64_t i = tb * K + tid; i < end; i += kRT)
        if (i >= int64_t(all)) a.order[i] = -1;
}

// out[t] = sum_j weights[t][j] * Y[place[t][j]] (+ residual[t]), j ascending.
// Memory bound: four columns a lane (600 tokens of 4 experts, 2048 columns: 6.9 us).
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    const int64_t quads = (a.cols + 3) / 4, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.tokens * quads) return;
    const int64_t t = i / quads;
    const int c = int(i % quads) * 4, C = int(a.cols);
    f32x4_t v{0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.top_k; ++j) {
        const int32_t p = a.place[t * a.top_k + j];
        if (p < 0 || p >= a.n) continue;
        const f32x4_t y = load4(a.Y, VT_F32, int64_t(p) * C + c, c, C);
        const float w = a.weights[t * a.top_k + j];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = fmaf(w, y[k], v[k]);
    }
    epilogue4(Epilogue{nullptr, a.residual, a.out, a.ldr, a.ldo, VT_F32, a.residual_type, a.out_type, ACT_NONE}, t, c, C, v);
}

}  // namespace

void route_blocks(int64_t tokens, int32_t* blocks, int32_t* per_block) {
    const int64_t unit = tokens <= 64 || tokens > 64 * kMaxBlocks ? 64 : 16;
    const int64_t per = ((tokens + kMaxBlocks - 1) / kMaxBlocks + unit - 1) / unit * unit;
    *per_block = int32_t(std::min<int64_t>(std::max<int64_t>(per, unit), 65472));   // counts fit 16 bits
    const int64_t n = (tokens + *per_block - 1) / *per_block;
    *blocks = int32_t(n > 1 ? n : 1);                      // no tokens: one block writes the offsets
}

namespace {
template <int V>
hipError_t launch(const RouteArgs& a, hipStream_t s) {
    if (a.blocks == 1) {
        route_kernel<0, V><<<1, kRT, 0, s>>>(a);
        return hipGetLastError();
    }
    // four tokens a wave at a time, as many waves as the block's tokens keep busy
    route_kernel<1, V><<<unsigned(a.blocks), unsigned(std::min(kRT, a.per_block * 16)), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_kernel<2, 1><<<unsigned(a.blocks), kRT, 0, s>>>(a);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    if (a.experts <= 16) return launch<1>(a, s);
    if (a.experts <= 32) return launch<2>(a, s);
    if (a.experts <= 64) return launch<4>(a, s);
    if (a.experts <= 128) return launch<8>(a, s);
    if (a.experts <= 256) return launch<16>(a, s);
    return launch<32>(a, s);
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
    if (a.tokens <= 0 || a.cols <= 0) return hipSuccess;
    const int64_t quads = a.tokens * ((a.cols + 3) / 4), blocks = (quads + 255) / 256;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    combine_kernel<<<unsigned(blocks), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace uwk

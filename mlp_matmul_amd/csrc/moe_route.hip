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
// Or by scores, s = sigmoid(l) or softmax(l): the largest keys s + bias, of the
// groups of neighbouring experts with the best keys (below).
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
// places, bound by the latency of a chain of small steps.  By scores: 16 tokens of
// 64 experts 5.8 us; 16384 of 256 in 8 groups 24 for the selection, a third of it
// the scores' 64-bit exponentials (which every logit needs: two scores may be a
// step apart).  Workgroups of 1024 threads leave a thread 128 registers: by scores 22 of
// them spill at 256 experts and 131 at 512, by logits none and 46.
#include <float.h>

#include <algorithm>
#include <type_traits>

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

// The expert that a lane's value c is, runs of four where V allows a wide load: part(c) and the lane's own share.
template <int V>
struct Experts {
    static constexpr int W = V < 4 ? 1 : 4;
    uint32_t lane;
    __device__ __forceinline__ explicit Experts(uint32_t sub) : lane(W * sub) {}
    __device__ __forceinline__ uint32_t part(int c) const { return uint32_t(16 * W * (c / W) + c % W); }
    __device__ __forceinline__ uint32_t operator()(int c) const { return part(c) + lane; }
};
template <int V>
__device__ __forceinline__ uint32_t expert_of(int c, uint32_t sub) { return Experts<V>(sub)(c); }

// The logits of token t (one per DPP row), V a lane.  Every load stays inside
// the logits and none waits for another.
template <int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, uint32_t sub, float (&f)[V]) {
    constexpr int W = V < 4 ? 1 : 4;
    const int E = a.experts;
    const int64_t row = min(t, a.tokens - 1) * a.ld;
    const float* const pf = static_cast<const float*>(a.logits) + row;
    const uint16_t* const ph = static_cast<const uint16_t*>(a.logits) + row;
    auto expert = [&](int c) { return int(expert_of<V>(c, sub)); };
    if (W == 4 && ((a.ld | E) & 3) == 0 && (reinterpret_cast<uint64_t>(a.logits) & 15) == 0) {
        if (a.type == VT_F32) {
#pragma unroll
            for (int c = 0; c + W <= V; c += W) {
                const f32x4_t q = *reinterpret_cast<const f32x4_t*>(pf + min(expert(c), E - W));
#pragma unroll
                for (int k = 0; k < W; ++k) f[c + k] = q[k];
            }
        } else {
#pragma unroll
            for (int c = 0; c + W <= V; c += W) {
                const u32x2_t q = *reinterpret_cast<const u32x2_t*>(ph + min(expert(c), E - W));
#pragma unroll
                for (int k = 0; k < W; ++k) f[c + k] = __uint_as_float(k & 1 ? q[k / 2] & 0xFFFF0000u : q[k / 2] << 16);
            }
        }
    } else if (a.type == VT_F32) {
#pragma unroll
        for (int c = 0; c < V; ++c) f[c] = pf[min(expert(c), E - 1)];
    } else {
#pragma unroll
        for (int c = 0; c < V; ++c) f[c] = bf16_value(ph[min(expert(c), E - 1)]);
    }
}

template <int V>
__device__ __forceinline__ uint32_t largest(const uint32_t (&key)[V]) {
    uint32_t m = key[0];
#pragma unroll
    for (int c = 1; c < V; ++c) m = max(m, key[c]);
    return row_max(m);
}

struct Choice {
    uint32_t key, id, top;   // lane j's: those of the j-th chosen; the first one's key
};

// The top_k largest keys, equal ones by the lowest index(c); taken ones become 0 (in every lane that holds it, where
// several hold the same index).
template <int V, class Index>
__device__ __forceinline__ Choice choose(uint32_t (&key)[V], int top_k, uint32_t sub, const Index& index) {
    Choice r{0, ~0u, 0};
    for (int j = 0; j < top_k; ++j) {
        const uint32_t m = largest(key), find = max(m, 1u);   // 1 is a NaN's key: with m = 0 nothing is found
        bool has[V];
        uint32_t at = ~0u;
#pragma unroll
        for (int c = V - 1; c >= 0; --c) {
            has[c] = key[c] == find;
            at = has[c] ? index.part(c) : at;              // (the whole index of every value would take V registers)
        }
        at = at == ~0u ? at : at + index.lane;
        const uint32_t e = row_min(at);
        bool open = m && at == e;                          // this lane has it: its lowest one goes
#pragma unroll
        for (int c = 0; c < V; ++c) {
            key[c] = has[c] && open ? 0 : key[c];
            open = open && !has[c];
        }
        r.top = j == 0 ? m : r.top;
        if (uint32_t(j) == sub) {
            r.key = m;
            r.id = e;
        }
    }
    return r;
}

// Selects the experts of tokens t (one per DPP row; t >= tokens: nothing) and
// counts them in cnt[expert].
template <int V>
__device__ void select(const RouteArgs& a, int64_t t, uint32_t sub, uint32_t* cnt) {
    const bool live = t < a.tokens;
    uint32_t key[V];
    float f[V];
    load_logits<V>(a, t, sub, f);
#pragma unroll
    for (int c = 0; c < V; ++c)
        key[c] = live && int(expert_of<V>(c, sub)) < a.experts && f[c] > -INFINITY ? order_key(fminf(f[c], FLT_MAX)) : 0;
    float sum = 0.f;
    if (!a.renorm) {
        const float top = order_value(largest(key));
#pragma unroll
        for (int c = 0; c < V; ++c) sum += key[c] ? expf(order_value(key[c]) - top) : 0.f;
        sum = row_sum(sum);
    }
    const Choice r = choose<V>(key, a.top_k, sub, Experts<V>(sub));
    const float w = r.key ? expf(order_value(r.key) - order_value(r.top)) : 0.f;
    if (a.renorm) sum = row_sum(w);
    if (live && int(sub) < a.top_k) {
        const int64_t o = t * a.top_k + sub;
        a.ids[o] = int32_t(r.id);
        a.weights[o] = r.key ? w / sum : 0.f;
        if (r.key) atomicAdd(cnt + r.id, 1u);
    }
}

// Scores decide here, and two of them may be next to each other: they are
// computed in 64 bits and rounded to fp32 once, so that equal scores are those
// that are equal after that rounding.
__device__ __forceinline__ double row_sum64(double v) {
    auto ror = [](double x, auto n) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const uint64_t lo = row_ror<decltype(n)::value>(uint32_t(b)), hi = row_ror<decltype(n)::value>(uint32_t(b >> 32));
        return __builtin_bit_cast(double, lo | (hi << 32));
    };
    v += ror(v, std::integral_constant<int, 8>{});
    v += ror(v, std::integral_constant<int, 4>{});
    v += ror(v, std::integral_constant<int, 2>{});
    return v + ror(v, std::integral_constant<int, 1>{});
}

// exp(x) for x <= 708 (0 for those below -708, nearly), to 2^-51: x = n ln 2 + r, the Taylor sum of e^r to the 13th power
// (|r| <= 0.347, the next term is below 2^-52), times 2^n.
__device__ __forceinline__ double exp64(double x) {
    x = fmax(x, -708.0);
    const double n = rint(x * 1.4426950408889634074);
    // ln 2 as the nearest double and what that leaves: the inner product is exact within its fma
    const double r = fma(n, -2.3190468138462996e-17, fma(n, -0.6931471805599453, x));
    double y = 1.0 / 6227020800.0;
    y = fma(y, r, 1.0 / 479001600.0);
    y = fma(y, r, 1.0 / 39916800.0);
    y = fma(y, r, 1.0 / 3628800.0);
    y = fma(y, r, 1.0 / 362880.0);
    y = fma(y, r, 1.0 / 40320.0);
    y = fma(y, r, 1.0 / 5040.0);
    y = fma(y, r, 1.0 / 720.0);
    y = fma(y, r, 1.0 / 120.0);
    y = fma(y, r, 1.0 / 24.0);
    y = fma(y, r, 1.0 / 6.0);
    y = fma(y, r, 0.5);
    y = fma(y, r, 1.0);
    y = fma(y, r, 1.0);
    return ldexp(y, int(n));
}

// 1 / d for d >= 1, to 2^-52: the hardware's estimate, off by 2^-23, and two steps of Newton's.
__device__ __forceinline__ double rcp64(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = fma(fma(-d, y, 1.0), y, y);
    return fma(fma(-d, y, 1.0), y, y);
}

// Scores, rounded to fp32 once.  Beyond 110 the sigmoid is 0 or 1 there.
__device__ __forceinline__ float sigmoid_of(float l) {
    return float(rcp64(1.0 + exp64(-double(fminf(fmaxf(l, -110.f), 110.f)))));
}
__device__ __forceinline__ float softmax_of(float l, float top, double scale) { return float(exp64(double(l) - double(top)) * scale); }

// v[c] = f(v[c]) for every c, four at a time in a loop that turns the array round: unrolled, the doubles of all of them
// would spill (16384 tokens of 256 experts: 43 us).
template <int V, class F>
__device__ __forceinline__ void in_fours(float (&v)[V], F&& f) {
    constexpr int N = V < 4 ? V : 4;
#pragma unroll 1
    for (int i = 0; i < V / N; ++i) {
        float r[N];
#pragma unroll
        for (int c = 0; c < N; ++c) r[c] = f(v[c]);
#pragma unroll
        for (int c = 0; c + N < V; ++c) v[c] = v[c + N];
#pragma unroll
        for (int c = 0; c < N; ++c) v[V - N + c] = r[c];
    }
}

// The two largest of two pairs (m >= n each).
__device__ __forceinline__ void merge2(uint32_t& m, uint32_t& n, uint32_t om, uint32_t on) {
    n = max(min(m, om), max(n, on));
    m = max(m, om);
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}

// The key of a group with the two largest keys m and n (0: none).
__device__ __forceinline__ uint32_t group_key(uint32_t m, uint32_t n, int group_top) {
    if (!m) return 0;
    const float one = order_value(m);
    return order_key(fminf(n && group_top > 1 ? one + order_value(n) : one, FLT_MAX));
}

// Clears the keys outside the top_groups groups with the largest keys.
template <int V>
__device__ __forceinline__ void choose_groups(const RouteArgs& a, uint32_t (&key)[V], uint32_t sub) {
    const uint32_t per = uint32_t(a.experts / a.groups);
    constexpr int NC = V < 4 ? 1 : V / 4;
    if (V >= 4 && (per & 3u) == 0 && per <= 64 && (64u % per) == 0) {
        // a lane's runs of four each lie in one group, of `lanes` neighbouring lanes
        const uint32_t lanes = per / 4;
        uint32_t g[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            uint32_t m = max(key[4 * c], key[(4 * c + 1) % V]), n = min(key[4 * c], key[(4 * c + 1) % V]);
            const uint32_t p = key[(4 * c + 2) % V], q = key[(4 * c + 3) % V];
            merge2(m, n, max(p, q), min(p, q));
            if (lanes > 1) merge2(m, n, dpp<0xB1>(m), dpp<0xB1>(n));           // lanes 1 0 3 2
            if (lanes > 2) merge2(m, n, dpp<0x4E>(m), dpp<0x4E>(n));           // lanes 2 3 0 1
            if (lanes > 4) merge2(m, n, dpp<0x141>(m), dpp<0x141>(n));         // the other half of eight
            if (lanes > 8) merge2(m, n, dpp<0x140>(m), dpp<0x140>(n));         // the other half of sixteen
            g[c] = group_key(m, n, a.group_top);
        }
        struct {
            uint32_t per_chunk, lane;
            __device__ __forceinline__ uint32_t part(int c) const { return uint32_t(c) * per_chunk; }
        } const index{16u / lanes, sub / lanes};
        choose<NC>(g, a.top_groups, sub, index);
#pragma unroll
        for (int c = 0; c < V; ++c) key[c] = g[c / 4 % NC] ? 0 : key[c];
        return;
    }
    uint32_t mine = 0;                                     // lane g: group g's key
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
        uint32_t m = 0, n = 0;
#pragma unroll
        for (int c = 0; c < V; ++c) merge2(m, n, expert_of<V>(c, sub) - uint32_t(g) * per < per ? key[c] : 0, 0);
        merge2(m, n, row_ror<8>(m), row_ror<8>(n));
        merge2(m, n, row_ror<4>(m), row_ror<4>(n));
        merge2(m, n, row_ror<2>(m), row_ror<2>(n));
        merge2(m, n, row_ror<1>(m), row_ror<1>(n));
        if (uint32_t(g) == sub) mine = group_key(m, n, a.group_top);
    }
    uint32_t keys[1] = {mine};
    choose<1>(keys, a.top_groups, sub, Experts<1>(sub));
    const uint64_t left = __builtin_amdgcn_ballot_w64(keys[0] != 0);           // groups that were not taken, of four tokens
    const uint32_t out = uint32_t(left >> (lane_id() & 48u));
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
        if (!((out >> g) & 1u)) continue;
#pragma unroll
        for (int c = 0; c < V; ++c) key[c] = expert_of<V>(c, sub) - uint32_t(g) * per < per ? 0 : key[c];
    }
}

// select by scores: key = score + bias, groups of experts by their best keys,
// then the best keys of the chosen groups.  The weights are the scores.
template <int V>
__device__ void select_scored(const RouteArgs& a, int64_t t, uint32_t sub, uint32_t* cnt, const float* bias) {
    const bool live = t < a.tokens;
    uint32_t key[V];
    float f[V], top = 0.f;
    double scale = 1.0;
    load_logits<V>(a, t, sub, f);
#pragma unroll
    for (int c = 0; c < V; ++c)
        f[c] = live && int(expert_of<V>(c, sub)) < a.experts && f[c] > -INFINITY ? fminf(f[c], FLT_MAX) : -INFINITY;
    // scores in the logits' place, -inf where there is none
    if (a.score == SCORE_SOFTMAX) {
        float m = f[0];
#pragma unroll
        for (int c = 1; c < V; ++c) m = fmaxf(m, f[c]);
        const uint32_t k = row_max(m > -INFINITY ? order_key(m) : 0);
        top = k ? order_value(k) : 0.f;
        double sum = 0.0;
        in_fours<V>(f, [&](float l) {
            sum += l > -INFINITY ? exp64(double(l) - double(top)) : 0.0;
            return l;
        });
        scale = 1.0 / row_sum64(sum);
        in_fours<V>(f, [&](float l) { return l > -INFINITY ? softmax_of(l, top, scale) : l; });
    } else {
        in_fours<V>(f, [&](float l) { return l > -INFINITY ? sigmoid_of(l) : l; });
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const float k = f[c] + bias[expert_of<V>(c, sub)]; // behind the last expert: -inf, or no number
        key[c] = k > -INFINITY ? order_key(fminf(k, FLT_MAX)) : 0;
    }
    if (a.groups > 1) choose_groups<V>(a, key, sub);
    const Choice r = choose<V>(key, a.top_k, sub, Experts<V>(sub));
    float w = 0.f;
    if (r.key) {
        const int64_t o = t * a.ld + r.id;
        const float l = a.type == VT_F32 ? static_cast<const float*>(a.logits)[o] : bf16_value(static_cast<const uint16_t*>(a.logits)[o]);
        w = a.score == SCORE_SIGMOID ? sigmoid_of(l) : softmax_of(fminf(l, FLT_MAX), top, scale);
    }
    if (a.renorm) {                                        // fp32: nothing is chosen by it (5.3e-8 off in the norm, 3.4e-8 in 64 bits)
        const float all = row_sum(w);
        w = all > 0.f ? w / all : 0.f;                     // every chosen score may be 0
    }
    if (live && int(sub) < a.top_k) {
        const int64_t o = t * a.top_k + sub;
        a.ids[o] = int32_t(r.id);
        a.weights[o] = w * a.scale;
        if (r.key) atomicAdd(cnt + r.id, 1u);
    }
}

// PHASE 0: everything (one block); 1: selection and the block's counts; 2:
// offsets and places.  Every block of phase 2 adds up the counts of all: 16
// bits each, so that 16-byte loads bring eight experts' and all of a thread's
// loads are on their way at once, from the kernel's first instruction on.
// V: logits a lane.
template <int PHASE, int V, bool SCORED>
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
    __shared__ __align__(16) float bias[SCORED ? kMaxExperts : 1];
    if (SCORED) {
        for (int e = tid; e < E; e += int(blockDim.x)) bias[e] = a.bias ? a.bias[e] : 0.f;
    }
    __syncthreads();
    if (PHASE != 2) {
        for (int64_t t = t_lo; t < t_hi; t += 4) {
            const int64_t mine = t + (lane >> 4);
            uint32_t* const counts_of = cnt[PHASE == 1 ? 0 : wave];
            if constexpr (SCORED) select_scored<V>(a, mine < t_hi ? mine : a.tokens, sub, counts_of, bias);
            else select<V>(a, mine < t_hi ? mine : a.tokens, sub, counts_of);
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
template <int V, bool SCORED>
hipError_t launch(const RouteArgs& a, hipStream_t s) {
    if (a.blocks == 1) {
        route_kernel<0, V, SCORED><<<1, kRT, 0, s>>>(a);
        return hipGetLastError();
    }
    // four tokens a wave at a time, as many waves as the block's tokens keep busy
    route_kernel<1, V, SCORED><<<unsigned(a.blocks), unsigned(std::min(kRT, a.per_block * 16)), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_kernel<2, 1, false><<<unsigned(a.blocks), kRT, 0, s>>>(a);
    return hipGetLastError();
}
}  // namespace

namespace {
template <bool SCORED>
hipError_t launch_width(const RouteArgs& a, hipStream_t s) {
    if (a.experts <= 16) return launch<1, SCORED>(a, s);
    if (a.experts <= 32) return launch<2, SCORED>(a, s);
    if (a.experts <= 64) return launch<4, SCORED>(a, s);
    if (a.experts <= 128) return launch<8, SCORED>(a, s);
    if (a.experts <= 256) return launch<16, SCORED>(a, s);
    return launch<32, SCORED>(a, s);
}
}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    return a.score == SCORE_LOGIT ? launch_width<false>(a, s) : launch_width<true>(a, s);
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
    if (a.tokens <= 0 || a.cols <= 0) return hipSuccess;
    const int64_t quads = a.tokens * ((a.cols + 3) / 4), blocks = (quads + 255) / 256;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    combine_kernel<<<unsigned(blocks), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace uwk

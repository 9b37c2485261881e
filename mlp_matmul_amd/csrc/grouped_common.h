// Device helpers of the products grouped by expert: which rows a workgroup
// multiplies, and the epilogue.
#pragma once

#include "device_common.h"
#include "experts.h"

namespace uwk {

// Rows [row0, row0 + rows) of expert e against weight rows of band `band`.
struct GroupTile {
    int32_t e, rows, band, slice;    // slice: of K, with a.split
    int64_t row0;
};

// Work unit `id` of `total` in an order that gives each XCD (workgroup id % 8)
// a contiguous run of units.
__device__ __forceinline__ uint32_t spread_unit(uint32_t total, uint32_t id) {
    const uint32_t xcd = id & 7u, q = total >> 3, r = total & 7u;
    return xcd * q + min(xcd, r) + (id >> 3);
}

// group_tile with offsets, CH * 64 experts at most: expert 64*c + lane of
// chunk c in this lane.  All loads go out together.
template <int NT, int CH>
__device__ __forceinline__ bool group_tile_of(const GroupArgs& a, uint32_t bands, GroupTile& t) {
    const int lane = int(lane_id());
    const int32_t n = int32_t(a.n);
    int32_t o0[CH], o1[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e = 64 * c + lane;
        o0[c] = a.offsets[min(e, a.E)];
        o1[c] = a.offsets[min(e + 1, a.E)];                // past the last expert: no rows
    }
    uint32_t lo[CH], rows[CH], end[CH];                    // first row, rows, tiles up to and with the expert's
    uint32_t total = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int32_t s = min(max(o0[c], 0), n), f = min(max(o1[c], s), n);
        lo[c] = uint32_t(s);
        rows[c] = 64 * c + lane < a.E ? uint32_t(f - s) : 0u;
        uint32_t incl = (rows[c] + NT - 1) / NT;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(incl, d, 64);
            if (lane >= d) incl += o;
        }
        end[c] = total + incl;
        total += uint32_t(__builtin_amdgcn_readlane(int(incl), 63));
    }
    const uint64_t units = uint64_t(total) * bands;        // below 2^31 where the grid is (overlapping offsets: more)
    if (blockIdx.x >= units) return false;
    const uint32_t u = spread_unit(uint32_t(min(units, uint64_t(gridDim.x))), blockIdx.x);
    const uint32_t tile = u / bands;                       // never past the last: u < total * bands
    bool found = false;
    t.slice = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const uint64_t past = __builtin_amdgcn_ballot_w64(end[c] > tile);
        if (found || !past) continue;
        found = true;
        const int l = __builtin_ctzll(past);
        const uint32_t nr = uint32_t(__builtin_amdgcn_readlane(int(rows[c]), l));
        const uint32_t first = uint32_t(__builtin_amdgcn_readlane(int(lo[c]), l));
        const uint32_t tiles = (nr + NT - 1) / NT;
        const uint32_t before = uint32_t(__builtin_amdgcn_readlane(int(end[c]), l)) - tiles;
        const uint32_t local = u - before * bands;
        t.e = 64 * c + l;
        t.band = int32_t(local / tiles);
        const uint32_t i = local % tiles;
        t.row0 = int64_t(first) + int64_t(i) * NT;
        t.rows = int32_t(min(uint32_t(NT), nr - i * NT));
    }
    return found;
}

// The unit of work of this workgroup: tiles of NT rows of every expert with
// rows, times `bands` bands of its weight rows, token tiles of a band next to
// each other (they read the same weights); false past the last one.  The grid
// holds the most there can be, the host does not know the offsets.  Offsets
// out of order or out of range are clamped, so no row outside [0, n) is
// touched.  Every wave finds the unit by itself: no barrier.
template <int NT>
__device__ __forceinline__ bool group_tile(const GroupArgs& a, uint32_t bands, GroupTile& t) {
    if (!a.offsets) {
        const uint32_t tiles = uint32_t((a.n + NT - 1) / NT), total = tiles * bands * uint32_t(a.split);
        if (blockIdx.x >= total) return false;
        const uint32_t u = spread_unit(total, blockIdx.x);
        t.e = 0;
        t.slice = int32_t(u / (tiles * bands));
        t.band = int32_t(u / tiles % bands);
        t.row0 = int64_t(u % tiles) * NT;
        t.rows = int32_t(min(int64_t(NT), a.n - t.row0));
        return true;
    }
    return a.E <= 64 ? group_tile_of<NT, 1>(a, bands, t) : group_tile_of<NT, kMaxExperts / 64>(a, bands, t);
}

// Most units a grid needs: every expert with rows has at most n_e/NT + 1 tiles.
inline int64_t group_units(const GroupArgs& a, int nt, int64_t bands) {
    if (!a.offsets) return (a.n + nt - 1) / nt * bands * a.split;
    return (a.n / nt + (a.n < a.E ? a.n : a.E)) * bands;
}

// The X row that sorted row s reads (an index outside X reads its row 0).
__device__ __forceinline__ const uint16_t* group_x_row(const GroupArgs& a, int64_t s) {
    int64_t r = s;
    if (a.order) {
        const int32_t o = a.order[s];
        r = o < 0 ? 0 : int64_t(uint32_t(o) / uint32_t(a.div));
        if (r >= a.x_rows) r = 0;
    }
    return a.X + r * a.ldx;
}

// 16 bytes a lane from memory to LDS; lane i's land at dst + 16 i.
__device__ __forceinline__ void dma16(const void* src, void* dst) {
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Waits until at most N vector memory operations are pending; LDS: and for every
// LDS operation.
template <int N, bool LDS>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (LDS ? 0 : 15 << 8));
}

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// x / (1 + exp(-x)) from the hardware's base-2 exponential and reciprocal, each
// within one unit in the last place.  The rounding of -x log2(e), and of log2(e),
// moves the exponent by 1.225 |x| 2^-24: no more than x off by 1.225 half steps
// would, which the fp32 sum that x is already is off by.  So the result, to (1.225 |x| +
// 6) 2^-24 of itself, is SiLU of a neighbour of x; an exponential without that error would
// take twice the instructions.  From x = -87.3 down exp(-x) passes 2^126 and the
// result may be 0 (its size is below 2^-119).
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case ACT_RELU: return v < 0.f ? 0.f : v;           // NaN stays
        case ACT_SILU: return silu(v);
        // (1 + erf cancels where v is below -2: within 3 min(|v|, 6) 2^-24)
        case ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        // 1 + tanh(u) = 2 / (1 + exp(-2u)), without the cancellation that tanh near
        // -1 has: within (8 |2u| + 6) 2^-24 of the result
        case ACT_GELU_TANH:
            return v * __builtin_amdgcn_rcpf(
                1.0f + __builtin_amdgcn_exp2f(-2.0f * 1.4426950408889634f * 0.79788456080286536f * fmaf(0.044715f * v * v, v, v)));
        default: return v;
    }
}

// The same for 4 N values, the choice made once.
template <int N>
__device__ __forceinline__ void activate_all(f32x4_t (&v)[N], int act) {
    auto each = [&](auto&& f) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k][j] = f(v[k][j]);
    };
    switch (act) {
        case ACT_RELU: each([](float x) { return activate(x, ACT_RELU); }); break;
        case ACT_SILU: each([](float x) { return activate(x, ACT_SILU); }); break;
        case ACT_GELU: each([](float x) { return activate(x, ACT_GELU); }); break;
        case ACT_GELU_TANH: each([](float x) { return activate(x, ACT_GELU_TANH); }); break;
        default: break;
    }
}

// Four elements that need not be aligned to four: the hardware takes any
// multiple of the element.
typedef uint32_t u32x2_e2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_e4_t __attribute__((ext_vector_type(4), aligned(4)));

// Four values of rows r .. r+3 from p[o..], of either type; those from R on are 0.
__device__ __forceinline__ f32x4_t load4(const void* p, int type, int64_t o, int r, int R) {
    f32x4_t v{0.f, 0.f, 0.f, 0.f};
    if (r + 3 < R) {
        if (type == VT_F32)
            return __builtin_bit_cast(f32x4_t, u32x4_t(*reinterpret_cast<const u32x4_e4_t*>(static_cast<const float*>(p) + o)));
        const u32x2_t q = *reinterpret_cast<const u32x2_e2_t*>(static_cast<const uint16_t*>(p) + o);
        return f32x4_t{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xFFFF0000u), __uint_as_float(q[1] << 16),
                       __uint_as_float(q[1] & 0xFFFF0000u)};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < R)
            v[i] = type == VT_F32 ? static_cast<const float*>(p)[o + i] : bf16_value(static_cast<const uint16_t*>(p)[o + i]);
    return v;
}

// Four values to rows r .. r+3, those below R.
__device__ __forceinline__ void store4(void* p, int type, int64_t o, int r, int R, f32x4_t v) {
    if (type == VT_BF16) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f32_to_bf16_rne(v[i]);
        uint16_t* const d = static_cast<uint16_t*>(p) + o;
        if (r + 3 < R) {
            *reinterpret_cast<u32x2_e2_t*>(d) = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) d[i] = uint16_t(h[i]);
        }
    } else {
        float* const d = static_cast<float*>(p) + o;
        if (r + 3 < R) {
            *reinterpret_cast<u32x4_e4_t*>(d) = __builtin_bit_cast(u32x4_t, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) d[i] = v[i];
        }
    }
}

// What the epilogue of weight rows r .. r+3 (those below R) and output row b
// reads.
struct EpilogueIn {
    f32x4_t bias, residual;
};

__device__ __forceinline__ EpilogueIn epilogue_load(const Epilogue& ep, int64_t b, int r, int R) {
    EpilogueIn in{};
    if (ep.bias) in.bias = load4(ep.bias, ep.bias_type, r, r, R);
    if (ep.residual) in.residual = load4(ep.residual, ep.residual_type, b * ep.ldr + r, r, R);
    return in;
}

// Bias, activation, residual, and the one rounding to the output's type.
__device__ __forceinline__ void epilogue_store(const Epilogue& ep, const EpilogueIn& in, int64_t b, int r, int R,
                                               f32x4_t v) {
    if (ep.bias) v += in.bias;
    if (ep.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(v[i], ep.act);
    }
    if (ep.residual) v += in.residual;
    store4(ep.out, ep.out_type, b * ep.ldo + r, r, R, v);
}

// The epilogue of a tile from LDS, in parts of `kIn` input rows by `kRows`
// weight rows (floats at part[n * ES + r]) that `kThreads` threads share, four
// elements of a row a lane.  A lane's weight rows are the same in every item and
// part, so that its bias is loaded once, and residuals of the next part are on
// their way while this one is stored.
template <int kRows, int kIn, int kThreads, int ES>
struct PartEpilogue {
    static constexpr int kItems = kRows * kIn / 4 / kThreads;
    static_assert(kItems >= 1 && kItems * 4 * kThreads == kRows * kIn && kThreads % (kRows / 4) == 0, "whole items");
    const Epilogue& ep;
    const float* const part;
    const int64_t first;                                     // the tile's first output row
    const int rows, r, R, tid;                               // its output rows, the lane's first weight row
    f32x4_t bias;
    u32x4_t res[kItems];                                     // as loaded: a conversion would wait for them

    __device__ __forceinline__ PartEpilogue(const Epilogue& e, const float* p, const GroupTile& t, uint32_t row0, int R_,
                                            int tid_)
        : ep(e), part(p), first(t.row0), rows(t.rows), r(int(row0) + tid_ % (kRows / 4) * 4), R(R_), tid(tid_),
          bias{0.f, 0.f, 0.f, 0.f} {
        if (ep.bias) bias = load4(ep.bias, ep.bias_type, r, r, R);
    }
    __device__ __forceinline__ int input_row(int k) const { return (tid + k * kThreads) / (kRows / 4); }
    __device__ __forceinline__ f32x4_t value(int k) const {
        return *reinterpret_cast<const f32x4_t*>(part + input_row(k) * ES + tid % (kRows / 4) * 4);
    }

    // row(n): input row n of the part in the tile
    template <class Row>
    __device__ __forceinline__ void load(Row&& row) {
        if (!ep.residual || r + 3 >= R) return;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int b = row(input_row(k));
            const int64_t o = (first + b) * ep.ldr + r;
            if (b >= rows) continue;
            if (ep.residual_type == VT_F32) {
                res[k] = *reinterpret_cast<const u32x4_e4_t*>(static_cast<const float*>(ep.residual) + o);
            } else {
                const u32x2_t h = *reinterpret_cast<const u32x2_e2_t*>(static_cast<const uint16_t*>(ep.residual) + o);
                res[k] = u32x4_t{h[0], h[1], 0u, 0u};
            }
        }
    }
    // stores the part with the residuals that were loaded for it, and loads the
    // next one's: row of this part, next of the next
    template <class Row, class Next>
    __device__ __forceinline__ void store(Row&& row, bool more, Next&& next) {
        if (r + 3 >= R) return store_last(row);
        f32x4_t v[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) v[k] = value(k) + bias;
        activate_all(v, ep.act);
        if (ep.residual) {
#pragma unroll
            for (int k = 0; k < kItems; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[k][j] += __uint_as_float(ep.residual_type == VT_F32 ? res[k][j]
                                               : j & 1                    ? res[k][j >> 1] & 0xFFFF0000u
                                                                          : res[k][j >> 1] << 16);
        }
        if (more) load(next);
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int b = row(input_row(k));
            if (b < rows) store4(ep.out, ep.out_type, (first + b) * ep.ldo + r, r, R, v[k]);
        }
    }
    // the lanes of the last weight rows, fewer than four
    template <class Row>
    __device__ __forceinline__ void store_last(Row&& row) {
#pragma unroll 1
        for (int k = 0; k < kItems; ++k) {
            const int b = row(input_row(k));
            if (b < rows && r < R) epilogue_store(ep, epilogue_load(ep, first + b, r, R), first + b, r, R, value(k));
        }
    }
};

__device__ __forceinline__ void epilogue4(const Epilogue& ep, int64_t b, int r, int R, f32x4_t v) {
    epilogue_store(ep, epilogue_load(ep, b, r, R), b, r, R, v);
}

}  // namespace uwk

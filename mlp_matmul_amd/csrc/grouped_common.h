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

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case ACT_RELU: return v < 0.f ? 0.f : v;           // NaN stays
        case ACT_SILU: return v / (1.0f + expf(-v));
        case ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
        case ACT_GELU_TANH: return 0.5f * v * (1.0f + tanhf(0.79788456080286536f * fmaf(0.044715f * v * v, v, v)));
        default: return v;
    }
}

// Four values of rows r .. r+3 from p[r..], of either type; those from R on are 0.
__device__ __forceinline__ f32x4_t load4(const void* p, int type, int64_t o, int r, int R, bool aligned) {
    f32x4_t v{0.f, 0.f, 0.f, 0.f};
    if (aligned && r + 3 < R) {
        if (type == VT_F32) return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + o);
        const u32x2_t q = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + o);
        return f32x4_t{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xFFFF0000u), __uint_as_float(q[1] << 16),
                       __uint_as_float(q[1] & 0xFFFF0000u)};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < R)
            v[i] = type == VT_F32 ? static_cast<const float*>(p)[o + i] : bf16_value(static_cast<const uint16_t*>(p)[o + i]);
    return v;
}

// What the epilogue of weight rows r .. r+3 (those below R) and output row b
// reads.
struct EpilogueIn {
    f32x4_t bias, residual;
};

__device__ __forceinline__ EpilogueIn epilogue_load(const Epilogue& ep, int64_t b, int r, int R) {
    EpilogueIn in{};
    if (ep.bias) in.bias = load4(ep.bias, ep.bias_type, r, r, R, true);
    if (ep.residual) in.residual = load4(ep.residual, ep.residual_type, b * ep.ldr + r, r, R, (ep.ldr & 3) == 0);
    return in;
}

// Bias, activation, residual, and the one rounding to the output's type;
// vector stores where rows are 4-element aligned.
__device__ __forceinline__ void epilogue_store(const Epilogue& ep, const EpilogueIn& in, int64_t b, int r, int R,
                                               f32x4_t v) {
    const bool whole = r + 3 < R && (ep.ldo & 3) == 0;
    if (ep.bias) v += in.bias;
    if (ep.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(v[i], ep.act);
    }
    if (ep.residual) v += in.residual;
    const int64_t o = b * ep.ldo + r;
    if (ep.out_type == VT_BF16) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f32_to_bf16_rne(v[i]);
        uint16_t* p = static_cast<uint16_t*>(ep.out) + o;
        if (whole) {
            *reinterpret_cast<u32x2_t*>(p) = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) p[i] = uint16_t(h[i]);
        }
    } else {
        float* p = static_cast<float*>(ep.out) + o;
        if (whole) {
            *reinterpret_cast<f32x4_t*>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) p[i] = v[i];
        }
    }
}

__device__ __forceinline__ void epilogue4(const Epilogue& ep, int64_t b, int r, int R, f32x4_t v) {
    epilogue_store(ep, epilogue_load(ep, b, r, R), b, r, R, v);
}

}  // namespace uwk

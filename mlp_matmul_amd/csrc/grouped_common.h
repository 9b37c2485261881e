// Device helpers of the products grouped by expert: which rows a workgroup
// multiplies, and the epilogue.
#pragma once

#include "device_common.h"
#include "experts.h"

namespace uwk {

// Rows [row0, row0 + rows) of expert e against weight rows of band `band`.
struct GroupTile {
    int32_t e, rows, band;
    int64_t row0;
};

// The unit of work of this workgroup: tiles of NT rows of every expert with
// rows, times `bands` bands of its weight rows, token tiles of a band next to
// each other (they read the same weights).  Units are numbered so that each
// XCD (workgroup id % 8) takes a contiguous run of those there are; false
// past the last one.  The grid holds the most there can be, the host does
// not know the offsets.  Offsets out of order or out of range are clamped,
// so no row outside [0, n) is touched.  Every wave finds the unit by itself
// (64 experts at a time, one a lane): no barrier.
template <int NT>
__device__ __forceinline__ bool group_tile(const GroupArgs& a, uint32_t bands, GroupTile& t) {
    auto spread = [](uint32_t total, uint32_t id) {
        const uint32_t xcd = id & 7u, q = total >> 3, r = total & 7u;
        return xcd * q + min(xcd, r) + (id >> 3);
    };
    if (!a.offsets) {
        const uint32_t tiles = uint32_t((a.n + NT - 1) / NT), total = tiles * bands;
        if (blockIdx.x >= total) return false;
        const uint32_t u = spread(total, blockIdx.x);
        t.e = 0;
        t.band = int32_t(u / tiles);
        t.row0 = int64_t(u % tiles) * NT;
        t.rows = int32_t(min(int64_t(NT), a.n - t.row0));
        return true;
    }
    constexpr int kChunks = kMaxExperts / 64;
    const int lane = int(lane_id()), chunks = (a.E + 63) / 64;
    uint32_t lo[kChunks], cnt[kChunks], end[kChunks];      // first row, tiles, tiles up to and with
    uint32_t total = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        lo[c] = cnt[c] = 0;
        if (c >= chunks) continue;
        const int e = 64 * c + lane;
        const int32_t n = int32_t(a.n);
        const int32_t o0 = e < a.E ? a.offsets[e] : 0, o1 = e < a.E ? a.offsets[e + 1] : 0;
        const int32_t s = min(max(o0, 0), n), f = min(max(o1, s), n);
        lo[c] = uint32_t(s);
        cnt[c] = uint32_t(f - s);                          // rows; tiles below
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        end[c] = total;
        if (c >= chunks) continue;
        uint32_t incl = (cnt[c] + NT - 1) / NT;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(incl, d, 64);
            if (lane >= d) incl += o;
        }
        end[c] = total + incl;
        total += uint32_t(__builtin_amdgcn_readlane(int(incl), 63));
    }
    const uint64_t units = uint64_t(total) * bands;
    if (blockIdx.x >= units) return false;
    const uint32_t u = spread(uint32_t(units), blockIdx.x);
    bool found = false;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (c >= chunks || found) continue;
        const uint64_t past = __builtin_amdgcn_ballot_w64(uint64_t(end[c]) * bands > u);
        if (!past) continue;
        found = true;
        const int l = __builtin_ctzll(past);
        const uint32_t rows = uint32_t(__builtin_amdgcn_readlane(int(cnt[c]), l));
        const uint32_t first = uint32_t(__builtin_amdgcn_readlane(int(lo[c]), l));
        const uint32_t tiles = (rows + NT - 1) / NT;
        const uint32_t before = uint32_t(__builtin_amdgcn_readlane(int(end[c]), l)) - tiles;
        const uint32_t local = u - before * bands;
        t.e = 64 * c + l;
        t.band = int32_t(local / tiles);
        const uint32_t i = local % tiles;
        t.row0 = int64_t(first) + int64_t(i) * NT;
        t.rows = int32_t(min(uint32_t(NT), rows - i * NT));
    }
    return found;
}

// Most units a grid needs: every expert with rows has at most n_e/NT + 1 tiles.
inline int64_t group_units(const GroupArgs& a, int nt, int64_t bands) {
    if (!a.offsets) return (a.n + nt - 1) / nt * bands;
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

// Four weight rows r .. r+3 (those below R) of output row b: bias,
// activation, residual, one rounding to the output's type.  The bias is
// `bias` (fp32) already; vector accesses where rows are 4-element aligned.
__device__ __forceinline__ void epilogue4(const Epilogue& ep, int64_t b, int r, int R, f32x4_t v) {
    const bool whole = r + 3 < R;
    if (ep.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ri = r + i < R ? r + i : R - 1;
            v[i] += ep.bias_type == VT_BF16 ? bf16_value(static_cast<const uint16_t*>(ep.bias)[ri])
                                            : static_cast<const float*>(ep.bias)[ri];
        }
    }
    if (ep.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(v[i], ep.act);
    }
    if (ep.residual) {
        const int64_t o = b * ep.ldr + r;
        if (ep.residual_type == VT_BF16) {
            const uint16_t* p = static_cast<const uint16_t*>(ep.residual) + o;
            if (whole && (ep.ldr & 3) == 0) {
                const u32x2_t q = *reinterpret_cast<const u32x2_t*>(p);
                v += f32x4_t{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xFFFF0000u),
                             __uint_as_float(q[1] << 16), __uint_as_float(q[1] & 0xFFFF0000u)};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + i < R) v[i] += bf16_value(p[i]);
            }
        } else {
            const float* p = static_cast<const float*>(ep.residual) + o;
            if (whole && (ep.ldr & 3) == 0) {
                v += *reinterpret_cast<const f32x4_t*>(p);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + i < R) v[i] += p[i];
            }
        }
    }
    const int64_t o = b * ep.ldo + r;
    if (ep.out_type == VT_BF16) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f32_to_bf16_rne(v[i]);
        uint16_t* p = static_cast<uint16_t*>(ep.out) + o;
        if (whole && (ep.ldo & 3) == 0) {
            *reinterpret_cast<u32x2_t*>(p) = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) p[i] = uint16_t(h[i]);
        }
    } else {
        float* p = static_cast<float*>(ep.out) + o;
        if (whole && (ep.ldo & 3) == 0) {
            *reinterpret_cast<f32x4_t*>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) p[i] = v[i];
        }
    }
}

}  // namespace uwk

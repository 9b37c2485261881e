// One or two rows per expert (a single token, or a batch of one or two of the
// epilogue matmul): the weight stream bounds the product, there is nothing to
// reuse, so a weight goes from memory to registers, is rebuilt there and
// multiplied with v_dot2 (two bf16 products, fp32 sum).
//
// A wave owns whole rows of the expert's matrix (of gate and up: the same row
// of both) and walks them in slabs of 1024 columns, 16 a lane; every load
// instruction reads one contiguous run.  The items (row, slab) run through a
// ring of D register sets: D items are in flight, the loop has no branch
// around a load.  The input rows are staged in LDS once per workgroup of four
// waves.  A row's 64 lane sums are added by a butterfly: the order is fixed.
// Verbatim groups: a wave keeps the bitmap word and the base of every tile its
// rows touch, one tile a lane; an item picks its 16 flags by lane reads, so
// flags and slots cost scalar instructions, and the raw exponents come with
// the item's other loads (lanes outside verbatim groups share one line).
//   Measured: gate/up of one token, two experts of 3584 x 4096, palette, 17.7 us
// for 90 MB, the read rate but for 3 us of launch and first loads; 1024 x 4096
// 5.4 us, nothing but those; bf16, one row of 14336 x 4096, 19.7 us for 117 MB.
#include "grouped_common.h"
#include "kernels.h"

namespace uwk {

namespace {

constexpr int kSlab = 1024;
constexpr int kGemvWaves = 4;

template <bool PAL>
struct Item {
    u32x4_t a, b;       // bf16: the halves; palette: a.xy indices, b sign/mantissa
    u32x4_t vx;         // palette: raw exponents
    uint32_t verb;
};

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int l) {
    return (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(v >> 32), l))) << 32) |
           uint32_t(__builtin_amdgcn_readlane(int(uint32_t(v)), l));
}

// The item's 16 weights as bf16 pairs; `lut` maps two indices to both exponents in place.
template <bool PAL>
__device__ __forceinline__ void item_weights(const Item<PAL>& it, const char* lut, uint32_t w[8]) {
    if (!PAL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = it.a[i];
            w[4 + i] = it.b[i];
        }
        return;
    }
    uint32_t e7[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e7[i] = *reinterpret_cast<const uint32_t*>(lut + (((it.a[i >> 2] >> (8 * (i & 3))) & 0xFFu) << 2));
    if (__builtin_amdgcn_ballot_w64(it.verb != 0)) {         // rare: raw exponents for verbatim lanes
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t raw = (i & 1) ? exp_pair<1>(it.vx[i >> 1]) : exp_pair<0>(it.vx[i >> 1]);
            e7[i] = it.verb ? raw : e7[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = (i & 1) ? join_pair<1>(it.b[i >> 1], e7[i]) : join_pair<0>(it.b[i >> 1], e7[i]);
}

// Zeros for the columns from `left` on of a slab (their inputs are zeros too).
template <bool PAL>
__device__ __forceinline__ void cut_weights(uint32_t left, int lane, uint32_t w[8]) {
    const bool z0 = PAL ? uint32_t(lane) * 16u >= left : uint32_t(lane) * 8u >= left;
    const bool z1 = PAL ? z0 : 512u + uint32_t(lane) * 8u >= left;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = z0 ? 0u : w[i];
        w[4 + i] = z1 ? 0u : w[4 + i];
    }
}

// s plus the item's products with the staged inputs of its two halves.
__device__ __forceinline__ float item_dot(const uint32_t w[8], const uint16_t* x, float s) {
    const u32x4_t x0 = load16(x), x1 = load16(x + 512);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = dot2_bf16(w[i], x0[i], s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = dot2_bf16(w[4 + i], x1[i], s);
    return s;
}

template <bool PAL, bool PAIR, int NB, int D>
__global__ __launch_bounds__(64 * kGemvWaves) void gemv_rows_kernel(GroupArgs a, uint32_t bands, int rows_per_wave) {
    constexpr int M = PAIR ? 2 : 1;
    __shared__ uint32_t lut[PAL ? 256 * M : 1];
    extern __shared__ __align__(16) uint16_t xs[];           // [NB][slabs * 1024]
    GroupTile t;
    if (!group_tile<NB>(a, bands, t)) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t R = uint32_t(a.R), C = uint32_t(a.C), slabs = (C + kSlab - 1) / kSlab;
    const uint32_t r0 = (uint32_t(t.band) * kGemvWaves + uint32_t(wave)) * uint32_t(rows_per_wave);
    // a wave past the matrix walks its last row and stores nothing
    const uint32_t my_rows = r0 < R ? min(uint32_t(rows_per_wave), R - r0) : 0u;
    const uint32_t rl = min(r0, R - 1u), total = max(my_rows, 1u) * slabs * M;
    const int64_t first = int64_t(t.e) * R * C;

    // verbatim tables of the wave's rows
    const int64_t g0 = (first + int64_t(rl) * C) >> 6;       // the first row's first group
    const int64_t t0 = g0 >> 6;
    uint64_t word[M];
    uint32_t base[M], ebase[M];
    if (PAL) {
        const int64_t tl = (g0 + int64_t(max(my_rows, 1u)) * (C >> 6) - 1) >> 6;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            word[m] = a.w[m].bitmap[min(t0 + lane, tl)];
            base[m] = a.w[m].tile_vbase[min(t0 + lane, tl)];
            ebase[m] = min(a.w[m].tile_vbase[first >> 12], a.w[m].last_slot);
        }
    }
    float bias = 0.f, residual[NB] = {};                     // of the next row to finish; lane 0 uses them

    struct Pos {
        uint32_t row, m, s;                                  // row from rl, matrix, slab
    };
    auto next = [&](Pos p) -> Pos {
        if (p.s + 1 < slabs) return {p.row, p.m, p.s + 1};
        if (PAIR && p.m == 0) return {p.row, 1u, 0u};
        return {p.row + 1, 0u, 0u};
    };
    const uint32_t lane16 = uint32_t(lane) * 16u;
    auto issue = [&](Pos p, Item<PAL>& it) {
        const Weight& w = PAIR && p.m ? a.w[M - 1] : a.w[0];
        const uint64_t pos = uint64_t(first) + uint64_t(rl + p.row) * C + p.s * kSlab;   // uniform
        const uint32_t left = C - p.s * kSlab;               // columns of the slab, 1024 or fewer
        if (!PAL) {
            const uint16_t* const b = static_cast<const uint16_t*>(w.w) + pos;
            const uint32_t k0 = uint32_t(lane) * 8u, k1 = 512u + k0;
            it.a = load_stream16(b + (k0 < left ? k0 : 0u));
            it.b = load_stream16(b + (k1 < left ? k1 : 0u));
            return;
        }
        const uint32_t k = lane16 < left ? lane16 : 0u;
        const u32x2_t n = load_stream8(static_cast<const uint8_t*>(w.w) + pos / 2 + k / 2);
        it.a = u32x4_t{n[0], n[1], 0u, 0u};
        it.b = load_stream16(w.sm + pos + k);
        // flags of the slab's 16 groups: uniform
        const uint32_t gi = uint32_t(int64_t(pos >> 6) - (t0 << 6)), tl = gi >> 6, gb = gi & 63u;
        const uint64_t mw = PAIR && p.m ? word[M - 1] : word[0];
        const uint32_t mb = PAIR && p.m ? base[M - 1] : base[0];
        const uint64_t w0 = readlane64(mw, int(tl));
        uint64_t bits = w0 >> gb;
        if (gb > 48u) bits |= readlane64(mw, int(min(tl + 1u, 63u))) << (64u - gb);
        // groups behind the row's end are other rows' (clamped lanes look at group 0)
        const uint32_t m16 = uint32_t(bits) & 0xFFFFu;
        const uint32_t start = uint32_t(__builtin_amdgcn_readlane(int(mb), int(tl))) -
                               (PAIR && p.m ? ebase[M - 1] : ebase[0]) +
                               uint32_t(__popcll(gb ? w0 & ((uint64_t(1) << gb) - 1) : 0));
        const uint32_t grp = k >> 6;
        it.verb = (m16 >> grp) & 1u;
        const uint32_t slot = start + uint32_t(__popc(m16 & ((1u << grp) - 1u)));
        const uint8_t* const vb = w.vexp + uint64_t(PAIR && p.m ? ebase[M - 1] : ebase[0]) * 64u;
        it.vx = load16(vb + (it.verb ? slot * 64u + (k & 63u) : 0u));
    };

    constexpr int NS = D + 1;                                // register sets: D items in flight past the one computed
    Item<PAL> ring[NS];
    Pos at[NS], last{0, 0, 0};
    // loads first: the input rows' addresses and the tables wait for other loads
    if (!PAL) {
        Pos p{0, 0, 0};
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (d > 0 && uint32_t(d) < total) p = next(p);
            at[d] = p;
            issue(p, ring[d]);
        }
        last = p;
    }
    if (PAL) {
#pragma unroll
        for (int m = 0; m < M; ++m)
            lut[256 * m + tid] = (pal_byte(a.w[m].pal, uint32_t(tid) & 15u) << 7) |
                                 (pal_byte(a.w[m].pal, uint32_t(tid) >> 4) << 23);
    }
    // input rows to LDS, zeros behind C; palette: the two halves of a lane's 16
    // columns 64 chunks apart, so that both are conflict-free 16-byte reads
    const uint32_t chunks = C / 8u, all = slabs * (kSlab / 8);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint16_t* const x = group_x_row(a, t.row0 + (b < t.rows ? b : 0));
        for (uint32_t c = uint32_t(tid); c < all; c += 64u * kGemvWaves) {
            const u32x4_t v = c < chunks ? load16(x + c * 8u) : u32x4_t{0u, 0u, 0u, 0u};
            const uint32_t in = c & 127u, to = PAL ? (c & ~127u) + (in & 1u) * 64u + (in >> 1) : c;
            store16(xs + (uint32_t(b) * all + to) * 8u, v);
        }
    }
    if (PAL) {
        Pos p{0, 0, 0};
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (d > 0 && uint32_t(d) < total) p = next(p);
            at[d] = p;
            issue(p, ring[d]);
        }
        last = p;
    }
    auto load_ends = [&](uint32_t row) {
        const uint32_t r = min(rl + row, R - 1u);
        if (a.ep.bias)
            bias = a.ep.bias_type == VT_F32 ? static_cast<const float*>(a.ep.bias)[r]
                                            : bf16_value(static_cast<const uint16_t*>(a.ep.bias)[r]);
        if (a.ep.residual) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int64_t o = (t.row0 + (b < t.rows ? b : 0)) * a.ep.ldr + r;
                residual[b] = a.ep.residual_type == VT_F32 ? static_cast<const float*>(a.ep.residual)[o]
                                                           : bf16_value(static_cast<const uint16_t*>(a.ep.residual)[o]);
            }
        }
    };
    if (!PAIR) load_ends(0);
    __syncthreads();

    float acc[NB], gate[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = gate[b] = 0.f;

    auto compute = [&](Pos p, const Item<PAL>& it) {
        uint32_t w[8];
        item_weights<PAL>(it, reinterpret_cast<const char*>(lut) + (PAIR && p.m ? 1024u : 0u), w);
        const uint32_t left = C - p.s * kSlab;
        if (left < uint32_t(kSlab)) cut_weights<PAL>(left, lane, w);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[b] = item_dot(w, xs + (uint32_t(b) * all + p.s * 128u + uint32_t(lane)) * 8u, acc[b]);
        if (p.s + 1 < slabs) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float v = wave_sum(acc[b]);
            acc[b] = 0.f;
            if (PAIR) {
                if (p.m == 0) {
                    gate[b] = v;
                    continue;
                }
                v = silu(gate[b]) * v;
            }
            if (lane == 0 && b < t.rows && p.row < my_rows) {
                if (a.ep.bias) v += bias;
                v = activate(v, a.ep.act);
                if (a.ep.residual) v += residual[b];
                const int64_t o = (t.row0 + b) * a.ep.ldo + r0 + p.row;
                if (a.ep.out_type == VT_BF16) static_cast<uint16_t*>(a.ep.out)[o] = uint16_t(f32_to_bf16_rne(v));
                else static_cast<float*>(a.ep.out)[o] = v;
            }
        }
        if (!PAIR && p.row + 1 < my_rows) load_ends(p.row + 1);
    };

    uint32_t done = 0;
    for (; done + NS <= total; done += NS) {
#pragma unroll
        for (int d = 0; d < NS; ++d) {
            // items past the end read the last one again
            if (done + uint32_t(d) + D < total) last = next(last);
            at[(d + D) % NS] = last;
            issue(last, ring[(d + D) % NS]);
            compute(at[d], ring[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < NS - 1; ++d)
        if (done + uint32_t(d) < total) compute(at[d], ring[d]);
}

// One token's down projection with the weighted sum of its experts:
//   out[r] = sum_j weights[j] * (D_e(j)[r] . h[place[j]]) (+ residual[r])
// A wave owns an output row and walks that row of every chosen expert's matrix
// in turn, so the sum stays in its registers: no array of the experts' outputs
// and no launch that adds it (a layer of one token, two of 8 experts of 3584 x
// 4096, palette: 32.4 us; with a launch for each 2.6 more).  Items, ring and rebuild
// as above; lane j*tiles + i keeps the verbatim word and base of tile i of expert j's row.
template <bool PAL, int D>
__global__ __launch_bounds__(64 * kGemvWaves) void gemv_combine_kernel(GroupArgs a, CombineArgs c) {
    __shared__ uint32_t lut[PAL ? 256 : 1];
    extern __shared__ __align__(16) uint16_t xs[];           // [chosen][slabs * 1024]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t R = uint32_t(a.R), C = uint32_t(a.C), slabs = (C + kSlab - 1) / kSlab;
    const uint32_t row = min(blockIdx.x * kGemvWaves + uint32_t(wave), R - 1u);
    const bool mine = blockIdx.x * kGemvWaves + uint32_t(wave) < R;

    // the chosen experts, in lane j; those without one come last
    const int32_t lj = min(lane, c.top_k - 1);
    const int32_t id = c.ids[lj], pl = c.place[lj];
    const float wt = c.weights[lj];
    const bool real = lane < c.top_k && id >= 0 && id < a.E && pl >= 0 && pl < c.n;
    const uint64_t some = __builtin_amdgcn_ballot_w64(real);
    const uint32_t chosen = uint32_t(__builtin_ctzll(~some)), total = chosen * slabs;
    auto expert = [&](uint32_t j) -> uint32_t { return uint32_t(__builtin_amdgcn_readlane(id, int(j))); };
    auto first_of = [&](uint32_t e) -> uint64_t { return uint64_t(e) * R * C; };

    const Weight& w = a.w[0];
    const uint32_t tiles = (C + 4095) / 4096 + 1;            // of a row, at most
    uint64_t word = 0;
    uint32_t base = 0, ebase = 0;
    if (PAL) {
        const uint32_t j = min(uint32_t(lane) / tiles, uint32_t(c.top_k) - 1u);
        const int32_t ej = __shfl(id, int(j));
        const uint64_t g = (first_of(uint32_t(ej < 0 || ej >= a.E ? 0 : ej)) + uint64_t(row) * C) >> 6;
        const uint64_t tl = min((g >> 6) + uint32_t(lane) % tiles, (g + (C >> 6) - 1) >> 6);
        word = w.bitmap[tl];
        base = w.tile_vbase[tl];
        ebase = min(w.tile_vbase[first_of(uint32_t(id < 0 || id >= a.E ? 0 : id)) >> 12], w.last_slot);   // lane j: expert j's
        lut[tid] = (pal_byte(w.pal, uint32_t(tid) & 15u) << 7) | (pal_byte(w.pal, uint32_t(tid) >> 4) << 23);
    }
    struct Pos {
        uint32_t j, s;
    };
    auto next = [&](Pos p) -> Pos { return p.s + 1 < slabs ? Pos{p.j, p.s + 1} : Pos{p.j + 1, 0u}; };
    const uint32_t lane16 = uint32_t(lane) * 16u;
    auto issue = [&](Pos p, Item<PAL>& it) {
        const uint64_t pos = first_of(expert(p.j)) + uint64_t(row) * C + p.s * kSlab;    // uniform
        const uint32_t left = C - p.s * kSlab;
        if (!PAL) {
            const uint16_t* const b = static_cast<const uint16_t*>(w.w) + pos;
            const uint32_t k0 = uint32_t(lane) * 8u, k1 = 512u + k0;
            it.a = load_stream16(b + (k0 < left ? k0 : 0u));
            it.b = load_stream16(b + (k1 < left ? k1 : 0u));
            return;
        }
        const uint32_t k = lane16 < left ? lane16 : 0u;
        const u32x2_t n = load_stream8(static_cast<const uint8_t*>(w.w) + pos / 2 + k / 2);
        it.a = u32x4_t{n[0], n[1], 0u, 0u};
        it.b = load_stream16(w.sm + pos + k);
        const uint64_t row_tile = (pos - p.s * kSlab) >> 12;
        const uint32_t gi = uint32_t((pos >> 6) - (row_tile << 6)), tl = p.j * tiles + (gi >> 6), gb = gi & 63u;
        const uint64_t w0 = readlane64(word, int(tl));
        uint64_t bits = w0 >> gb;
        if (gb > 48u) bits |= readlane64(word, int(min(tl + 1u, p.j * tiles + tiles - 1u))) << (64u - gb);
        const uint32_t m16 = uint32_t(bits) & 0xFFFFu;
        const uint32_t eb = uint32_t(__builtin_amdgcn_readlane(int(ebase), int(p.j)));
        const uint32_t start = uint32_t(__builtin_amdgcn_readlane(int(base), int(tl))) - eb +
                               uint32_t(__popcll(gb ? w0 & ((uint64_t(1) << gb) - 1) : 0));
        const uint32_t grp = k >> 6;
        it.verb = (m16 >> grp) & 1u;
        const uint32_t slot = start + uint32_t(__popc(m16 & ((1u << grp) - 1u)));
        it.vx = load16(w.vexp + uint64_t(eb) * 64u + (it.verb ? slot * 64u + (k & 63u) : 0u));
    };

    constexpr int NS = D + 1;
    Item<PAL> ring[NS];
    Pos at[NS], last{0, 0};
    if (total) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (d > 0 && uint32_t(d) < total) last = next(last);
            at[d] = last;
            issue(last, ring[d]);
        }
    }
    const uint32_t chunks = C / 8u, all = slabs * (kSlab / 8);
    for (uint32_t j = 0; j < chosen; ++j) {
        const uint16_t* const x = a.X + int64_t(__builtin_amdgcn_readlane(pl, int(j))) * a.ldx;
        for (uint32_t i = uint32_t(tid); i < all; i += 64u * kGemvWaves) {
            const u32x4_t v = i < chunks ? load16(x + i * 8u) : u32x4_t{0u, 0u, 0u, 0u};
            const uint32_t in = i & 127u, to = PAL ? (i & ~127u) + (in & 1u) * 64u + (in >> 1) : i;
            store16(xs + (j * all + to) * 8u, v);
        }
    }
    float residual = 0.f;
    if (c.residual)
        residual = c.residual_type == VT_F32 ? static_cast<const float*>(c.residual)[row]
                                             : bf16_value(static_cast<const uint16_t*>(c.residual)[row]);
    __syncthreads();

    float acc = 0.f, sum = 0.f;
    auto compute = [&](Pos p, const Item<PAL>& it) {
        uint32_t v[8];
        item_weights<PAL>(it, reinterpret_cast<const char*>(lut), v);
        const uint32_t left = C - p.s * kSlab;
        if (left < uint32_t(kSlab)) cut_weights<PAL>(left, lane, v);
        acc = item_dot(v, xs + (p.j * all + p.s * 128u + uint32_t(lane)) * 8u, acc);
        if (p.s + 1 < slabs) return;
        sum = fmaf(__uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(wt)), int(p.j)))),
                   wave_sum(acc), sum);
        acc = 0.f;
    };
    uint32_t done = 0;
    for (; done + NS <= total; done += NS) {
#pragma unroll
        for (int d = 0; d < NS; ++d) {
            if (done + uint32_t(d) + D < total) last = next(last);
            at[(d + D) % NS] = last;
            issue(last, ring[(d + D) % NS]);
            compute(at[d], ring[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < NS - 1; ++d)
        if (done + uint32_t(d) < total) compute(at[d], ring[d]);
    if (lane == 0 && mine) {
        if (c.residual) sum += residual;
        if (c.out_type == VT_BF16) static_cast<uint16_t*>(c.out)[row] = uint16_t(f32_to_bf16_rne(sum));
        else static_cast<float*>(c.out)[row] = sum;
    }
}

// The input rows of a workgroup fit 48 KB of LDS: 24 slabs.  So do the tables of a
// wave's tiles its 64 lanes: those of two rows in a run, or of a row of every
// chosen expert, each with a tile that another row has a part of.
constexpr int kStagedSlabs = 24;
static_assert(2 * kStagedSlabs * kSlab / 4096 + 1 <= 64 && 2 * kStagedSlabs <= 64, "tiles fit the lanes");

// Rows of a wave: one, or two on tall matrices (a wave's start is paid for half
// as often; single matrices only, 65536 x 4096: 65 us against 77).
int rows_of_wave(const GroupArgs& a, bool pair) { return !pair && a.R >= 8192 ? 2 : 1; }

size_t staged_bytes(const GroupArgs& a, int nb) { return size_t(nb) * ((a.C + kSlab - 1) / kSlab) * kSlab * 2; }

// Two items in flight; one for the palette pair and for two input rows, where
// the registers of the second cost more waves than it gains (palette pair, two
// experts of 3584 x 4096: 20.0 us against 21.9).
template <bool PAL, bool PAIR, int NB>
hipError_t launch(const GroupArgs& a, hipStream_t s) {
    constexpr int D = NB > 1 || (PAL && PAIR) ? 1 : 2;
    const int rpw = rows_of_wave(a, PAIR);
    const int64_t bands = (a.R + kGemvWaves * rpw - 1) / (kGemvWaves * rpw);
    const int64_t units = group_units(a, NB, bands);
    if (units > 0x7FFFFFFF) return hipErrorInvalidValue;
    launch_timed(gemv_rows_kernel<PAL, PAIR, NB, D>, dim3(unsigned(units)), dim3(64 * kGemvWaves), staged_bytes(a, NB),
                 s, a, uint32_t(bands), rpw);
    return hipGetLastError();
}

}  // namespace

bool gemv_rows_supported(const GroupArgs& a, int nb) { return staged_bytes(a, nb) <= size_t(kStagedSlabs) * kSlab * 2; }

hipError_t launch_gemv_rows(bool pal, bool pair, const GroupArgs& a, int nb, hipStream_t s) {
    if (nb == 1)
        return pal ? (pair ? launch<true, true, 1>(a, s) : launch<true, false, 1>(a, s))
                   : (pair ? launch<false, true, 1>(a, s) : launch<false, false, 1>(a, s));
    return pal ? (pair ? launch<true, true, 2>(a, s) : launch<true, false, 2>(a, s))
               : (pair ? launch<false, true, 2>(a, s) : launch<false, false, 2>(a, s));
}

bool gemv_combine_supported(const GroupArgs& a, int top_k) { return gemv_rows_supported(a, top_k); }

hipError_t launch_gemv_combine(bool pal, const GroupArgs& a, const CombineArgs& c, hipStream_t s) {
    const dim3 grid(unsigned((a.R + kGemvWaves - 1) / kGemvWaves)), block(64 * kGemvWaves);
    if (pal) launch_timed(gemv_combine_kernel<true, 2>, grid, block, staged_bytes(a, c.top_k), s, a, c);
    else launch_timed(gemv_combine_kernel<false, 2>, grid, block, staged_bytes(a, c.top_k), s, a, c);
    return hipGetLastError();
}

}  // namespace uwk

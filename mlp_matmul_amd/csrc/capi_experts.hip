// C ABI entry points of the epilogue matmul and of the mixture-of-experts
// operators: argument checks, scratch layout and composition.  See unweight.h
// for the contract.
#include <algorithm>
#include <exception>
#include <utility>

#include "capi_common.h"
#include "experts.h"

using uw::align256;
using uw::aligned16;
using uw::as_stream;
using uw::fail;
using uw::hip_fail;

namespace {

// No C++ exception leaves an entry point (the error text itself allocates).
template <class F>
int guarded(F&& f) noexcept {
    try {
        uw::clear_error();
        return f();
    } catch (const std::exception&) {
        return UW_ENOMEM;
    }
}

int bad(const char* who, const char* what) { return fail(UW_EINVAL, std::string(who) + ": " + what); }

bool value_type(int t) { return t == UW_F32 || t == UW_BF16; }
int64_t value_bytes(int t) { return t == UW_BF16 ? 2 : 4; }

// Bytes from the first to behind the last element of [rows, cols] with row stride ld.
uint64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
    return rows > 0 && cols > 0 ? (uint64_t(rows - 1) * uint64_t(ld) + uint64_t(cols)) * uint64_t(bytes) : 0;
}

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// Memory that a call reads (or writes).
struct Inputs {
    struct {
        const void* p;
        uint64_t bytes;
    } span[24];
    int count = 0;

    void add(const void* p, uint64_t bytes) {
        if (p && bytes) span[count++] = {p, bytes};
    }
    bool meet(const void* p, uint64_t bytes) const {
        for (int i = 0; i < count; ++i)
            if (overlap(p, bytes, span[i].p, span[i].bytes)) return true;
        return false;
    }
};

// The weight of an operator: exactly one of w (bf16) and d (compressed, with
// its NIB section), [experts*rows, cols].
int take_weight(const uint16_t* w, const uw_dmat* d, int64_t experts, int64_t rows, int64_t cols, uwk::Weight* out,
                Inputs* in, const char* who) {
    *out = uwk::Weight{};
    if (rows < 0 || cols < uw::kGroup || cols % uw::kGroup)
        return bad(who, "bad shape (cols must be a positive multiple of 64)");
    if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) || rows * cols >= (int64_t(1) << 31))
        return fail(UW_EUNSUPPORTED, std::string(who) + ": a matrix of 2^31 weights or more");
    if (rows == 0 && !d) return UW_OK;
    if ((w != nullptr) == (d != nullptr)) return bad(who, "give a bf16 weight or a compressed one, and not both");
    if (w) {
        if (!aligned16(w)) return bad(who, "misaligned weight");
        in->add(w, uint64_t(experts * rows * cols) * 2);
        out->w = w;
        return UW_OK;
    }
    int rc = uw::check_dmat(d, who);
    if (rc) return rc;
    if (d->rows != experts * rows || d->cols != cols)
        return bad(who, "the compressed matrix is not [experts*rows, cols]");
    if (d->groups && (!d->nib || !d->sm || !d->bitmap || !d->tile_vbase || (d->verbatim_groups && !d->vexp)))
        return bad(who, "the compressed matrix lacks its NIB/SM/BITMAP/TILE_VBASE/VEXP sections");
    if (!aligned16(d->nib) || !aligned16(d->sm) || !aligned16(d->vexp) || !aligned16(d->bitmap) ||
        !aligned16(d->tile_vbase))
        return bad(who, "misaligned section of the compressed matrix");
    in->add(d->nib, uint64_t(d->groups) * 32);
    in->add(d->sm, uint64_t(d->groups) * 64);
    in->add(d->vexp, uint64_t(d->verbatim_groups) * 64);
    in->add(d->bitmap, uint64_t(d->tiles) * 8);
    in->add(d->tile_vbase, uint64_t(d->tiles + 1) * 4);
    out->w = d->nib;
    out->sm = d->sm;
    out->vexp = uw::vexp_of(d) ? d->vexp : d->sm;   // never read as exponents without verbatim groups
    out->bitmap = d->bitmap;
    out->tile_vbase = d->tile_vbase;
    uw::pack_palette(d->palette, out->pal);
    out->last_slot = d->verbatim_groups ? uint32_t(d->verbatim_groups) - 1 : 0;
    return UW_OK;
}

int check_rows(const void* p, int64_t ld, int64_t cols, int64_t multiple, const char* who, const char* name) {
    if (!p || !aligned16(p)) return fail(UW_EINVAL, std::string(who) + ": NULL or misaligned " + name);
    if (ld < cols || ld % multiple || ld >= (int64_t(1) << 40))
        return fail(UW_EINVAL, std::string(who) + ": bad row stride of " + name);
    return UW_OK;
}

// out (and the residual it may replace) against what the call reads while out is written.
int check_epilogue(const uwk::Epilogue& e, int64_t n, int64_t rows, const Inputs& in, const char* who) {
    if (!value_type(e.out_type) || (e.bias && !value_type(e.bias_type)) || (e.residual && !value_type(e.residual_type)))
        return bad(who, "a value type is neither UW_F32 nor UW_BF16");
    if (e.act < 0 || e.act >= uwk::ACT_COUNT) return bad(who, "unknown activation");
    int rc = check_rows(e.out, e.ldo, rows, 1, who, "out");
    if (rc) return rc;
    if (e.residual && (rc = check_rows(e.residual, e.ldr, rows, 1, who, "residual"))) return rc;
    if (e.bias && !aligned16(e.bias)) return bad(who, "misaligned bias");
    const uint64_t ob = span(n, rows, e.ldo, value_bytes(e.out_type));
    if (in.meet(e.out, ob)) return bad(who, "out overlaps an input");
    if (e.residual && overlap(e.out, ob, e.residual, span(n, rows, e.ldr, value_bytes(e.residual_type))) &&
        (e.out != e.residual || e.ldo != e.ldr || e.out_type != e.residual_type))
        return bad(who, "out overlaps the residual without being it");
    return UW_OK;
}

// Optional scratch, which no input, residual or output may lie in.
int check_scratch(const void* scratch, uint64_t* bytes, const uwk::Epilogue& e, int64_t n, int64_t rows,
                  const Inputs& in, const char* who) {
    if (!aligned16(scratch)) return bad(who, "misaligned scratch");
    if (!scratch) *bytes = 0;
    if (overlap(e.out, span(n, rows, e.ldo, value_bytes(e.out_type)), scratch, *bytes) || in.meet(scratch, *bytes) ||
        (e.residual && overlap(e.residual, span(n, rows, e.ldr, value_bytes(e.residual_type)), scratch, *bytes)))
        return bad(who, "the scratch overlaps an input or out");
    return UW_OK;
}

int check_groups(int experts, int64_t n, const int32_t* offsets, const int32_t* order, int top_k, int64_t x_rows,
                 const char* who) {
    if (experts < 1 || experts > uwk::kMaxExperts) return bad(who, "experts must be 1..512");
    if (n < 0 || x_rows < 0 || n >= (int64_t(1) << 31) || x_rows >= (int64_t(1) << 31))
        return bad(who, "bad number of rows");
    if (top_k < 1) return bad(who, "top_k must be at least 1");
    if (n == 0) return UW_OK;
    if (!offsets || !aligned16(offsets) || !aligned16(order)) return bad(who, "NULL or misaligned offsets or order");
    if (order ? x_rows == 0 : x_rows < n) return bad(who, "X has too few rows");
    return UW_OK;
}

// What a grouped call reads beside its weights.
void add_rows(Inputs* in, const uwk::GroupArgs& a) {
    in->add(a.X, span(a.x_rows, a.C, a.ldx, 2));
    in->add(a.offsets, uint64_t(a.E + 1) * 4);
    in->add(a.order, uint64_t(a.n) * 4);
}

uwk::GroupArgs group_args(const uint16_t* X, int64_t x_rows, int64_t ldx, const int32_t* offsets, const int32_t* order,
                          int top_k, int64_t n, int64_t experts, int64_t rows, int64_t cols) {
    uwk::GroupArgs a{};
    a.X = X;
    a.offsets = offsets;
    a.order = order;
    a.ldx = ldx;
    a.x_rows = x_rows;
    a.n = n;
    a.E = int32_t(experts);
    a.R = int32_t(rows);
    a.C = int32_t(cols);
    a.div = top_k;
    a.split = 1;
    a.cus = uw::device_cus();
    return a;
}

// Scratch of a routing call with more than one block of tokens.
uint64_t route_scratch(int64_t tokens, int64_t experts) {
    int32_t blocks, per;
    uwk::route_blocks(tokens, &blocks, &per);
    return blocks > 1 ? align256(uint64_t(blocks) * uint64_t((experts + 7) / 8) * 16) : 0;
}

int check_routing(int64_t tokens, int experts, int top_k, const char* who) {
    if (tokens < 0 || tokens >= (int64_t(1) << 31)) return bad(who, "bad number of tokens");
    if (experts < 1 || experts > uwk::kMaxExperts) return bad(who, "experts must be 1..512");
    if (top_k < 1 || top_k > uwk::kMaxTopK || top_k > experts) return bad(who, "top_k must be 1..16 and at most experts");
    if (tokens * top_k >= (int64_t(1) << 31)) return bad(who, "tokens * top_k must be below 2^31");
    return UW_OK;
}

// Scratch of a whole layer.
struct LayerLayout {
    uint64_t ids, weights, offsets, order, place, route, h, y, total;   // total: what a call cannot do without
    uint64_t expand;                                                    // behind it: room for expanded weights
};

LayerLayout layer_layout(bool pal, int64_t tokens, int experts, int64_t top_k, int64_t F, int64_t H) {
    LayerLayout l{};
    const uint64_t slots = uint64_t(tokens) * uint64_t(top_k);
    uint64_t off = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t at = off;
        off += align256(bytes);
        return at;
    };
    l.ids = take(slots * 4);
    l.weights = take(slots * 4);
    l.offsets = take(uint64_t(experts + 1) * 4);
    l.order = take(slots * 4);
    l.place = take(slots * 4);
    l.route = take(route_scratch(tokens, experts));
    // bf16, as uw_mlp_layer's: the type that the instructions that multiply it take (MFMA, and v_dot2
    // for a single token, which a second bf16 term would double), alike for every number of tokens so
    // that a token's result does not change with its batch.  At most half a step, 2^-8, of each h:
    // 0.0017 of the experts' sum in the norm, what rounding the output to bf16 costs too
    l.h = take(slots * uint64_t(F) * 2);
    l.y = take(slots * uint64_t(H) * 4);
    l.total = off;
    l.expand = std::max(uwk::grouped_scratch(pal, true, experts, F, H, int64_t(slots), uw::device_cus()),
                        uwk::grouped_scratch(pal, false, experts, H, F, int64_t(slots), uw::device_cus()));
    return l;
}

}  // namespace

extern "C" {

int64_t uw_linear_scratch_bytes(int compressed, int64_t rows, int64_t cols, int64_t batch) {
    int64_t out = 0;
    const int rc = guarded([&]() -> int {
        const char* who = "uw_linear_scratch_bytes";
        if (rows < 0 || cols < uw::kGroup || batch < 0 || batch >= (int64_t(1) << 31) || cols % uw::kGroup)
            return bad(who, "bad argument (cols must be a positive multiple of 64)");
        if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) || rows * cols >= (int64_t(1) << 31))
            return fail(UW_EUNSUPPORTED, std::string(who) + ": a matrix of 2^31 weights or more");
        out = int64_t(uwk::linear_scratch(compressed != 0, rows, cols, batch, uw::device_cus()));
        return UW_OK;
    });
    return rc ? rc : out;
}

int uw_linear(const uint16_t* w, const uw_dmat* d, int64_t rows, int64_t cols, const uint16_t* X, int64_t ldx,
              int64_t batch, const void* bias, int bias_type, int act, const void* residual, int residual_type,
              int64_t ldr, void* out, int out_type, int64_t ldo, void* scratch, uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_linear";
        uwk::GroupArgs a = group_args(X, batch, ldx, nullptr, nullptr, 1, batch, 1, rows, cols);
        Inputs in;
        int rc = take_weight(w, d, 1, rows, cols, &a.w[0], &in, who);
        if (rc) return rc;
        if (batch < 0 || batch >= (int64_t(1) << 31)) return bad(who, "bad batch");
        if (rows == 0 || batch == 0) return UW_OK;
        if ((rc = check_rows(X, ldx, cols, 8, who, "X"))) return rc;
        a.ep = {bias, residual, out, ldr, ldo, bias_type, residual_type, out_type, act};
        in.add(X, span(batch, cols, ldx, 2));
        in.add(bias, uint64_t(rows) * value_bytes(bias_type));
        if ((rc = check_epilogue(a.ep, batch, rows, in, who))) return rc;
        if ((rc = check_scratch(scratch, &scratch_bytes, a.ep, batch, rows, in, who))) return rc;
        const hipError_t e = uwk::launch_linear(d != nullptr, a, scratch, scratch_bytes, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int64_t uw_moe_route_scratch_bytes(int64_t tokens, int experts, int top_k) {
    int64_t out = 0;
    const int rc = guarded([&]() -> int {
        int r = check_routing(tokens, experts, top_k, "uw_moe_route_scratch_bytes");
        if (r) return r;
        out = int64_t(route_scratch(tokens, experts));
        return UW_OK;
    });
    return rc ? rc : out;
}

int uw_moe_route(const void* logits, int logits_type, int64_t ld, int64_t tokens, int experts, int top_k,
                 int renormalize, int32_t* ids, float* weights, int32_t* offsets, int32_t* order, int32_t* place,
                 void* scratch, uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_moe_route";
        int rc = check_routing(tokens, experts, top_k, who);
        if (rc) return rc;
        if (!value_type(logits_type)) return bad(who, "logits are UW_F32 or UW_BF16");
        if (!offsets || !aligned16(offsets)) return bad(who, "NULL or misaligned offsets");
        if (tokens) {
            if ((rc = check_rows(logits, ld, experts, 1, who, "logits"))) return rc;
            for (const void* p : {static_cast<const void*>(ids), static_cast<const void*>(weights),
                                  static_cast<const void*>(order), static_cast<const void*>(place)})
                if (!p || !aligned16(p)) return bad(who, "NULL or misaligned output");
        }
        const uint64_t need = route_scratch(tokens, experts);
        if (need && (!scratch || !aligned16(scratch) || scratch_bytes < need))
            return bad(who, "scratch smaller than uw_moe_route_scratch_bytes()");
        // every block reads its logits while others write: nothing shares memory
        const uint64_t slots = uint64_t(tokens) * uint64_t(top_k) * 4;
        const std::pair<const void*, uint64_t> writes[] = {{ids, slots},   {weights, slots}, {offsets, uint64_t(experts + 1) * 4},
                                                           {order, slots}, {place, slots},   {scratch, need}};
        Inputs others;
        others.add(logits, span(tokens, experts, ld, value_bytes(logits_type)));
        for (const auto& w : writes) {
            if (others.meet(w.first, w.second)) return bad(who, "an output or the scratch overlaps another or the logits");
            others.add(w.first, w.second);
        }
        uwk::RouteArgs a{logits, ld,  tokens,  logits_type, experts, top_k, renormalize != 0, ids, weights,
                         offsets, order, place, static_cast<uint16_t*>(scratch), 0, 0};
        uwk::route_blocks(tokens, &a.blocks, &a.per_block);
        const hipError_t e = uwk::launch_route(a, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int64_t uw_grouped_scratch_bytes(int compressed, int pair, int experts, int64_t rows, int64_t cols, int64_t n) {
    int64_t out = 0;
    const int rc = guarded([&]() -> int {
        const char* who = "uw_grouped_scratch_bytes";
        if (experts < 1 || experts > uwk::kMaxExperts) return bad(who, "experts must be 1..512");
        if (rows < 0 || cols < uw::kGroup || n < 0 || n >= (int64_t(1) << 31) || cols % uw::kGroup)
            return bad(who, "bad argument (cols must be a positive multiple of 64)");
        if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) || rows * cols >= (int64_t(1) << 31))
            return fail(UW_EUNSUPPORTED, std::string(who) + ": a matrix of 2^31 weights or more");
        out = int64_t(uwk::grouped_scratch(compressed != 0, pair != 0, experts, rows, cols, n, uw::device_cus()));
        return UW_OK;
    });
    return rc ? rc : out;
}

int uw_gemm_grouped(const uint16_t* w, const uw_dmat* d, int experts, int64_t rows, int64_t cols, const uint16_t* X,
                    int64_t x_rows, int64_t ldx, const int32_t* offsets, const int32_t* order, int top_k, int64_t n,
                    void* out, int out_type, int64_t ldo, void* scratch, uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_gemm_grouped";
        int rc = check_groups(experts, n, offsets, order, top_k, x_rows, who);
        if (rc) return rc;
        uwk::GroupArgs a = group_args(X, x_rows, ldx, offsets, order, top_k, n, experts, rows, cols);
        Inputs in;
        if ((rc = take_weight(w, d, experts, rows, cols, &a.w[0], &in, who))) return rc;
        if (rows == 0 || n == 0) return UW_OK;
        if ((rc = check_rows(X, ldx, cols, 8, who, "X"))) return rc;
        a.ep = {nullptr, nullptr, out, 0, ldo, UW_F32, UW_F32, out_type, UW_ACT_NONE};
        add_rows(&in, a);
        if ((rc = check_epilogue(a.ep, n, rows, in, who))) return rc;
        if ((rc = check_scratch(scratch, &scratch_bytes, a.ep, n, rows, in, who))) return rc;
        const hipError_t e = uwk::launch_grouped(d != nullptr, false, a, scratch, scratch_bytes, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int uw_moe_gate_up(const uint16_t* gate_w, const uw_dmat* gate_d, const uint16_t* up_w, const uw_dmat* up_d,
                   int experts, int64_t rows, int64_t cols, const uint16_t* X, int64_t x_rows, int64_t ldx,
                   const int32_t* offsets, const int32_t* order, int top_k, int64_t n, uint16_t* h, int64_t ldh,
                   void* scratch, uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_moe_gate_up";
        int rc = check_groups(experts, n, offsets, order, top_k, x_rows, who);
        if (rc) return rc;
        uwk::GroupArgs a = group_args(X, x_rows, ldx, offsets, order, top_k, n, experts, rows, cols);
        Inputs in;
        if ((rc = take_weight(gate_w, gate_d, experts, rows, cols, &a.w[0], &in, who))) return rc;
        if ((rc = take_weight(up_w, up_d, experts, rows, cols, &a.w[1], &in, who))) return rc;
        if ((gate_d != nullptr) != (up_d != nullptr)) return bad(who, "gate and up must both be bf16 or both compressed");
        if (rows == 0 || n == 0) return UW_OK;
        if ((rc = check_rows(X, ldx, cols, 8, who, "X"))) return rc;
        a.ep = {nullptr, nullptr, h, 0, ldh, UW_F32, UW_F32, UW_BF16, UW_ACT_NONE};
        add_rows(&in, a);
        if ((rc = check_epilogue(a.ep, n, rows, in, who))) return rc;
        if ((rc = check_scratch(scratch, &scratch_bytes, a.ep, n, rows, in, who))) return rc;
        const hipError_t e = uwk::launch_grouped(gate_d != nullptr, true, a, scratch, scratch_bytes, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int uw_moe_combine(const float* Y, int64_t n, int64_t cols, const int32_t* place, const float* weights, int64_t tokens,
                   int top_k, const void* residual, int residual_type, int64_t ldr, void* out, int out_type,
                   int64_t ldo, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_moe_combine";
        if (n < 0 || cols < 0 || tokens < 0 || n >= (int64_t(1) << 31) || tokens >= (int64_t(1) << 31) ||
            cols >= (int64_t(1) << 31))
            return bad(who, "bad shape");
        if (top_k < 1 || top_k > uwk::kMaxTopK) return bad(who, "top_k must be 1..16");
        if (tokens == 0 || cols == 0) return UW_OK;
        if ((n && (!Y || !aligned16(Y))) || !place || !weights || !aligned16(place) || !aligned16(weights))
            return bad(who, "NULL or misaligned Y, place or weights");
        const uwk::Epilogue ep{nullptr, residual, out, ldr, ldo, UW_F32, residual_type, out_type, UW_ACT_NONE};
        Inputs in;
        in.add(Y, span(n, cols, cols, 4));
        in.add(place, uint64_t(tokens) * top_k * 4);
        in.add(weights, uint64_t(tokens) * top_k * 4);
        int rc = check_epilogue(ep, tokens, cols, in, who);
        if (rc) return rc;
        const uwk::CombineArgs a{Y, place, nullptr, weights, n, cols, tokens, top_k, residual, out, ldr, ldo,
                                 residual_type, out_type};
        const hipError_t e = uwk::launch_combine(a, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int64_t uw_moe_scratch_bytes(int compressed, int64_t tokens, int experts, int top_k, int64_t rows, int64_t cols) {
    int64_t out = 0;
    const int rc = guarded([&]() -> int {
        const char* who = "uw_moe_scratch_bytes";
        int r = check_routing(tokens, experts, top_k, who);
        if (r) return r;
        if (rows < uw::kGroup || cols < uw::kGroup || rows % uw::kGroup || cols % uw::kGroup)
            return bad(who, "rows and cols must be positive multiples of 64");
        if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) || rows * cols >= (int64_t(1) << 31))
            return fail(UW_EUNSUPPORTED, std::string(who) + ": a matrix of 2^31 weights or more");
        const LayerLayout l = layer_layout(compressed != 0, tokens, experts, top_k, rows, cols);
        out = int64_t(l.total + l.expand);
        return UW_OK;
    });
    return rc ? rc : out;
}

int uw_moe_layer(const uint16_t* gate_w, const uw_dmat* gate_d, const uint16_t* up_w, const uw_dmat* up_d,
                 const uint16_t* down_w, const uw_dmat* down_d, int experts, int64_t rows, int64_t cols,
                 const uint16_t* X, int64_t ldx, int64_t tokens, const void* logits, int logits_type, int64_t ldl,
                 int top_k, int renormalize, const void* residual, int residual_type, int64_t ldr, void* out,
                 int out_type, int64_t ldo, void* scratch, uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_moe_layer";
        int rc = check_routing(tokens, experts, top_k, who);
        if (rc) return rc;
        if (rows < uw::kGroup || cols < uw::kGroup || rows % uw::kGroup || cols % uw::kGroup)
            return bad(who, "gate and up are [rows, cols], down [cols, rows], rows and cols positive multiples of 64");
        uwk::Weight probe, down;
        Inputs in;
        if ((rc = take_weight(gate_w, gate_d, experts, rows, cols, &probe, &in, who)) ||
            (rc = take_weight(up_w, up_d, experts, rows, cols, &probe, &in, who)) ||
            (rc = take_weight(down_w, down_d, experts, cols, rows, &down, &in, who)))
            return rc;
        if ((gate_d != nullptr) != (up_d != nullptr)) return bad(who, "gate and up must both be bf16 or both compressed");
        if (tokens == 0) return UW_OK;
        if ((rc = check_rows(X, ldx, cols, 8, who, "X")) || (rc = check_rows(logits, ldl, experts, 1, who, "logits")))
            return rc;
        if (!value_type(logits_type)) return bad(who, "logits are UW_F32 or UW_BF16");
        // out is written by the last step alone, which reads down: it may be X or the residual
        const uwk::Epilogue ep{nullptr, residual, out, ldr, ldo, UW_F32, residual_type, out_type, UW_ACT_NONE};
        if ((rc = check_epilogue(ep, tokens, cols, in, who))) return rc;
        const LayerLayout l = layer_layout(gate_d || down_d, tokens, experts, top_k, rows, cols);
        if (!scratch || !aligned16(scratch) || scratch_bytes < l.total)
            return bad(who, "scratch smaller than uw_moe_scratch_bytes()");
        in.add(X, span(tokens, cols, ldx, 2));
        in.add(logits, span(tokens, experts, ldl, value_bytes(logits_type)));
        if ((rc = check_scratch(scratch, &scratch_bytes, ep, tokens, cols, in, who))) return rc;
        uint8_t* const base = static_cast<uint8_t*>(scratch);
        int32_t* const ids = reinterpret_cast<int32_t*>(base + l.ids);
        float* const weights = reinterpret_cast<float*>(base + l.weights);
        int32_t* const offsets = reinterpret_cast<int32_t*>(base + l.offsets);
        int32_t* const order = reinterpret_cast<int32_t*>(base + l.order);
        int32_t* const place = reinterpret_cast<int32_t*>(base + l.place);
        uint16_t* const h = reinterpret_cast<uint16_t*>(base + l.h);
        float* const y = reinterpret_cast<float*>(base + l.y);
        void* const room = base + l.total;
        const uint64_t room_bytes = scratch_bytes - l.total;
        const int64_t n = tokens * top_k;
        if ((rc = uw_moe_route(logits, logits_type, ldl, tokens, experts, top_k, renormalize, ids, weights, offsets,
                               order, place, base + l.route, l.h - l.route, stream)))
            return rc;
        if ((rc = uw_moe_gate_up(gate_w, gate_d, up_w, up_d, experts, rows, cols, X, tokens, ldx, offsets, order,
                                 top_k, n, h, rows, room, room_bytes, stream)))
            return rc;
        if (tokens == 1) {                      // a single token's sum needs no array of the experts' outputs
            uwk::GroupArgs a = group_args(h, n, rows, offsets, nullptr, 1, n, experts, cols, rows);
            a.w[0] = down;
            if (uwk::gemv_combine_supported(a, top_k)) {
                const uwk::CombineArgs c{nullptr, place, ids, weights, n, cols, 1, top_k, residual, out, ldr, ldo,
                                         residual_type, out_type};
                const hipError_t e = uwk::launch_gemv_combine(down_d != nullptr, a, c, as_stream(stream));
                return e == hipSuccess ? UW_OK : hip_fail(e, who);
            }
        }
        if ((rc = uw_gemm_grouped(down_w, down_d, experts, cols, rows, h, n, rows, offsets, nullptr, 1, n, y, UW_F32,
                                  cols, room, room_bytes, stream)))
            return rc;
        return uw_moe_combine(y, n, cols, place, weights, tokens, top_k, residual, residual_type, ldr, out, out_type,
                              ldo, stream);
    });
}

}  // extern "C"

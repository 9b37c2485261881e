// C ABI entry points of the epilogue matmul and of the mixture-of-experts
// operators: argument checks, scratch layout and composition.  See unweight.h
// for the contract.
#include <cmath>

#include "capi_experts.h"

using namespace uw;

namespace {

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

// A routing call: a has everything but its blocks and scratch.
int route(uwk::RouteArgs a, void* scratch, uint64_t scratch_bytes, void* stream, const char* who) {
    int rc = check_routing(a.tokens, a.experts, a.top_k, who);
    if (rc) return rc;
    if (!value_type(a.type)) return bad(who, "logits are UW_F32 or UW_BF16");
    if (!a.offsets || !aligned16(a.offsets)) return bad(who, "NULL or misaligned offsets");
    if (a.tokens) {
        if ((rc = check_rows(a.logits, a.ld, a.experts, 1, who, "logits"))) return rc;
        for (const void* p : {static_cast<const void*>(a.ids), static_cast<const void*>(a.weights),
                              static_cast<const void*>(a.order), static_cast<const void*>(a.place)})
            if (!p || !aligned16(p)) return bad(who, "NULL or misaligned output");
    }
    const uint64_t need = route_scratch(a.tokens, a.experts);
    if (need && (!scratch || !aligned16(scratch) || scratch_bytes < need))
        return bad(who, "scratch smaller than uw_moe_route_scratch_bytes()");
    // every block reads its logits while others write: nothing shares memory
    const uint64_t slots = uint64_t(a.tokens) * uint64_t(a.top_k) * 4;
    const std::pair<const void*, uint64_t> writes[] = {
        {a.ids, slots}, {a.weights, slots}, {a.offsets, uint64_t(a.experts + 1) * 4}, {a.order, slots}, {a.place, slots}, {scratch, need}};
    Inputs others;
    others.add(a.logits, span(a.tokens, a.experts, a.ld, value_bytes(a.type)));
    others.add(a.bias, uint64_t(a.experts) * 4);
    for (const auto& w : writes) {
        if (others.meet(w.first, w.second)) return bad(who, "an output or the scratch overlaps another or the logits");
        others.add(w.first, w.second);
    }
    a.counts = static_cast<uint16_t*>(scratch);
    uwk::route_blocks(a.tokens, &a.blocks, &a.per_block);
    const hipError_t e = uwk::launch_route(a, as_stream(stream));
    return e == hipSuccess ? UW_OK : hip_fail(e, who);
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
        const uwk::RouteArgs a{logits, ld,  tokens,  logits_type, experts, top_k, renormalize != 0, ids, weights,
                               offsets, order, place, nullptr, 0, 0, uwk::SCORE_LOGIT, nullptr, 1, 1, 1, 1.f};
        return route(a, scratch, scratch_bytes, stream, "uw_moe_route");
    });
}

int uw_moe_route_scored(const void* logits, int logits_type, int64_t ld, int64_t tokens, int experts, int top_k,
                        int score, const float* bias, int groups, int top_groups, int group_top, int renormalize,
                        float scale, int32_t* ids, float* weights, int32_t* offsets, int32_t* order, int32_t* place,
                        void* scratch, uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_moe_route_scored";
        if (score != UW_SCORE_SIGMOID && score != UW_SCORE_SOFTMAX) return bad(who, "unknown score");
        if (groups < 1 || groups > uwk::kMaxGroups || experts < 1 || experts % groups)
            return bad(who, "groups must be 1..16 and divide experts");
        if (top_groups < 1 || top_groups > groups) return bad(who, "top_groups must be 1..groups");
        if (group_top < 1 || group_top > 2) return bad(who, "group_top must be 1 or 2");
        if (int64_t(top_groups) * (experts / groups) < top_k) return bad(who, "the chosen groups have fewer than top_k experts");
        if (!std::isfinite(scale)) return bad(who, "scale must be finite");
        if (!aligned16(bias)) return bad(who, "misaligned bias");
        const uwk::RouteArgs a{logits, ld,  tokens,  logits_type, experts, top_k, renormalize != 0, ids, weights,
                               offsets, order, place, nullptr, 0, 0, score, bias, groups, top_groups, group_top, scale};
        return route(a, scratch, scratch_bytes, stream, who);
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

// C ABI entry points of the microscaled 4-bit operators and of the experts'
// part of a layer on a given routing: argument checks, scratch layout and
// composition.  See unweight.h for the contract.
#include "capi_experts.h"
#include "mx4.h"

using namespace uw;

namespace {

// A 4-bit matrix [rows, cols] that a call reads.
int take_mx4(const uw_mx4* m, int64_t rows, int64_t cols, uwk::Mx4Mat* out, Inputs* in, const char* who) {
    if (!m) return bad(who, "NULL 4-bit matrix");
    if (m->rows != rows || m->cols != cols) return bad(who, "the 4-bit matrix has another shape");
    if (m->ldc < cols / 2 || m->lds < cols / uwk::kMx4Block || m->ldc % 16 || m->lds % 16 ||
        m->ldc >= (int64_t(1) << 40) || m->lds >= (int64_t(1) << 40))
        return bad(who, "bad row stride of codes or scales (multiples of 16)");
    if (rows && (!m->codes || !m->scales || !aligned16(m->codes) || !aligned16(m->scales)))
        return bad(who, "NULL or misaligned codes or scales");
    in->add(m->codes, span(rows, cols / 2, m->ldc, 1));
    in->add(m->scales, span(rows, cols / uwk::kMx4Block, m->lds, 1));
    *out = {m->codes, m->scales, m->ldc, m->lds};
    return UW_OK;
}

int check_cols(int64_t rows, int64_t cols, const char* who) {
    if (rows < 0 || cols < uwk::kMx4Block || cols % uwk::kMx4Block)
        return bad(who, "bad shape (cols must be a positive multiple of 32)");
    if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) || rows * cols >= (int64_t(1) << 31))
        return fail(UW_EUNSUPPORTED, std::string(who) + ": a matrix of 2^31 weights or more");
    return UW_OK;
}

// The weights of experts: offsets inside one expert's fit 32 bits.
int take_experts(const uw_mx4* m, int64_t experts, int64_t rows, int64_t cols, uwk::Mx4Mat* out, Inputs* in,
                 const char* who) {
    int rc = check_cols(rows, cols, who);
    if (rc || (rc = take_mx4(m, experts * rows, cols, out, in, who))) return rc;
    if (rows && (m->ldc >= (int64_t(1) << 31) / rows || m->lds >= (int64_t(1) << 31) / rows))
        return fail(UW_EUNSUPPORTED, std::string(who) + ": rows of one matrix span 2^31 bytes or more");
    return UW_OK;
}

// The rows that are multiplied: bf16 X or a 4-bit matrix.
int take_rows(const uint16_t* X, int64_t ldx, const uw_mx4* x4, int64_t rows, int64_t cols, uwk::Mx4Args* a, Inputs* in,
              const char* who) {
    if ((X != nullptr) == (x4 != nullptr)) return bad(who, "give bf16 rows or 4-bit ones, and not both");
    if (x4) return take_mx4(x4, rows, cols, &a->x, in, who);
    const int rc = check_rows(X, ldx, cols, 8, who, "X");
    if (rc) return rc;
    a->g.X = X;
    a->g.ldx = ldx;
    in->add(X, span(rows, cols, ldx, 2));
    return UW_OK;
}

int run_mx4(bool x4, bool pair, const uwk::Mx4Args& a, void* stream, const char* who) {
    const hipError_t e = uwk::launch_mx4(x4, pair, a, as_stream(stream));
    return e == hipSuccess ? UW_OK : hip_fail(e, who);
}

// Scratch of the experts' part of a layer.
struct ExpertsLayout {
    uint64_t h, y, total, expand;
};

ExpertsLayout experts_layout(int form, int experts, int64_t n, int64_t F, int64_t H) {
    ExpertsLayout l{};
    // bf16, as uw_moe_layer's: the type that the instructions which multiply it with bf16, compressed or 4-bit weights
    // take.  At most half a step, 2^-8, of each h, 0.0017 of the experts' sum in the norm: next to a residual and with
    // a bf16 output the error against 64 bits is 0.0018 for one token of 6 of 64 experts (0.0017 with h in fp32) and
    // 0.0019 for 600 tokens of 4 of 32 (0.0016)
    l.h = 0;
    l.y = align256(uint64_t(n) * uint64_t(F) * 2);
    l.total = l.y + align256(uint64_t(n) * uint64_t(H) * 4);
    if (form == 1)
        l.expand = std::max(uwk::grouped_scratch(true, true, experts, F, H, n, device_cus()),
                            uwk::grouped_scratch(true, false, experts, H, F, n, device_cus()));
    return l;
}

int check_layer(int64_t tokens, int experts, int top_k, int64_t rows, int64_t cols, int64_t multiple, const char* who) {
    const int rc = check_routing(tokens, experts, top_k, who);
    if (rc) return rc;
    if (rows < multiple || cols < multiple || rows % multiple || cols % multiple)
        return bad(who, "gate and up are [rows, cols], down [cols, rows], rows and cols positive multiples of 64 (of 32 in 4 bits)");
    if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) || rows * cols >= (int64_t(1) << 31))
        return fail(UW_EUNSUPPORTED, std::string(who) + ": a matrix of 2^31 weights or more");
    return UW_OK;
}

}  // namespace

extern "C" {

int uw_mx4_quantize(const void* X, int type, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes, int64_t ldc,
                    uint8_t* scales, int64_t lds, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_mx4_quantize";
        if (!value_type(type)) return bad(who, "X is UW_F32 or UW_BF16");
        if (rows < 0 || rows >= (int64_t(1) << 31) || cols < 0 || cols >= (int64_t(1) << 31) || cols % uwk::kMx4Block)
            return bad(who, "bad shape (cols must be a multiple of 32)");
        if (rows == 0 || cols == 0) return UW_OK;
        int rc = check_rows(X, ldx, cols, type == UW_F32 ? 4 : 8, who, "X");
        if (rc) return rc;
        if ((rc = check_rows(codes, ldc, cols / 2, 16, who, "codes"))) return rc;
        if ((rc = check_rows(scales, lds, cols / uwk::kMx4Block, 16, who, "scales"))) return rc;
        const uint64_t nc = span(rows, cols / 2, ldc, 1), ns = span(rows, cols / uwk::kMx4Block, lds, 1);
        Inputs in;
        in.add(X, span(rows, cols, ldx, value_bytes(type)));
        if (in.meet(codes, nc) || in.meet(scales, ns) || overlap(codes, nc, scales, ns))
            return bad(who, "an output overlaps another or X");
        const hipError_t e = uwk::launch_mx4_quantize(X, type, ldx, rows, cols, codes, ldc, scales, lds, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int uw_mx4_dequantize(const uw_mx4* m, void* out, int out_type, int64_t ldo, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_mx4_dequantize";
        if (!m) return bad(who, "NULL 4-bit matrix");
        if (!value_type(out_type)) return bad(who, "out is UW_F32 or UW_BF16");
        if (m->rows < 0 || m->rows >= (int64_t(1) << 31) || m->cols < 0 || m->cols >= (int64_t(1) << 31) || m->cols % uwk::kMx4Block)
            return bad(who, "bad shape (cols must be a multiple of 32)");
        if (m->rows == 0 || m->cols == 0) return UW_OK;
        Inputs in;
        uwk::Mx4Mat mat;
        int rc = take_mx4(m, m->rows, m->cols, &mat, &in, who);
        if (rc) return rc;
        if ((rc = check_rows(out, ldo, m->cols, 1, who, "out"))) return rc;
        if (in.meet(out, span(m->rows, m->cols, ldo, value_bytes(out_type)))) return bad(who, "out overlaps an input");
        const hipError_t e = uwk::launch_mx4_dequantize(mat, m->rows, m->cols, out, out_type, ldo, as_stream(stream));
        return e == hipSuccess ? UW_OK : hip_fail(e, who);
    });
}

int uw_mx4_linear(const uw_mx4* w, const uint16_t* X, int64_t ldx, const uw_mx4* x4, int64_t batch, const void* bias,
                  int bias_type, int act, const void* residual, int residual_type, int64_t ldr, void* out, int out_type,
                  int64_t ldo, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_mx4_linear";
        if (!w) return bad(who, "NULL 4-bit matrix");
        const int64_t rows = w->rows, cols = w->cols;
        uwk::Mx4Args a{};
        Inputs in;
        int rc = take_experts(w, 1, rows, cols, &a.w[0], &in, who);
        if (rc) return rc;
        if (batch < 0 || batch >= (int64_t(1) << 31)) return bad(who, "bad batch");
        if (rows == 0 || batch == 0) return UW_OK;
        a.g = group_args(nullptr, batch, 0, nullptr, nullptr, 1, batch, 1, rows, cols);
        if ((rc = take_rows(X, ldx, x4, batch, cols, &a, &in, who))) return rc;
        a.g.ep = {bias, residual, out, ldr, ldo, bias_type, residual_type, out_type, act};
        in.add(bias, uint64_t(rows) * value_bytes(bias_type));
        if ((rc = check_epilogue(a.g.ep, batch, rows, in, who))) return rc;
        return run_mx4(x4 != nullptr, false, a, stream, who);
    });
}

int uw_mx4_gemm_grouped(const uw_mx4* w, int experts, const uint16_t* X, int64_t x_rows, int64_t ldx, const uw_mx4* x4,
                        const int32_t* offsets, const int32_t* order, int top_k, int64_t n, void* out, int out_type,
                        int64_t ldo, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_mx4_gemm_grouped";
        int rc = check_groups(experts, n, offsets, order, top_k, x_rows, who);
        if (rc) return rc;
        if (!w || w->rows % experts) return bad(who, "NULL 4-bit matrix or rows that are not a multiple of experts");
        const int64_t rows = w->rows / experts, cols = w->cols;
        uwk::Mx4Args a{};
        Inputs in;
        if ((rc = take_experts(w, experts, rows, cols, &a.w[0], &in, who))) return rc;
        if (rows == 0 || n == 0) return UW_OK;
        a.g = group_args(nullptr, x_rows, 0, offsets, order, top_k, n, experts, rows, cols);
        if ((rc = take_rows(X, ldx, x4, x_rows, cols, &a, &in, who))) return rc;
        a.g.ep = {nullptr, nullptr, out, 0, ldo, UW_F32, UW_F32, out_type, UW_ACT_NONE};
        add_rows(&in, a.g);
        if ((rc = check_epilogue(a.g.ep, n, rows, in, who))) return rc;
        return run_mx4(x4 != nullptr, false, a, stream, who);
    });
}

int uw_mx4_gate_up(const uw_mx4* gate, const uw_mx4* up, int experts, const uint16_t* X, int64_t x_rows, int64_t ldx,
                   const uw_mx4* x4, const int32_t* offsets, const int32_t* order, int top_k, int64_t n, uint16_t* h,
                   int64_t ldh, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_mx4_gate_up";
        int rc = check_groups(experts, n, offsets, order, top_k, x_rows, who);
        if (rc) return rc;
        if (!gate || gate->rows % experts) return bad(who, "NULL 4-bit matrix or rows that are not a multiple of experts");
        const int64_t rows = gate->rows / experts, cols = gate->cols;
        uwk::Mx4Args a{};
        Inputs in;
        if ((rc = take_experts(gate, experts, rows, cols, &a.w[0], &in, who)) ||
            (rc = take_experts(up, experts, rows, cols, &a.w[1], &in, who)))
            return rc;
        if (rows == 0 || n == 0) return UW_OK;
        a.g = group_args(nullptr, x_rows, 0, offsets, order, top_k, n, experts, rows, cols);
        if ((rc = take_rows(X, ldx, x4, x_rows, cols, &a, &in, who))) return rc;
        a.g.ep = {nullptr, nullptr, h, 0, ldh, UW_F32, UW_F32, UW_BF16, UW_ACT_NONE};
        add_rows(&in, a.g);
        if ((rc = check_epilogue(a.g.ep, n, rows, in, who))) return rc;
        return run_mx4(x4 != nullptr, true, a, stream, who);
    });
}

int64_t uw_moe_experts_scratch_bytes(int form, int64_t tokens, int experts, int top_k, int64_t rows, int64_t cols) {
    int64_t out = 0;
    const int rc = guarded([&]() -> int {
        const char* who = "uw_moe_experts_scratch_bytes";
        if (form < UW_FORM_BF16 || form > UW_FORM_MX4) return bad(who, "unknown form of the weights");
        const int r = check_layer(tokens, experts, top_k, rows, cols, form == UW_FORM_MX4 ? uwk::kMx4Block : kGroup, who);
        if (r) return r;
        const ExpertsLayout l = experts_layout(form, experts, tokens * top_k, rows, cols);
        out = int64_t(l.total + l.expand);
        return UW_OK;
    });
    return rc ? rc : out;
}

int uw_moe_experts(int form, const void* gate, const void* up, const void* down, int experts, int64_t rows, int64_t cols,
                   const uint16_t* X, int64_t ldx, int64_t tokens, int top_k, const float* weights,
                   const int32_t* offsets, const int32_t* order, const int32_t* place, const void* residual,
                   int residual_type, int64_t ldr, void* out, int out_type, int64_t ldo, void* scratch,
                   uint64_t scratch_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* who = "uw_moe_experts";
        if (form < UW_FORM_BF16 || form > UW_FORM_MX4) return bad(who, "unknown form of the weights");
        const bool mx4 = form == UW_FORM_MX4;
        int rc = check_layer(tokens, experts, top_k, rows, cols, mx4 ? uwk::kMx4Block : kGroup, who);
        if (rc) return rc;
        Inputs in;
        const void* const given[] = {gate, up, down};
        const uint16_t* w[3] = {};
        const uw_dmat* d[3] = {};
        const uw_mx4* m[3] = {};
        uwk::Mx4Mat mats[3];
        for (int i = 0; i < 3; ++i) {
            const int64_t r = i < 2 ? rows : cols, c = i < 2 ? cols : rows;
            if (mx4) {
                m[i] = static_cast<const uw_mx4*>(given[i]);
                rc = take_experts(m[i], experts, r, c, &mats[i], &in, who);
            } else {
                uwk::Weight probe;
                if (form == UW_FORM_BF16) w[i] = static_cast<const uint16_t*>(given[i]);
                else d[i] = static_cast<const uw_dmat*>(given[i]);
                rc = take_weight(w[i], d[i], experts, r, c, &probe, &in, who);
            }
            if (rc) return rc;
        }
        if (tokens == 0) return UW_OK;
        const int64_t n = tokens * top_k;
        if ((rc = check_rows(X, ldx, cols, 8, who, "X"))) return rc;
        for (const void* p : {static_cast<const void*>(weights), static_cast<const void*>(offsets),
                              static_cast<const void*>(order), static_cast<const void*>(place)})
            if (!p || !aligned16(p)) return bad(who, "NULL or misaligned weights, offsets, order or place");
        // read by the last step, which writes out; X is not: out may be X or the residual
        in.add(weights, uint64_t(n) * 4);
        in.add(place, uint64_t(n) * 4);
        const uwk::Epilogue ep{nullptr, residual, out, ldr, ldo, UW_F32, residual_type, out_type, UW_ACT_NONE};
        in.add(offsets, uint64_t(experts + 1) * 4);
        in.add(order, uint64_t(n) * 4);
        if ((rc = check_epilogue(ep, tokens, cols, in, who))) return rc;
        const ExpertsLayout l = experts_layout(form, experts, n, rows, cols);
        if (!scratch || !aligned16(scratch) || scratch_bytes < l.total)
            return bad(who, "scratch smaller than uw_moe_experts_scratch_bytes()");
        in.add(X, span(tokens, cols, ldx, 2));
        if ((rc = check_scratch(scratch, &scratch_bytes, ep, tokens, cols, in, who))) return rc;
        uint8_t* const base = static_cast<uint8_t*>(scratch);
        uint16_t* const h = reinterpret_cast<uint16_t*>(base + l.h);
        float* const y = reinterpret_cast<float*>(base + l.y);
        if (mx4) {
            if ((rc = uw_mx4_gate_up(m[0], m[1], experts, X, tokens, ldx, nullptr, offsets, order, top_k, n, h, rows, stream)))
                return rc;
            if (tokens == 1) {                  // a single token's sum needs no array of the experts' outputs
                const uwk::Mx4OneArgs a{mats[2], h, rows, offsets, place, weights, experts, top_k, int32_t(cols), int32_t(rows), ep};
                if (uwk::mx4_one_supported(a)) {
                    const hipError_t e = uwk::launch_mx4_one(a, as_stream(stream));
                    return e == hipSuccess ? UW_OK : hip_fail(e, who);
                }
            }
            if ((rc = uw_mx4_gemm_grouped(m[2], experts, h, n, rows, nullptr, offsets, nullptr, 1, n, y, UW_F32, cols, stream)))
                return rc;
        } else {
            void* const room = base + l.total;
            const uint64_t room_bytes = scratch_bytes - l.total;
            if ((rc = uw_moe_gate_up(w[0], d[0], w[1], d[1], experts, rows, cols, X, tokens, ldx, offsets, order, top_k, n,
                                     h, rows, room, room_bytes, stream)) ||
                (rc = uw_gemm_grouped(w[2], d[2], experts, cols, rows, h, n, rows, offsets, nullptr, 1, n, y, UW_F32, cols,
                                      room, room_bytes, stream)))
                return rc;
        }
        return uw_moe_combine(y, n, cols, place, weights, tokens, top_k, residual, residual_type, ldr, out, out_type,
                              ldo, stream);
    });
}

}  // extern "C"

// Argument checks that the entry points of the epilogue matmul, of the
// mixture-of-experts operators and of the microscaled 4-bit ones share.
#pragma once

#include <algorithm>
#include <exception>
#include <string>
#include <utility>

#include "capi_common.h"
#include "experts.h"

namespace uw {

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

inline int bad(const char* who, const char* what) { return fail(UW_EINVAL, std::string(who) + ": " + what); }

inline bool value_type(int t) { return t == UW_F32 || t == UW_BF16; }
inline int64_t value_bytes(int t) { return t == UW_BF16 ? 2 : 4; }

// Bytes from the first to behind the last element of [rows, cols] with row stride ld.
inline uint64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
    return rows > 0 && cols > 0 ? (uint64_t(rows - 1) * uint64_t(ld) + uint64_t(cols)) * uint64_t(bytes) : 0;
}

inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
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
inline int take_weight(const uint16_t* w, const uw_dmat* d, int64_t experts, int64_t rows, int64_t cols, uwk::Weight* out,
                Inputs* in, const char* who) {
    *out = uwk::Weight{};
    if (rows < 0 || cols < kGroup || cols % kGroup)
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
    int rc = check_dmat(d, who);
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
    out->vexp = vexp_of(d) ? d->vexp : d->sm;   // never read as exponents without verbatim groups
    out->bitmap = d->bitmap;
    out->tile_vbase = d->tile_vbase;
    pack_palette(d->palette, out->pal);
    out->last_slot = d->verbatim_groups ? uint32_t(d->verbatim_groups) - 1 : 0;
    return UW_OK;
}

inline int check_rows(const void* p, int64_t ld, int64_t cols, int64_t multiple, const char* who, const char* name) {
    if (!p || !aligned16(p)) return fail(UW_EINVAL, std::string(who) + ": NULL or misaligned " + name);
    if (ld < cols || ld % multiple || ld >= (int64_t(1) << 40))
        return fail(UW_EINVAL, std::string(who) + ": bad row stride of " + name);
    return UW_OK;
}

// out (and the residual it may replace) against what the call reads while out is written.
inline int check_epilogue(const uwk::Epilogue& e, int64_t n, int64_t rows, const Inputs& in, const char* who) {
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
inline int check_scratch(const void* scratch, uint64_t* bytes, const uwk::Epilogue& e, int64_t n, int64_t rows,
                  const Inputs& in, const char* who) {
    if (!aligned16(scratch)) return bad(who, "misaligned scratch");
    if (!scratch) *bytes = 0;
    if (overlap(e.out, span(n, rows, e.ldo, value_bytes(e.out_type)), scratch, *bytes) || in.meet(scratch, *bytes) ||
        (e.residual && overlap(e.residual, span(n, rows, e.ldr, value_bytes(e.residual_type)), scratch, *bytes)))
        return bad(who, "the scratch overlaps an input or out");
    return UW_OK;
}

inline int check_groups(int experts, int64_t n, const int32_t* offsets, const int32_t* order, int top_k, int64_t x_rows,
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
inline void add_rows(Inputs* in, const uwk::GroupArgs& a) {
    in->add(a.X, span(a.x_rows, a.C, a.ldx, 2));
    in->add(a.offsets, uint64_t(a.E + 1) * 4);
    in->add(a.order, uint64_t(a.n) * 4);
}

inline uwk::GroupArgs group_args(const uint16_t* X, int64_t x_rows, int64_t ldx, const int32_t* offsets, const int32_t* order,
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
    a.cus = device_cus();
    return a;
}

// Scratch of a routing call with more than one block of tokens.
inline uint64_t route_scratch(int64_t tokens, int64_t experts) {
    int32_t blocks, per;
    uwk::route_blocks(tokens, &blocks, &per);
    return blocks > 1 ? align256(uint64_t(blocks) * uint64_t((experts + 7) / 8) * 16) : 0;
}

inline int check_routing(int64_t tokens, int experts, int top_k, const char* who) {
    if (tokens < 0 || tokens >= (int64_t(1) << 31)) return bad(who, "bad number of tokens");
    if (experts < 1 || experts > uwk::kMaxExperts) return bad(who, "experts must be 1..512");
    if (top_k < 1 || top_k > uwk::kMaxTopK || top_k > experts) return bad(who, "top_k must be 1..16 and at most experts");
    if (tokens * top_k >= (int64_t(1) << 31)) return bad(who, "tokens * top_k must be below 2^31");
    return UW_OK;
}

}  // namespace uw

// C ABI of the residual addition with its RMS norm, and of the rotary positions. Declared in
// include/muon_rocm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include "../../include/muon_rocm.h"
#include "abi_internal.hpp"
#include "blocks8.hpp"

#define MUON_API extern "C" __attribute__((visibility("default")))

namespace muon {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxSpan = int64_t(1) << 46;

int fail(int code, const std::string& what) { return set_last_error(code, what); }

// Rows of `cols` elements a stride apart; *range is empty where there are none.
int check_rows(const norm_rows* t, int64_t rows, int64_t cols, int dtype, const char* name, bool write, Range* range) {
    const std::string who(name);
    *range = {0, 0, write};
    if (!t) return fail(MUON_ERR_INVALID_ARG, who + " is NULL");
    if (rows == 0 || cols == 0) return MUON_OK;
    if (!t->data) return fail(MUON_ERR_INVALID_ARG, who + "->data is NULL");
    if (t->stride0 < 0) return fail(MUON_ERR_INVALID_ARG, who + " has a negative stride");
    if (write && rows > 1 && t->stride0 < cols) return fail(MUON_ERR_ALIAS, who + " has rows that overlap");
    const __int128 span = __int128(rows - 1) * t->stride0 + cols;
    if (span > kMaxSpan) return fail(MUON_ERR_TOO_LARGE, who + " spans more than 2^46 elements");
    const int e = elem_size(dtype);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t->data);
    if (lo % e) return fail(MUON_ERR_ALIGN, who + " is not aligned to its element");
    *range = {lo, lo + uintptr_t(span) * e, write};
    return MUON_OK;
}

bool present(const norm_rows* t) { return t && t->data; }
bool present(const norm_param* t) { return t && t->data; }

// Whether an output's rows are an input's: the same elements at the same places.
bool same(const norm_rows& a, const norm_rows& b, int64_t rows, int ta, int tb) {
    return ta == tb && a.data == b.data && (rows <= 1 || a.stride0 == b.stride0);
}

int check_desc(const add_norm_desc* d) {
    if (!d) return fail(MUON_ERR_INVALID_ARG, "desc is NULL");
    if (d->rows < 0 || d->cols < 0) return fail(MUON_ERR_INVALID_ARG, "negative dimension");
    if (d->dtype < MUON_DTYPE_F32 || d->dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (d->rdtype != MUON_DTYPE_F32 && d->rdtype != d->dtype) return fail(MUON_ERR_INVALID_ARG, "rdtype must be fp32 or dtype");
    if (d->wdtype != MUON_DTYPE_F32 && d->wdtype != d->dtype) return fail(MUON_ERR_INVALID_ARG, "wdtype must be fp32 or dtype");
    if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return fail(MUON_ERR_INVALID_ARG, "eps must be finite and > 0");
    if (!std::isfinite(d->weight_offset)) return fail(MUON_ERR_INVALID_ARG, "weight_offset must be finite");
    if (d->cols > MUON_NORM_MAX_COLS) return fail(MUON_ERR_TOO_LARGE, "cols above " + std::to_string(MUON_NORM_MAX_COLS));
    if (d->rows > kMaxRows) return fail(MUON_ERR_TOO_LARGE, "rows above 2^30");
    return MUON_OK;
}

int check_vector(const void* p, int64_t n, int bytes, const char* name, bool write, std::vector<Range>& ranges) {
    if (!p || n == 0) return MUON_OK;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo % bytes) return fail(MUON_ERR_ALIGN, std::string(name) + " is not aligned to its element");
    ranges.push_back({lo, lo + uintptr_t(n) * bytes, write});
    return MUON_OK;
}

AddNormArgs base_args(const add_norm_desc& d, const NormPlan& p) {
    AddNormArgs a{};
    a.rows = int32_t(d.rows);
    a.cols = int32_t(d.cols);
    a.wdtype = d.wdtype;
    a.chunks = p.chunks;
    a.team_waves = p.lanes / 64;
    a.teams = p.teams;
    a.eps = d.eps;
    a.offset = d.weight_offset;
    a.inv_cols = 1.0 / double(d.cols);
    return a;
}

size_t partial_bytes(const add_norm_desc& d, const NormPlan& p) {
    return p.chunks > 1 ? size_t(p.chunks) * size_t(d.cols) * 4 : 0;
}

// ---- rotary ----
int check_rotary_rows(const rotary_desc& d, const rotary_rows* t, const char* name, bool write, Range* range) {
    const std::string who(name);
    *range = {0, 0, write};
    if (!t) return fail(MUON_ERR_INVALID_ARG, who + " is NULL");
    if (d.batch == 0 || d.tokens == 0 || d.heads == 0 || d.dim == 0) return MUON_OK;
    if (!t->data) return fail(MUON_ERR_INVALID_ARG, who + "->data is NULL");
    struct {
        int64_t n, s;
    } level[3] = {{d.batch, t->stride_batch}, {d.tokens, t->stride_token}, {d.heads, t->stride_head}};
    for (auto& l : level) {
        if (l.n > 1 && l.s < 0) return fail(MUON_ERR_INVALID_ARG, who + " has a negative stride");
        if (l.n == 1) l.s = 0;
    }
    std::sort(level, level + 3, [](auto& a, auto& b) { return a.s < b.s; });
    __int128 span = d.dim;
    for (auto& l : level) {
        if (l.n == 1) continue;
        if (write && l.s < span) return fail(MUON_ERR_ALIAS, who + " has heads that overlap");
        span += __int128(l.n - 1) * l.s;
        if (span > kMaxSpan) return fail(MUON_ERR_TOO_LARGE, who + " spans more than 2^46 elements");
    }
    const int e = elem_size(d.dtype);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t->data);
    if (lo % e) return fail(MUON_ERR_ALIGN, who + " is not aligned to its element");
    *range = {lo, lo + uintptr_t(span) * e, write};
    return MUON_OK;
}

bool same(const rotary_desc& d, const rotary_rows& a, const rotary_rows& b) {
    return a.data == b.data && (d.batch <= 1 || a.stride_batch == b.stride_batch) &&
           (d.tokens <= 1 || a.stride_token == b.stride_token) && (d.heads <= 1 || a.stride_head == b.stride_head);
}

}  // namespace
}  // namespace muon

using namespace muon;

MUON_API int add_rms_norm_forward(const add_norm_desc* desc, const norm_rows* x, const norm_rows* residual, const norm_param* w,
                                  const norm_rows* h, const norm_rows* y, const blocks8* codes, float* rstd, void* stream) {
    return guarded([&]() -> int {
        int rc = check_desc(desc);
        if (rc) return rc;
        const add_norm_desc& d = *desc;
        const bool res = present(residual);
        if (!res && present(h)) return fail(MUON_ERR_INVALID_ARG, "h without residual");
        std::vector<Range> ranges;
        Range r;
        if ((rc = check_rows(x, d.rows, d.cols, d.dtype, "x", false, &r))) return rc;
        // h may be the residual or x
        const bool on_x = res && present(h) && same(*h, *x, d.rows, d.rdtype, d.dtype);
        if (!on_x) ranges.push_back(r);
        if (res) {
            if ((rc = check_rows(residual, d.rows, d.cols, d.rdtype, "residual", false, &r))) return rc;
            if (!(present(h) && same(*h, *residual, d.rows, d.rdtype, d.rdtype))) ranges.push_back(r);
            if ((rc = check_rows(h, d.rows, d.cols, d.rdtype, "h", true, &r))) return rc;
            ranges.push_back(r);
        }
        if (present(y)) {
            if ((rc = check_rows(y, d.rows, d.cols, d.dtype, "y", true, &r))) return rc;
            ranges.push_back(r);
        }
        if (codes) {
            if (codes->rows != d.rows || codes->cols != d.cols || codes->tiles)
                return fail(MUON_ERR_INVALID_ARG, "codes is not [rows, cols] in blocks of 1 x 128");
            if ((rc = check_blocks(codes, "codes", true, ranges))) return rc;
        }
        if (present(w) && (rc = check_vector(w->data, d.cols, elem_size(d.wdtype), "w", false, ranges))) return rc;
        if ((rc = check_vector(rstd, d.rows, 4, "rstd", true, ranges)) || (rc = check_overlaps(ranges))) return rc;
        if (d.rows == 0 || d.cols == 0) return MUON_OK;
        const NormPlan p = plan_add_norm(true, d.dtype, d.cols, d.rows);
        AddNormArgs a = base_args(d, p);
        a.x = x->data;
        a.x_stride = x->stride0;
        if (res) {
            a.r = residual->data;
            a.r_stride = residual->stride0;
            a.h = h->data;
            a.h_stride = h->stride0;
        }
        if (present(y)) {
            a.y = y->data;
            a.y_stride = y->stride0;
        }
        if (codes) a.q = Blocks8Ptr{codes->codes, codes->scales, codes->ld, codes->scale_ld};
        if (present(w)) a.w = w->data;
        a.rstd = rstd;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_ADD_NORM_FORWARD, s, "add norm forward", [&] {
            return launch_add_norm_forward(d.dtype, d.rdtype != d.dtype, p, a, s);
        });
    });
}

MUON_API int add_rms_norm_backward_workspace_bytes(const add_norm_desc* desc, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
        const int rc = check_desc(desc);
        if (rc) return rc;
        *bytes = desc->rows == 0 || desc->cols == 0
                     ? 0
                     : partial_bytes(*desc, plan_add_norm(false, desc->dtype, desc->cols, desc->rows));
        return MUON_OK;
    });
}

MUON_API int add_rms_norm_backward(const add_norm_desc* desc, const norm_rows* dy, const norm_rows* dh, const norm_rows* h,
                                   const norm_param* w, const float* rstd, const norm_rows* dr, const norm_rows* dx,
                                   const norm_param* dw, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_desc(desc);
        if (rc) return rc;
        const add_norm_desc& d = *desc;
        const bool has = d.rows > 0 && d.cols > 0;
        if (has && !rstd) return fail(MUON_ERR_INVALID_ARG, "rstd is NULL");
        if (present(dw) && !present(w)) return fail(MUON_ERR_INVALID_ARG, "dw without w");
        if (present(dx) && d.dtype == d.rdtype) return fail(MUON_ERR_INVALID_ARG, "dx is dr where the types are the same");
        std::vector<Range> ranges;
        Range r, rr;
        if ((rc = check_rows(dr, d.rows, d.cols, d.rdtype, "dr", true, &rr))) return rc;
        // an output may be an input that has its type and rows
        auto shared = [&](const norm_rows& t, int type) {
            return same(*dr, t, d.rows, d.rdtype, type) || (present(dx) && same(*dx, t, d.rows, d.dtype, type));
        };
        if ((rc = check_rows(dy, d.rows, d.cols, d.dtype, "dy", false, &r))) return rc;
        if (!shared(*dy, d.dtype)) ranges.push_back(r);
        if (present(dh)) {
            if ((rc = check_rows(dh, d.rows, d.cols, d.rdtype, "dh", false, &r))) return rc;
            if (!shared(*dh, d.rdtype)) ranges.push_back(r);
        }
        if ((rc = check_rows(h, d.rows, d.cols, d.rdtype, "h", false, &r))) return rc;
        if (!shared(*h, d.rdtype)) ranges.push_back(r);
        ranges.push_back(rr);
        if (present(dx)) {
            if ((rc = check_rows(dx, d.rows, d.cols, d.dtype, "dx", true, &r))) return rc;
            ranges.push_back(r);
        }
        if (present(w) && (rc = check_vector(w->data, d.cols, elem_size(d.wdtype), "w", false, ranges))) return rc;
        if (present(dw) && (rc = check_vector(dw->data, d.cols, elem_size(d.wdtype), "dw", true, ranges))) return rc;
        if ((rc = check_vector(rstd, d.rows, 4, "rstd", false, ranges))) return rc;
        const NormPlan p = plan_add_norm(false, d.dtype, std::max<int64_t>(d.cols, 1), d.rows);
        const size_t need = has && present(dw) ? partial_bytes(d, p) : 0;
        if (need) {
            if (!workspace) return fail(MUON_ERR_WORKSPACE, "workspace is NULL");
            if (workspace_bytes < need)
                return fail(MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
            const uintptr_t lo = reinterpret_cast<uintptr_t>(workspace);
            if (lo & 255) return fail(MUON_ERR_ALIGN, "workspace not 256-byte aligned");
            ranges.push_back({lo, lo + need, true});
        }
        if ((rc = check_overlaps(ranges))) return rc;
        if (d.cols == 0 || (d.rows == 0 && !present(dw))) return MUON_OK;
        AddNormArgs a = base_args(d, p);
        a.x = dy->data;
        a.x_stride = dy->stride0;
        if (present(dh)) {
            a.r = dh->data;
            a.r_stride = dh->stride0;
        }
        a.h = h->data;
        a.h_stride = h->stride0;
        a.d = dr->data;
        a.d_stride = dr->stride0;
        if (present(dx)) {
            a.y = dx->data;
            a.y_stride = dx->stride0;
        }
        if (present(w)) a.w = w->data;
        a.rstd = const_cast<float*>(rstd);
        if (present(dw)) a.dw = dw->data;
        a.partial = static_cast<float*>(workspace);
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        rc = run_timed(MUON_KCLASS_ADD_NORM_BACKWARD, s, "add norm backward", [&] {
            return launch_add_norm_backward(d.dtype, d.rdtype != d.dtype, p, a, s);
        });
        if (rc || need == 0) return rc;
        NormArgs g{};
        g.partial = a.partial;
        g.dw = a.dw;
        g.groups = 1;
        g.chunks = p.chunks;
        g.cols = a.cols;
        g.wdtype = a.wdtype;
        return run_timed(MUON_KCLASS_NORM_WGRAD, s, "norm weight gradient", [&] { return launch_norm_wgrad(g, s); });
    });
}

MUON_API int rotary_apply(const rotary_desc* desc, const rotary_rows* x, const rotary_positions* positions, const double* freq,
                          const int32_t* axis, const rotary_rows* y, void* stream) {
    return guarded([&]() -> int {
        if (!desc) return fail(MUON_ERR_INVALID_ARG, "desc is NULL");
        const rotary_desc& d = *desc;
        if (d.batch < 0 || d.tokens < 0 || d.heads < 0 || d.dim < 0) return fail(MUON_ERR_INVALID_ARG, "negative dimension");
        if (d.pairs < 1 || d.axes < 1) return fail(MUON_ERR_INVALID_ARG, "pairs and axes must be >= 1");
        if (d.dtype < MUON_DTYPE_F32 || d.dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
        if (d.layout != MUON_ROTARY_HALVES && d.layout != MUON_ROTARY_ADJACENT) return fail(MUON_ERR_INVALID_ARG, "unknown layout");
        if (d.position_type < MUON_POSITION_I32 || d.position_type > MUON_POSITION_F32)
            return fail(MUON_ERR_INVALID_ARG, "unknown position_type");
        if (d.dim > MUON_ROTARY_MAX_DIM || d.heads > MUON_ROTARY_MAX_HEADS || d.batch > kMaxRows || d.tokens > kMaxRows ||
            __int128(d.batch) * d.tokens > kMaxRows)
            return fail(MUON_ERR_TOO_LARGE, "dim above 1024, heads above 2^16 or more than 2^30 tokens");
        if (2 * int64_t(d.pairs) > d.dim && d.dim > 0) return fail(MUON_ERR_INVALID_ARG, "more pairs than a head has");
        std::vector<Range> ranges;
        Range rx, ry;
        int rc;
        if ((rc = check_rotary_rows(d, x, "x", false, &rx)) || (rc = check_rotary_rows(d, y, "y", true, &ry))) return rc;
        if (d.batch == 0 || d.tokens == 0 || d.heads == 0 || d.dim == 0) return MUON_OK;
        if (!same(d, *x, *y)) ranges.push_back(rx);
        ranges.push_back(ry);
        if (!positions || !positions->data || !freq || !axis)
            return fail(MUON_ERR_INVALID_ARG, "positions, freq or axis is NULL");
        if (positions->stride_batch < 0 || positions->stride_token < 0)
            return fail(MUON_ERR_INVALID_ARG, "positions has a negative stride");
        const __int128 span = __int128(d.batch - 1) * positions->stride_batch + __int128(d.tokens - 1) * positions->stride_token + d.axes;
        if (span > kMaxSpan) return fail(MUON_ERR_TOO_LARGE, "positions spans more than 2^46 elements");
        if ((rc = check_vector(positions->data, int64_t(span), d.position_type == MUON_POSITION_I64 ? 8 : 4, "positions", false, ranges)) ||
            (rc = check_vector(freq, d.pairs, 8, "freq", false, ranges)) ||
            (rc = check_vector(axis, d.pairs, 4, "axis", false, ranges)) || (rc = check_overlaps(ranges)))
            return rc;
        RotaryArgs a{};
        a.x = {x->data, x->stride_batch, x->stride_token, x->stride_head};
        a.y = {y->data, y->stride_batch, y->stride_token, y->stride_head};
        a.pos = positions->data;
        a.pb = positions->stride_batch;
        a.pt = positions->stride_token;
        a.freq = freq;
        a.axis = axis;
        a.rows = uint32_t(d.batch * d.tokens);
        a.tokens = uint32_t(d.tokens);
        a.heads = int32_t(d.heads);
        a.dim = int32_t(d.dim);
        a.pairs = d.pairs;
        a.axes = d.axes;
        a.pos_type = d.position_type;
        int l = 0;
        while ((int64_t(1) << l) < d.heads) ++l;
        a.heads_shift = l;
        a.heads_mul = uint32_t((((uint64_t(1) << l) - uint64_t(d.heads)) << 32) / uint64_t(d.heads) + 1);
        a.sign = d.inverse ? -1.f : 1.f;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_ROTARY, s, "rotary",
                         [&] { return launch_rotary(d.dtype, d.layout == MUON_ROTARY_ADJACENT, a, s); });
    });
}

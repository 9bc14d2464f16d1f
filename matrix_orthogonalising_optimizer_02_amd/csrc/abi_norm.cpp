// C ABI of the normalisation layers: argument validation, the split into blocks and the
// launches. Declared in include/muon_rocm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include "../../include/muon_rocm.h"
#include "abi_internal.hpp"
#include "train.hpp"

#define MUON_API extern "C" __attribute__((visibility("default")))

namespace muon {
namespace {

static_assert(kF32 == MUON_DTYPE_F32 && kBF16 == MUON_DTYPE_BF16 && kF16 == MUON_DTYPE_F16, "type codes");
static_assert(kNormMaxCols == MUON_NORM_MAX_COLS, "column limit");

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of a launch, a dimension
constexpr int64_t kMaxSpan = int64_t(1) << 46;

int fail(int code, const std::string& what) { return set_last_error(code, what); }

int check_desc(const norm_desc* d) {
    if (!d) return fail(MUON_ERR_INVALID_ARG, "desc is NULL");
    if (d->kind != MUON_NORM_LAYER && d->kind != MUON_NORM_RMS) return fail(MUON_ERR_INVALID_ARG, "unknown kind");
    if (d->dtype < MUON_DTYPE_F32 || d->dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (d->wdtype != MUON_DTYPE_F32 && d->wdtype != d->dtype)
        return fail(MUON_ERR_INVALID_ARG, "wdtype must be fp32 or dtype");
    if (d->rows < 0 || d->cols < 0) return fail(MUON_ERR_INVALID_ARG, "negative dimension");
    if (d->groups < 1 || d->rows % d->groups) return fail(MUON_ERR_INVALID_ARG, "groups must be >= 1 and divide rows");
    if (d->inner < 1 || d->rows % d->inner) return fail(MUON_ERR_INVALID_ARG, "inner must be >= 1 and divide rows");
    if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return fail(MUON_ERR_INVALID_ARG, "eps must be finite and > 0");
    if (!std::isfinite(d->weight_offset)) return fail(MUON_ERR_INVALID_ARG, "weight_offset must be finite");
    if (d->cols > kNormMaxCols)
        return fail(MUON_ERR_TOO_LARGE, "cols above " + std::to_string(kNormMaxCols));
    if (d->rows > kMaxRows || d->groups > kMaxRows || d->inner > kMaxRows)
        return fail(MUON_ERR_TOO_LARGE, "rows, groups or inner above 2^30");
    return MUON_OK;
}

// The span of a strided tensor, checked; *range is empty where the tensor has no elements.
int check_rows(const norm_desc& d, const norm_rows* t, const char* name, bool write, Range* range) {
    *range = {0, 0, write};
    if (!t) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if (d.rows == 0 || d.cols == 0) return MUON_OK;
    if (!t->data) return fail(MUON_ERR_INVALID_ARG, std::string(name) + "->data is NULL");
    if (t->stride0 < 0 || t->stride1 < 0) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " has a negative stride");
    const int64_t n0 = d.rows / d.inner, n1 = d.inner;
    const int64_t s0 = n0 > 1 ? t->stride0 : 0, s1 = n1 > 1 ? t->stride1 : 0;
    const __int128 span = __int128(n0 - 1) * s0 + __int128(n1 - 1) * s1 + d.cols;
    if (span > kMaxSpan) return fail(MUON_ERR_TOO_LARGE, std::string(name) + " spans more than 2^46 elements");
    if (write) {
        const bool first = (n0 > 1 ? s0 : kMaxSpan) < (n1 > 1 ? s1 : kMaxSpan);  // the closer rows
        const int64_t near_n = first ? n0 : n1, near_s = first ? s0 : s1;
        const int64_t far_n = first ? n1 : n0, far_s = first ? s1 : s0;
        if ((near_n > 1 && near_s < d.cols) || (far_n > 1 && far_s < (near_n - 1) * near_s + d.cols))
            return fail(MUON_ERR_ALIAS, std::string(name) + " has rows that overlap");
    }
    const int e = elem_size(d.dtype);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t->data);
    if (lo % e) return fail(MUON_ERR_ALIGN, std::string(name) + " is not aligned to its element");
    *range = {lo, lo + uintptr_t(span) * e, write};
    return MUON_OK;
}

int check_param(const norm_desc& d, const norm_param* p, const char* name, bool write, std::vector<Range>& ranges) {
    if (!p || !p->data || d.cols == 0) return MUON_OK;
    if (p->stride < 0) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " has a negative stride");
    const int64_t s = d.groups > 1 ? p->stride : 0;
    if (write && d.groups > 1 && s < d.cols) return fail(MUON_ERR_ALIAS, std::string(name) + " has rows that overlap");
    const __int128 span = __int128(d.groups - 1) * s + d.cols;
    if (span > kMaxSpan) return fail(MUON_ERR_TOO_LARGE, std::string(name) + " spans more than 2^46 elements");
    const int e = elem_size(d.wdtype);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p->data);
    if (lo % e) return fail(MUON_ERR_ALIGN, std::string(name) + " is not aligned to its element");
    ranges.push_back({lo, lo + uintptr_t(span) * e, write});
    return MUON_OK;
}

int check_stats(const norm_desc& d, const float* p, const char* name, bool write, std::vector<Range>& ranges) {
    if (!p || d.rows == 0) return MUON_OK;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo & 3) return fail(MUON_ERR_ALIGN, std::string(name) + " is not 4-byte aligned");
    ranges.push_back({lo, lo + uintptr_t(d.rows) * 4, write});
    return MUON_OK;
}

bool same_rows(const norm_desc& d, const norm_rows& a, const norm_rows& b) {
    return a.data == b.data && (d.rows / d.inner <= 1 || a.stride0 == b.stride0) && (d.inner <= 1 || a.stride1 == b.stride1);
}

RowsPtr rows_ptr(const norm_rows& t) { return {t.data, t.stride0, t.stride1}; }

bool present(const norm_param* p) { return p && p->data; }

NormArgs base_args(const norm_desc& d, const NormPlan& p) {
    NormArgs a{};
    a.rows_per_group = int32_t(d.rows / d.groups);
    a.groups = int32_t(d.groups);
    a.cols = int32_t(d.cols);
    a.inner = int32_t(d.inner);
    // division by a constant (Granlund and Montgomery 1994): l = ceil(log2 inner),
    // multiplier floor(2^32 (2^l - inner) / inner) + 1, exact for every 32-bit dividend
    int l = 0;
    while ((int64_t(1) << l) < d.inner) ++l;
    a.inner_shift = l;
    a.inner_mul = uint32_t(((uint64_t((int64_t(1) << l) - d.inner) << 32) / uint64_t(d.inner)) + 1);
    a.chunks = p.chunks;
    a.chunk_rows = p.chunk_rows;
    a.team_waves = p.lanes / 64;
    a.teams = p.teams;
    a.wdtype = d.wdtype;
    a.eps = d.eps;
    a.offset = d.weight_offset;
    a.inv_cols = float(1.0 / double(d.cols));
    return a;
}

size_t partial_bytes(const norm_desc& d, const NormPlan& p) {
    return p.chunks > 1 ? size_t(2) * size_t(d.groups) * size_t(p.chunks) * size_t(d.cols) * 4 : 0;
}

}  // namespace
}  // namespace muon

using namespace muon;

MUON_API int norm_forward(const norm_desc* desc, const norm_rows* x, const norm_param* w, const norm_param* b,
                          const norm_rows* y, float* mean, float* rstd, void* stream) {
    return guarded([&]() -> int {
        int rc = check_desc(desc);
        if (rc) return rc;
        const norm_desc& d = *desc;
        if (d.kind == MUON_NORM_RMS) mean = nullptr;
        std::vector<Range> ranges;
        Range rx, ry;
        if ((rc = check_rows(d, x, "x", false, &rx)) || (rc = check_rows(d, y, "y", true, &ry))) return rc;
        if (!same_rows(d, *x, *y)) ranges.push_back(rx);
        ranges.push_back(ry);
        if ((rc = check_param(d, w, "w", false, ranges)) || (rc = check_param(d, b, "b", false, ranges)) ||
            (rc = check_stats(d, mean, "mean", true, ranges)) || (rc = check_stats(d, rstd, "rstd", true, ranges)))
            return rc;
        if ((rc = check_overlaps(ranges))) return rc;
        if (d.rows == 0 || d.cols == 0) return MUON_OK;
        const NormPlan p = plan_norm_forward(d.dtype, d.cols, d.rows / d.groups, d.groups);
        if (d.groups * int64_t(p.chunks) > kMaxThreads / p.threads)
            return fail(MUON_ERR_TOO_LARGE, "more groups than a launch takes");
        NormArgs a = base_args(d, p);
        a.x = rows_ptr(*x);
        a.y = rows_ptr(*y);
        if (present(w)) {
            a.w = w->data;
            a.w_stride = w->stride;
        }
        if (present(b)) {
            a.b = b->data;
            a.b_stride = b->stride;
        }
        a.mean = mean;
        a.rstd = rstd;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_NORM_FORWARD, s, "norm forward",
                         [&] { return launch_norm_forward(d.kind == MUON_NORM_RMS, d.dtype, p, a, s); });
    });
}

MUON_API int norm_backward_workspace_bytes(const norm_desc* desc, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
        const int rc = check_desc(desc);
        if (rc) return rc;
        *bytes = desc->cols == 0 ? 0
                                 : partial_bytes(*desc, plan_norm_backward(desc->dtype, desc->cols,
                                                                           desc->rows / desc->groups, desc->groups));
        return MUON_OK;
    });
}

MUON_API int norm_backward(const norm_desc* desc, const norm_rows* dy, const norm_rows* x, const norm_param* w,
                           const float* mean, const float* rstd, const norm_rows* dx, const norm_param* dw,
                           const norm_param* db, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> int {
        int rc = check_desc(desc);
        if (rc) return rc;
        const norm_desc& d = *desc;
        const bool layer = d.kind == MUON_NORM_LAYER;
        if (!layer) mean = nullptr;
        const bool has_rows = d.rows > 0 && d.cols > 0;
        if (has_rows && (!rstd || (layer && !mean))) return fail(MUON_ERR_INVALID_ARG, "mean or rstd is NULL");
        if (present(dw) && !present(w)) return fail(MUON_ERR_INVALID_ARG, "dw without w");
        std::vector<Range> ranges;
        Range rdy, rx, rdx;
        if ((rc = check_rows(d, dy, "dy", false, &rdy)) || (rc = check_rows(d, x, "x", false, &rx)) ||
            (rc = check_rows(d, dx, "dx", true, &rdx)))
            return rc;
        if (!same_rows(d, *dy, *dx)) ranges.push_back(rdy);
        if (!same_rows(d, *x, *dx)) ranges.push_back(rx);
        ranges.push_back(rdx);
        if ((rc = check_param(d, w, "w", false, ranges)) || (rc = check_param(d, dw, "dw", true, ranges)) ||
            (rc = check_param(d, db, "db", true, ranges)) || (rc = check_stats(d, mean, "mean", false, ranges)) ||
            (rc = check_stats(d, rstd, "rstd", false, ranges)))
            return rc;
        if (d.cols == 0) return MUON_OK;
        const NormPlan p = plan_norm_backward(d.dtype, d.cols, d.rows / d.groups, d.groups);
        if (d.groups * int64_t(p.chunks) > kMaxThreads / p.threads)
            return fail(MUON_ERR_TOO_LARGE, "more groups than a launch takes");
        const bool grads = present(dw) || present(db);
        const size_t need = grads ? partial_bytes(d, p) : 0;
        if (need) {
            if (!workspace) return fail(MUON_ERR_WORKSPACE, "workspace is NULL");
            if (workspace_bytes < need)
                return fail(MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
            const uintptr_t lo = reinterpret_cast<uintptr_t>(workspace);
            if (lo & 255) return fail(MUON_ERR_ALIGN, "workspace not 256-byte aligned");
            ranges.push_back({lo, lo + need, true});
        }
        if ((rc = check_overlaps(ranges))) return rc;
        if (!has_rows && !grads) return MUON_OK;
        NormArgs a = base_args(d, p);
        a.x = rows_ptr(*x);
        a.dy = rows_ptr(*dy);
        a.y = rows_ptr(*dx);
        if (present(w)) {
            a.w = w->data;
            a.w_stride = w->stride;
        }
        a.mean = const_cast<float*>(mean);
        a.rstd = const_cast<float*>(rstd);
        if (present(dw)) {
            a.dw = dw->data;
            a.dw_stride = dw->stride;
        }
        if (present(db)) {
            a.db = db->data;
            a.db_stride = db->stride;
        }
        a.partial = static_cast<float*>(workspace);
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        rc = run_timed(MUON_KCLASS_NORM_BACKWARD, s, "norm backward",
                       [&] { return launch_norm_backward(!layer, d.dtype, p, a, s); });
        if (rc || need == 0) return rc;
        return run_timed(MUON_KCLASS_NORM_WGRAD, s, "norm weight gradient", [&] { return launch_norm_wgrad(a, s); });
    });
}

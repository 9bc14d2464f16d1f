// C ABI of the 8-bit matrices: quantising, reading back, and their products. Declared in
// include/muon_rocm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <iterator>
#include <string>
#include <vector>

#include "../../include/muon_rocm.h"
#include "abi_internal.hpp"
#include "blocks8.hpp"

#define MUON_API extern "C" __attribute__((visibility("default")))

namespace muon {
namespace {

static_assert(kBlock8 == MUON_BLOCK8, "block size");

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxCols = MUON_BLOCKS8_MAX_COLS;
constexpr int64_t kMaxSpan = int64_t(1) << 46;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of a launch

int fail(int code, const std::string& what) { return set_last_error(code, what); }

int64_t blocks_of(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }

// A [rows, cols] matrix of `dtype` with adjacent elements in a row.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype, const char* name, bool write,
                 std::vector<Range>& ranges) {
    const std::string who(name);
    if (dtype < MUON_DTYPE_F32 || dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (rows == 0 || cols == 0) return MUON_OK;
    if (!p) return fail(MUON_ERR_INVALID_ARG, who + " is NULL");
    if (stride < 0) return fail(MUON_ERR_INVALID_ARG, who + " has a negative stride");
    if (write && rows > 1 && stride < cols) return fail(MUON_ERR_ALIAS, who + " has rows that overlap");
    const __int128 span = __int128(rows - 1) * stride + cols;
    if (span > kMaxSpan) return fail(MUON_ERR_TOO_LARGE, who + " spans more than 2^46 elements");
    const int e = elem_size(dtype);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo % e) return fail(MUON_ERR_ALIGN, who + " is not aligned to its element");
    ranges.push_back({lo, lo + uintptr_t(span) * e, write});
    return MUON_OK;
}

Blocks8Ptr ptr_of(const blocks8* b) {
    return b ? Blocks8Ptr{b->codes, b->scales, b->ld, b->scale_ld} : Blocks8Ptr{nullptr, nullptr, 0, 0};
}

int check_product(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t products) {
    if (m < 0 || n < 0 || k < 0) return fail(MUON_ERR_INVALID_ARG, "negative dimension");
    if (dtype < MUON_DTYPE_F32 || dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (products != 0 && products != 8 && products != 16) return fail(MUON_ERR_INVALID_ARG, "products must be 0, 8 or 16");
    if (m > kMaxRows || n > kMaxRows || k > kMaxCols) return fail(MUON_ERR_TOO_LARGE, "rows above 2^30 or cols above 2^22");
    if (__int128(blocks_of(m)) * blocks_of(n) > kMaxThreads / 256 / 8 || __int128(m) * ((n + 7) / 8) > kMaxThreads)
        return fail(MUON_ERR_TOO_LARGE, "more of the product than a launch takes");
    return MUON_OK;
}

bool wide(int32_t dtype, int32_t products) { return products ? products == 16 : dtype == MUON_DTYPE_F32; }

}  // namespace

int check_blocks(const blocks8* b, const char* name, bool write, std::vector<Range>& ranges) {
    const std::string who(name);
    if (!b) return fail(MUON_ERR_INVALID_ARG, who + " is NULL");
    if (b->rows < 0 || b->cols < 0) return fail(MUON_ERR_INVALID_ARG, who + " has a negative dimension");
    if (b->tiles != 0 && b->tiles != 1) return fail(MUON_ERR_INVALID_ARG, who + "->tiles must be 0 or 1");
    if (b->rows > kMaxRows || b->cols > kMaxCols) return fail(MUON_ERR_TOO_LARGE, who + ": rows above 2^30 or cols above 2^22");
    if (b->rows == 0 || b->cols == 0) return MUON_OK;
    if (!b->codes || !b->scales) return fail(MUON_ERR_INVALID_ARG, who + ": codes or scales is NULL");
    const int64_t kb = blocks_of(b->cols), width = kb * kBlock8, powers = (kb + 3) / 4 * 4;
    if (b->ld < width || b->ld % 16) return fail(MUON_ERR_INVALID_ARG, who + "->ld must be a multiple of 16, cols rounded up to 128 at least");
    if (b->scale_ld < powers || b->scale_ld % 4)
        return fail(MUON_ERR_INVALID_ARG, who + "->scale_ld must be a multiple of 4, cols / 128 rounded up at least");
    if (b->ld > kMaxCols || b->scale_ld > kMaxCols) return fail(MUON_ERR_TOO_LARGE, who + ": ld above 2^22");
    const uintptr_t c = reinterpret_cast<uintptr_t>(b->codes), s = reinterpret_cast<uintptr_t>(b->scales);
    if (c % 16 || s % 4) return fail(MUON_ERR_ALIGN, who + ": codes not 16-byte or scales not 4-byte aligned");
    const int64_t srows = b->tiles ? blocks_of(b->rows) : b->rows;
    ranges.push_back({c, c + uintptr_t((b->rows - 1) * b->ld + width), write});
    ranges.push_back({s, s + uintptr_t((srows - 1) * b->scale_ld + powers), write});
    return MUON_OK;
}

}  // namespace muon

using namespace muon;

MUON_API int quantise8(const void* x, int64_t rows, int64_t cols, int64_t stride, int32_t dtype, const blocks8* direct,
                       const blocks8* transposed, void* stream) {
    return guarded([&]() -> int {
        if (rows < 0 || cols < 0) return fail(MUON_ERR_INVALID_ARG, "negative dimension");
        if (rows > kMaxRows || cols > kMaxRows) return fail(MUON_ERR_TOO_LARGE, "rows or cols above 2^30");
        if (!direct && !transposed) return fail(MUON_ERR_INVALID_ARG, "neither direct nor transposed is wanted");
        std::vector<Range> ranges;
        int rc = check_matrix(x, rows, cols, stride, dtype, "x", false, ranges);
        if (rc) return rc;
        if (direct) {
            if ((rc = check_blocks(direct, "direct", true, ranges))) return rc;
            if (direct->rows != rows || direct->cols != cols) return fail(MUON_ERR_INVALID_ARG, "direct is not [rows, cols]");
        }
        if (transposed) {
            if ((rc = check_blocks(transposed, "transposed", true, ranges))) return rc;
            if (transposed->rows != cols || transposed->cols != rows)
                return fail(MUON_ERR_INVALID_ARG, "transposed is not [cols, rows]");
        }
        if (direct && transposed && direct->tiles != transposed->tiles)
            return fail(MUON_ERR_INVALID_ARG, "direct and transposed differ in tiles");
        if ((rc = check_overlaps(ranges))) return rc;
        if (rows == 0 || cols == 0) return MUON_OK;
        if (blocks_of(rows) * blocks_of(cols) > kMaxThreads / 256)
            return fail(MUON_ERR_TOO_LARGE, "more elements than a launch takes");
        Quant8Args a{};
        a.x = x;
        a.stride = stride;
        a.rows = int32_t(rows);
        a.cols = int32_t(cols);
        a.col_blocks = int32_t(blocks_of(cols));
        a.direct = ptr_of(direct);
        a.transposed = ptr_of(transposed);
        const bool tiles = (direct ? direct : transposed)->tiles != 0;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_QUANTISE8, s, "quantise8", [&] { return launch_quantise8(dtype, tiles, a, s); });
    });
}

MUON_API int dequantise8(const blocks8* q, void* y, int64_t stride, int32_t dtype, void* stream) {
    return guarded([&]() -> int {
        std::vector<Range> ranges;
        int rc = check_blocks(q, "q", false, ranges);
        if (rc || (rc = check_matrix(y, q->rows, q->cols, stride, dtype, "y", true, ranges)) || (rc = check_overlaps(ranges)))
            return rc;
        if (q->rows == 0 || q->cols == 0) return MUON_OK;
        const int64_t vec = dtype == MUON_DTYPE_F32 ? 4 : 8, per_row = (q->cols + vec - 1) / vec;
        if (__int128(per_row) * q->rows > kMaxThreads - 2048) return fail(MUON_ERR_TOO_LARGE, "more elements than a launch takes");
        Dequant8Args a{};
        a.q = ptr_of(q);
        a.y = y;
        a.stride = stride;
        a.total = uint32_t(per_row * q->rows);
        a.cols = int32_t(q->cols);
        a.per_row = uint32_t(per_row);
        // division by a constant (Granlund and Montgomery 1994), as for strided norm rows
        int l = 0;
        while ((int64_t(1) << l) < per_row) ++l;
        a.shift = l;
        a.mul = uint32_t((((uint64_t(1) << l) - uint64_t(per_row)) << 32) / uint64_t(per_row) + 1);
        a.row_shift = q->tiles ? 7 : 0;
        a.dtype = dtype;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_DEQUANTISE8, s, "dequantise8", [&] { return launch_dequantise8(a, s); });
    });
}

MUON_API int matmul8_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t products, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
        const int rc = check_product(m, n, k, dtype, products);
        if (rc) return rc;
        *bytes = m == 0 || n == 0 ? 0 : plan_matmul8(m, n, k, wide(dtype, products)).partial_bytes;
        return MUON_OK;
    });
}

MUON_API int matmul8_plan(int64_t m, int64_t n, int64_t k, int32_t dtype, int32_t products, int32_t* out) {
    return guarded([&]() -> int {
        if (!out) return fail(MUON_ERR_INVALID_ARG, "out is NULL");
        const int rc = check_product(m, n, k, dtype, products);
        if (rc) return rc;
        const Mat8Plan p = m == 0 || n == 0 ? Mat8Plan{} : plan_matmul8(m, n, k, wide(dtype, products));
        const int32_t record[MUON_MATMUL8_PLAN_INTS] = {p.tile, p.splits, p.few, p.stream, p.waves, p.stream ? 0 : p.share};
        std::copy(std::begin(record), std::end(record), out);
        return MUON_OK;
    });
}

MUON_API int matmul8(const blocks8* a, const blocks8* b, void* c, int64_t ldc, int32_t dtype, int32_t products,
                     int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> int {
        std::vector<Range> ranges;
        int rc;
        if ((rc = check_blocks(a, "a", false, ranges)) || (rc = check_blocks(b, "b", false, ranges))) return rc;
        if (a->cols != b->cols) return fail(MUON_ERR_INVALID_ARG, "a and b differ in cols");
        const int64_t m = a->rows, n = b->rows, k = a->cols;
        if ((rc = check_product(m, n, k, dtype, products)) || (rc = check_matrix(c, m, n, ldc, dtype, "c", true, ranges)))
            return rc;
        const bool w = wide(dtype, products);
        if (m == 0 || n == 0) return MUON_OK;
        const Mat8Plan p = plan_matmul8(m, n, k, w);
        if (p.partial_bytes) {
            if (!workspace) return fail(MUON_ERR_WORKSPACE, "workspace is NULL");
            if (workspace_bytes < p.partial_bytes)
                return fail(MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(p.partial_bytes) + " bytes");
            const uintptr_t lo = reinterpret_cast<uintptr_t>(workspace);
            if (lo & 255) return fail(MUON_ERR_ALIGN, "workspace not 256-byte aligned");
            ranges.push_back({lo, lo + p.partial_bytes, true});
        }
        if ((rc = check_overlaps(ranges))) return rc;
        Mat8Args g{};
        g.a = a->codes;
        g.b = b->codes;
        g.as = a->scales;
        g.bs = b->scales;
        g.lda = a->ld;
        g.ldb = b->ld;
        g.lsa = a->scale_ld;
        g.lsb = b->scale_ld;
        g.sha = a->tiles ? 7 : 0;
        g.shb = b->tiles ? 7 : 0;
        g.m = int32_t(m);
        g.n = int32_t(n);
        g.steps = int32_t(blocks_of(k));
        g.dtype = dtype;
        g.accumulate = accumulate != 0;
        g.c = c;
        g.ldc = ldc;
        g.splits = p.splits;
        g.partial = static_cast<float*>(workspace);
        if (p.tile) {
            g.tiles_m = int32_t((m + p.tile - 1) / p.tile);
            g.tiles_n = int32_t((n + p.tile - 1) / p.tile);
        }
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        rc = run_timed(MUON_KCLASS_MATMUL8, s, "matmul8", [&] { return launch_matmul8(p, w, g, s); });
        if (rc || p.partial_bytes == 0) return rc;
        return run_timed(MUON_KCLASS_MATMUL8_JOIN, s, "matmul8 join", [&] { return launch_matmul8_join(g, s); });
    });
}

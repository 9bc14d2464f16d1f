// Matrices in 8 bits with a power of two for every 128 elements: kernel descriptors, the rule
// that gives a block its power, and the conversion. A block is 1 x 128 elements of a row, or
// 128 x 128. Its power is the least 2^e that brings its largest finite magnitude to 448, e4m3's
// largest value, or less. Dividing by it is exact, so an element is rounded once, by the
// conversion; and the matrix instructions of gfx950 take such powers (a byte, e + 127) beside
// their 8-bit operands, so that a product needs no arithmetic for its scales. Against a scale
// of amax / 448 at most half of the largest binade stays unused: e4m3 is a floating format, so
// that costs no precision but for magnitudes 2^-14 below the block's largest.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "train.hpp"

namespace muon {

constexpr int kBlock8 = 128;

// Codes [rows, ld] with zeros from the matrix's last column to a multiple of 128, powers
// [rows or row blocks, scale_ld]. codes == nullptr: not wanted.
struct Blocks8Ptr {
    uint8_t* codes;
    uint8_t* scales;
    int64_t ld, scale_ld;
};

struct Quant8Args {
    const void* x;
    int64_t stride;
    int32_t rows, cols;
    int32_t col_blocks;
    Blocks8Ptr direct, transposed;
};

struct Dequant8Args {
    Blocks8Ptr q;
    void* y;
    int64_t stride;
    uint32_t total;        // chunks of 16 bytes of y
    int32_t cols;
    uint32_t per_row;      // chunks of a row
    uint32_t mul;          // i / per_row = (mulhi(i, mul) + i) >> shift, 33-bit sum, for per_row > 1
    int32_t shift;
    int32_t row_shift;     // 7 for 128 x 128 blocks
    int32_t dtype;
};

// C[i][j] = sum_k A[i][k] B[j][k]
struct Mat8Args {
    const uint8_t *a, *b;      // codes
    const uint8_t *as, *bs;    // powers
    int64_t lda, ldb, lsa, lsb;
    int32_t sha, shb;          // row i's powers are row i >> sh
    int32_t m, n;
    int32_t steps;             // blocks of 128 along k
    int32_t dtype;             // of c
    int32_t accumulate;
    void* c;
    int64_t ldc;
    int32_t tiles_m, tiles_n;
    int32_t splits;            // parts of k, each a multiple of 4 steps but for the last
    int32_t share;             // few rows: waves that take turns along k
    float* partial;            // [splits][m][n], used when splits > 1
};

// How a product is cut.
struct Mat8Plan {
    int few;                   // groups of 16 rows of A, 0 where they are many
    int stream;                // few: 1 = a large B, through LDS
    int waves, share;          // few, a small B: of a block, and of those that take turns at the same rows of B
    int tile;                  // many: side of a block's tile, 128 or 256
    int splits;
    size_t partial_bytes;
};
Mat8Plan plan_matmul8(int64_t m, int64_t n, int64_t k, bool wide);

// ---- residual addition, RMS norm, 8-bit output ------------------------------------------
// Rows of `cols` elements, a stride apart each.
struct AddNormArgs {
    const void* x;         // forward: the block's output; backward: dy
    const void* r;         // forward: the residual, null = none; backward: dh, null = none
    void* h;               // forward: x + r in the residual's type, null without one; backward: h, read
    void* y;               // forward: the norm's output, null = not wanted; backward: d in x's type, null = not wanted
    void* d;               // backward: d in the residual's type
    int64_t x_stride, r_stride, h_stride, y_stride, d_stride;
    const void* w;         // null: factor 1
    float* rstd;
    Blocks8Ptr q;          // forward: the norm's output in 8 bits
    float* partial;        // backward: [chunks][cols]
    void* dw;              // backward: null = not wanted
    int32_t rows, cols;
    int32_t wdtype;
    int32_t chunks;        // blocks
    int32_t team_waves, teams;
    float eps, offset;
    double inv_cols;
};
NormPlan plan_add_norm(bool forward, int dtype, int64_t cols, int64_t rows);
hipError_t launch_add_norm_forward(int dtype, bool res32, const NormPlan& p, const AddNormArgs& a, hipStream_t s);
hipError_t launch_add_norm_backward(int dtype, bool res32, const NormPlan& p, const AddNormArgs& a, hipStream_t s);

hipError_t launch_quantise8(int dtype, bool tiles, const Quant8Args& a, hipStream_t s);
hipError_t launch_dequantise8(const Dequant8Args& a, hipStream_t s);
hipError_t launch_matmul8(const Mat8Plan& p, bool wide, const Mat8Args& a, hipStream_t s);
hipError_t launch_matmul8_join(const Mat8Args& a, hipStream_t s);

// Bits of f's magnitude, 0 where it is infinite or NaN.
__device__ __forceinline__ unsigned finite_bits(float f) {
    const unsigned u = __float_as_uint(f) & 0x7FFFFFFFu;
    return u >= 0x7F800000u ? 0u : u;
}

// The byte e + 127 of a block with largest magnitude `top` (bits): 448 is 1.75 2^8, so a
// mantissa up to 1.75 (0x600000) takes the exponent less 8 and a larger one carries into the
// next. At least 0: a block below 2^-118 loses what lies under 2^-136.
__device__ __forceinline__ unsigned block_power(unsigned top) {
    const unsigned e = (top + 0x1FFFFFu) >> 23;
    return e > 8u ? e - 8u : 0u;
}

// 2^-e and 2^e of the byte: 2^-127 (a byte of 0) is a subnormal, 255 is NaN.
__device__ __forceinline__ float power_inverse(unsigned byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float power_value(unsigned byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : max(byte << 23, 0x00400000u));
}
// 2^e as the instructions that widen codes take it: of a float they read the exponent alone.
__device__ __forceinline__ float power_operand(unsigned byte) { return __uint_as_float(byte << 23); }

// Four values of at most 448 to four codes, ties to even; an infinity or NaN gives NaN.
__device__ __forceinline__ unsigned pack_codes(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

}  // namespace muon

// Kernel descriptors and host-side launchers of the training-step operators beside the
// optimizer's own kernels: normalisation layers, many-tensor AdamW and the gradient norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace muon {

enum ElemType : int { kF32 = 0, kBF16 = 1, kF16 = 2 };  // MUON_DTYPE_*

inline int elem_size(int t) { return t == kF32 ? 4 : 2; }

// ---- normalisation layers --------------------------------------------------------
// Row r of a strided [rows, cols] tensor starts at data + (r / inner) s0 + (r % inner) s1
// elements.
struct RowsPtr {
    void* data;
    int64_t s0, s1;
};

struct NormArgs {
    RowsPtr x, y;              // backward: y is dx
    RowsPtr dy;                // backward only
    const void* w;             // [groups, cols] with stride w_stride; null = no weight (factor 1)
    const void* b;             // forward only; null = no bias
    int64_t w_stride, b_stride;
    float* mean;               // written by the forward pass, read by the backward pass; null for rms
    float* rstd;
    void* dw;                  // backward: gradients in wdtype, null = not wanted
    void* db;
    int64_t dw_stride, db_stride;
    float* partial;            // backward: [2][groups * chunks][cols] when chunks > 1
    int32_t rows_per_group;
    int32_t groups;
    int32_t cols;
    int32_t inner;             // >= 1
    uint32_t inner_mul;        // r / inner = (mulhi(r, inner_mul) + r) >> inner_shift, 33-bit sum, for inner > 1
    int32_t inner_shift;
    int32_t chunks;            // blocks of a group
    int32_t chunk_rows;        // rows of a block, for rows shorter than a vector
    int32_t team_waves;        // waves that share a row (rows of whole waves)
    int32_t teams;             // rows that a block takes at a time
    int32_t wdtype;
    float eps, offset;
    float inv_cols;
};

// Columns up to this fit the registers of one 1024-thread block, 16 a thread.
constexpr int kNormMaxCols = 16 * 1024;

// How the kernels split a norm's rows: `lanes` threads share a row (1 for rows shorter than
// a vector, 8 to 64, or the whole block), each holding `vecs` 16-byte vectors of it.
struct NormPlan {
    int lanes;
    int vecs;
    int teams;         // rows that a block takes at a time
    int threads;       // of a block
    int chunks;        // blocks of a group
    int chunk_rows;    // rows of a block (lanes == 1)
    bool stream;       // backward: inputs too large for the caches
};
NormPlan plan_norm_forward(int dtype, int64_t cols, int64_t rows_per_group, int64_t groups);
NormPlan plan_norm_backward(int dtype, int64_t cols, int64_t rows_per_group, int64_t groups);

hipError_t launch_norm_forward(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_wgrad(const NormArgs& a, hipStream_t s);

// ---- rotary positions ---------------------------------------------------------------
struct RotaryRows {
    void* data;
    int64_t sb, st, sh;    // batch, token, head
};

struct RotaryArgs {
    RotaryRows x, y;
    const void* pos;       // axis adjacent
    int64_t pb, pt;
    const double* freq;    // turns per unit of position, a pair each
    const int32_t* axis;   // of each pair
    uint32_t rows;         // batch * tokens
    uint32_t tokens;
    int32_t heads, dim, pairs, axes;
    int32_t pos_type;      // 0 int32, 1 int64, 2 float
    int32_t block_rows;    // tokens of a block
    uint32_t heads_mul;    // i / heads, as inner_mul above
    int32_t heads_shift;
    int32_t lane_bits;     // log2 of the threads that share a head
    float sign;            // -1: turned back
};
hipError_t launch_rotary(int dtype, bool adjacent, const RotaryArgs& a, hipStream_t s);

// ---- many tensors in one launch ----------------------------------------------------
// A table in device memory holds the descriptors and, for every block, its tensor. Both
// are written by kernels whose arguments carry the descriptors: no copy from host memory,
// so nothing of the caller's has to outlive the call.
constexpr int kQBlock = 256;             // elements of 8-bit state that share a scale
constexpr int kMultiThreads = 256;       // of a block of the AdamW step
constexpr int kMultiBlockElems = 16 * kMultiThreads;  // its elements

struct MultiDesc {
    float* w;
    void* copy;            // null = not wanted
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    int64_t n;
    int32_t blk_begin;
    int32_t index;         // position in the caller's list
    float lr_scale, wd_scale;
    int8_t g_type, copy_type, bits, pad_;
    int32_t pad2_;
};

constexpr int kMultiPerLaunch = 32;
struct MultiDescArgs {
    MultiDesc d[kMultiPerLaunch];
    MultiDesc* table;
    int32_t first, n;
};

// A step's scalars that follow from its counter and learning rate.
struct MultiScalars {
    float lr_bc1;          // lr / (1 - beta1^t)
    float inv_sqrt_bc2;    // 1 / sqrt(1 - beta2^t)
    double lr_wd;          // lr * weight_decay
    uint32_t key;          // of (seed, step)
    uint32_t pad_;
};

struct MultiArgs {
    const MultiDesc* table;
    const int32_t* tensor_of_block;
    int32_t blocks;
    int32_t bits;          // 8 or 32: the width of all states; 0: both occur
    float beta1, beta2, one_minus_beta1, one_minus_beta2;
    float eps;
    MultiScalars host;     // used where `scalars` is null
    const MultiScalars* scalars;  // on the device
    const float* grad_scale;
};

struct MultiScalarArgs {
    MultiScalars* out;
    int64_t* counter;
    const float* lr;       // null: lr_host
    float lr_host, beta1, beta2, weight_decay;
    uint32_t seed_key;     // of the seed alone
};

struct GradDesc {
    void* g;
    int64_t n;
    int32_t blk_begin;
    int32_t blk_end;
    int32_t type;
    int32_t pad_;
};

constexpr int kGradPerLaunch = 96;
struct GradDescArgs {
    GradDesc d[kGradPerLaunch];
    GradDesc* table;
    int32_t first, n;
};

struct GradArgs {
    const GradDesc* table;
    const int32_t* tensor_of_block;
    double* partial;       // one a block
    int64_t block_elems;   // of every tensor
    int32_t count, blocks;
    float max_norm;
    float* total;
    float* norms;          // null = not wanted
    const float* factor;   // grad_scale
};

__host__ __device__ inline uint32_t mix32(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}

hipError_t launch_multi_table(const MultiDescArgs& a, hipStream_t s);
hipError_t launch_multi_map(const MultiDesc* table, int count, int32_t* map, int blocks, hipStream_t s);
hipError_t launch_multi_scalars(const MultiScalarArgs& a, hipStream_t s);
hipError_t launch_multi_step(const MultiArgs& a, hipStream_t s);
hipError_t launch_grad_table(const GradDescArgs& a, hipStream_t s);
hipError_t launch_grad_map(const GradDesc* table, int count, int32_t* map, int blocks, hipStream_t s);
hipError_t launch_grad_norm(const GradArgs& a, hipStream_t s);
hipError_t launch_grad_total(const GradArgs& a, hipStream_t s);
hipError_t launch_grad_scale(const GradArgs& a, hipStream_t s);

}  // namespace muon

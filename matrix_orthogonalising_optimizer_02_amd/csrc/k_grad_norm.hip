// Norms of many gradients and the clip factor, and their scaling in place.
//   n_i = sqrt(sum g^2),  total = sqrt(sum n_i^2),  factor = min(1, max_norm / (total + 1e-6))
// HBM-bound: the gradients are read once. A block sums the squares of one run of a tensor
// in fp64 (fp32 squares would overflow from 1.8e19 and vanish below 1e-23; the vector
// units have fp64 to spare at this rate) and leaves one partial sum; a second launch adds
// them, one block a tensor and one for the total, each in a fixed order. Loads carry the
// non-temporal hint: 700 M fp32 elements in 405 us (6.9 TB/s), 459 us without; bf16 209 us.
// Scaling in place: 1074 us (5.2 TB/s), 5 us where the factor is 1.
#include "lanes.hpp"
#include "train.hpp"

namespace muon {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf162_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));

// Sum over a block of kThreads; the result in thread 0.
template <int kThreads>
__device__ __forceinline__ double block_sum_d(double v) {
    __shared__ double red[kThreads / 64];
    v = wave_sum_d(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = red[0];
    for (int i = 1; i < kThreads / 64; ++i) s += red[i];
    return s;
}

__device__ __forceinline__ double square_add(float f, double acc) { return fma((double)f, (double)f, acc); }

// The squares of the elements of 16 bytes, added to acc[0..3].
template <int T>
__device__ __forceinline__ void add16(u32x4 r, double* acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const unsigned u = r[e];
        if constexpr (T == kF32) {
            acc[e] = square_add(__uint_as_float(u), acc[e]);
        } else if constexpr (T == kBF16) {
            acc[e] = square_add(__uint_as_float(u << 16), acc[e]);
            acc[e] = square_add(__uint_as_float(u & 0xFFFF0000u), acc[e]);
        } else {
            const half2_t h = __builtin_bit_cast(half2_t, u);
            acc[e] = square_add((float)h[0], acc[e]);
            acc[e] = square_add((float)h[1], acc[e]);
        }
    }
}

template <int T>
__device__ __forceinline__ float element(const void* g, int64_t i) {
    if constexpr (T == kF32) return reinterpret_cast<const float*>(g)[i];
    else if constexpr (T == kBF16) return bf2f(reinterpret_cast<const unsigned short*>(g)[i]);
    else return (float)reinterpret_cast<const _Float16*>(g)[i];
}

template <int T>
__device__ __forceinline__ double run_squares(const void* g, int64_t begin, int64_t end) {
    constexpr int kVec = T == kF32 ? 4 : 8, kUnroll = 8;
    constexpr int kSize = T == kF32 ? 4 : 2;
    const char* p = reinterpret_cast<const char*>(g);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    int64_t i = begin;
    for (; i + 256 * kVec * kUnroll <= end; i += 256 * kVec * kUnroll) {
        u32x4 r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) r[k] = stream16(p + (i + (int64_t)(k * 256 + threadIdx.x) * kVec) * kSize);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) add16<T>(r[k], acc);
    }
    for (; i + 256 * kVec <= end; i += 256 * kVec) add16<T>(stream16(p + (i + (int64_t)threadIdx.x * kVec) * kSize), acc);
    for (i += threadIdx.x; i < end; i += 256) acc[0] = square_add(element<T>(g, i), acc[0]);
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

__global__ __launch_bounds__(256) void k_grad_norm(GradArgs a) {
    const GradDesc& d = a.table[a.tensor_of_block[blockIdx.x]];
    const int64_t begin = (int64_t)(blockIdx.x - d.blk_begin) * a.block_elems;
    const int64_t end = min(begin + a.block_elems, d.n);
    double s;
    if (d.type == kF32) s = run_squares<kF32>(d.g, begin, end);
    else if (d.type == kBF16) s = run_squares<kBF16>(d.g, begin, end);
    else s = run_squares<kF16>(d.g, begin, end);
    s = block_sum_d<256>(s);
    if (threadIdx.x == 0) a.partial[blockIdx.x] = s;
}

constexpr int kTotalThreads = 1024;
__global__ __launch_bounds__(kTotalThreads) void k_grad_total(GradArgs a) {
    const int t = blockIdx.x;
    const bool total = t == a.count;
    const int begin = total ? 0 : a.table[t].blk_begin, end = total ? a.blocks : a.table[t].blk_end;
    double s = 0.0;
    for (int i = begin + threadIdx.x; i < end; i += kTotalThreads) s += a.partial[i];
    s = sqrt(block_sum_d<kTotalThreads>(s));
    if (threadIdx.x != 0) return;
    if (!total) {
        if (a.norms) a.norms[t] = (float)s;
        return;
    }
    const double f = (double)a.max_norm / (s + 1e-6);
    a.total[0] = (float)s;
    a.total[1] = f >= 1.0 ? 1.f : (float)f;  // a NaN stays one
}

// 16 bytes of elements times f, rounded to their type.
template <int T>
__device__ __forceinline__ u32x4 scale16(u32x4 r, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const unsigned u = r[e];
        if constexpr (T == kF32) {
            r[e] = __float_as_uint(__uint_as_float(u) * f);
        } else if constexpr (T == kBF16) {
            const float2_t t = {__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f};
            r[e] = __builtin_bit_cast(unsigned, __builtin_convertvector(t, bf162_t));
        } else {
            const half2_t h = __builtin_bit_cast(half2_t, u);
            const float2_t t = {(float)h[0] * f, (float)h[1] * f};
            r[e] = __builtin_bit_cast(unsigned, __builtin_convertvector(t, half2_t));
        }
    }
    return r;
}

template <int T>
__device__ __forceinline__ void run_scale(void* g, float f, int64_t begin, int64_t end) {
    constexpr int kVec = T == kF32 ? 4 : 8, kSize = T == kF32 ? 4 : 2, kUnroll = 4;
    char* p = reinterpret_cast<char*>(g) + (int64_t)threadIdx.x * kVec * kSize;
    int64_t i = begin;
    for (; i + 256 * kVec * kUnroll <= end; i += 256 * kVec * kUnroll) {
        u32x4 r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) r[k] = stream16(p + (i + k * 256 * kVec) * kSize);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) put_stream16(p + (i + k * 256 * kVec) * kSize, scale16<T>(r[k], f));
    }
    for (; i + 256 * kVec <= end; i += 256 * kVec) put_stream16(p + i * kSize, scale16<T>(stream16(p + i * kSize), f));
    for (i += threadIdx.x; i < end; i += 256) {
        const float v = element<T>(g, i) * f;
        if constexpr (T == kF32) reinterpret_cast<float*>(g)[i] = v;
        else if constexpr (T == kBF16) reinterpret_cast<unsigned short*>(g)[i] = f2bf(v);
        else reinterpret_cast<_Float16*>(g)[i] = (_Float16)v;
    }
}

__global__ __launch_bounds__(256) void k_grad_scale(GradArgs a) {
    const float f = *a.factor;
    if (f == 1.f) return;
    const GradDesc& d = a.table[a.tensor_of_block[blockIdx.x]];
    const int64_t begin = (int64_t)(blockIdx.x - d.blk_begin) * a.block_elems;
    const int64_t end = min(begin + a.block_elems, d.n);
    if (d.type == kF32) run_scale<kF32>(d.g, f, begin, end);
    else if (d.type == kBF16) run_scale<kBF16>(d.g, f, begin, end);
    else run_scale<kF16>(d.g, f, begin, end);
}

}  // namespace

hipError_t launch_grad_norm(const GradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_grad_norm, dim3(a.blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_total(const GradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_grad_total, dim3(unsigned(a.count) + 1), dim3(kTotalThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const GradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_grad_scale, dim3(a.blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace muon

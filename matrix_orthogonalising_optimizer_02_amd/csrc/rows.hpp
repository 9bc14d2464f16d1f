// Rows of a tensor in registers: element types, a lane's vectors of a row, the threads that
// share a row and their sums. Shared by the kernels that hold a row between its statistics
// and its output.
#pragma once

#include "lanes.hpp"
#include "train.hpp"

namespace muon {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf162_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));

template <int T>
struct Elem;
template <>
struct Elem<kF32> {
    typedef float type;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ void unpack(u32x4 r, float* f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(r[e]);
    }
    static __device__ __forceinline__ u32x4 pack(const float* f) {
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __float_as_uint(f[e]);
        return r;
    }
};
template <>
struct Elem<kBF16> {
    typedef __bf16 type;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ void unpack(u32x4 r, float* f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(r[e] << 16);
            f[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ u32x4 pack(const float* f) {
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = __builtin_bit_cast(unsigned, __builtin_convertvector((float2_t){f[2 * e], f[2 * e + 1]}, bf162_t));
        return r;
    }
};
template <>
struct Elem<kF16> {
    typedef _Float16 type;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ void unpack(u32x4 r, float* f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned u = r[e];  // a bit cast of a vector's element reads element 0
            const half2_t h = __builtin_bit_cast(half2_t, u);
            f[2 * e] = (float)h[0];
            f[2 * e + 1] = (float)h[1];
        }
    }
    static __device__ __forceinline__ u32x4 pack(const float* f) {
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] = __builtin_bit_cast(unsigned, __builtin_convertvector((float2_t){f[2 * e], f[2 * e + 1]}, half2_t));
        return r;
    }
};

// A lane's vector of a row of at least kVec elements. The last vector of a row whose length
// kVec does not divide starts kVec elements before the row's end, so that every access is
// whole and unconditional; its first `skip` elements are the vector before's, count in no
// sum and are written twice with the same bits. A lane past the row's end has skip == kVec
// and writes nothing.
template <int kVec>
struct Span {
    int col, skip;
    __device__ __forceinline__ Span(int cols, int index) {
        const int c = index * kVec;
        col = min(c, cols - kVec);
        skip = min(c - col, kVec);
    }
};

// f with the elements that do not count set to 0. kExact: the row fills all lanes' vectors.
template <bool kExact, int kVec>
__device__ __forceinline__ float counted(const Span<kVec>& sp, int e, float f) {
    return kExact || e >= sp.skip ? f : 0.f;
}

// kVec weights (or biases) from element `at` of a row of type `wdtype`, in fp32.
template <int kVec>
__device__ __forceinline__ void load_params(const void* base, int64_t at, int wdtype, float* f) {
    if (wdtype == kF32) {
        const float* p = reinterpret_cast<const float*>(base) + at;
#pragma unroll
        for (int q = 0; q < kVec / 4; ++q) Elem<kF32>::unpack(load16(p + 4 * q), f + 4 * q);
    } else {
        // the two 16-bit types differ in the conversion alone
        const unsigned short* p = reinterpret_cast<const unsigned short*>(base) + at;
        if constexpr (kVec == 8) {
            const u32x4 r = load16(p);
            if (wdtype == kBF16) Elem<kBF16>::unpack(r, f);
            else Elem<kF16>::unpack(r, f);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = wdtype == kBF16 ? bf2f(p[e]) : (float)__builtin_bit_cast(_Float16, p[e]);
        }
    }
}

__device__ __forceinline__ void store_param(void* base, int64_t at, int wdtype, float f) {
    if (wdtype == kF32) reinterpret_cast<float*>(base)[at] = f;
    else if (wdtype == kBF16) reinterpret_cast<unsigned short*>(base)[at] = f2bf(f);
    else reinterpret_cast<_Float16*>(base)[at] = (_Float16)f;
}

// The threads that share a row: kLanes of a wave, or (0) a.team_waves whole waves.
template <int kLanes>
struct Team {
    int lane, team, lanes, teams;
    __device__ __forceinline__ Team(int team_waves, int teams_) {
        if constexpr (kLanes != 0) {
            lanes = kLanes;
            lane = threadIdx.x & (kLanes - 1);
            team = threadIdx.x / (kLanes ? kLanes : 1);
            teams = blockDim.x / (kLanes ? kLanes : 1);
        } else {
            lanes = team_waves * 64;
            teams = teams_;
            team = __builtin_amdgcn_readfirstlane((int)threadIdx.x / lanes);
            lane = threadIdx.x - team * lanes;
        }
    }
};

constexpr int kMaxWaves = 16;
constexpr int kSubThreads = 512;  // most threads of a block whose rows share a wave

// kCount sums over the row's lanes. Teams of several waves exchange them through `red`,
// one slot a wave, behind one barrier of the whole block: every team runs the same number
// of sums. The caller alternates between two buffers, so that the next sum's barrier
// stands between a buffer's reads and its next writes.
template <int kLanes, int kCount>
__device__ __forceinline__ void row_sums(float (&v)[kCount], float (*red)[kCount], const Team<kLanes>& t, int team_waves) {
    if constexpr (kLanes != 0) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] = lanes_sum<kLanes>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] = lanes_sum<64>(v[i]);
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < kCount; ++i) red[threadIdx.x >> 6][i] = v[i];
        }
        __syncthreads();
        // at most 16 waves: a lane of each 16 reads a wave's sums, and they add up by exchange
        const int slot = threadIdx.x & 15;
        const bool one = slot < team_waves;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const float r = red[one ? t.team * team_waves + slot : 0][i];
            v[i] = lanes_sum<16>(one ? r : 0.f);
        }
    }
}

}  // namespace muon

// Device helpers shared by the training-step kernels: reductions across the lanes of a
// wave without LDS, and unaligned 16-byte accesses.
#pragma once

#include "common.hpp"

namespace muon {

// 16 bytes at any element alignment (global memory takes unaligned dword accesses).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 load16(const void* p) { return *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void store16(void* p, u32x4 v) { *reinterpret_cast<u32x4_any*>(p) = v; }
// The same with the non-temporal hint, for data that a kernel touches once.
__device__ __forceinline__ u32x4 stream16(const void* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ void put_stream16(void* p, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
}

template <int kCtrl>
__device__ __forceinline__ unsigned dpp(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}

// op over aligned groups of kLanes lanes, the same bits in every lane of the group (op
// commutes). Steps 1 to 8 exchange through DPP (pairs, quads, mirrored halves of a
// 16-lane row), 16 and 32 through the row and half-wave swaps.
template <int kLanes, class Op>
__device__ __forceinline__ unsigned lanes_reduce(unsigned v, Op op) {
    if constexpr (kLanes >= 2) v = op(v, dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
    if constexpr (kLanes >= 4) v = op(v, dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
    if constexpr (kLanes >= 8) v = op(v, dpp<0x141>(v));   // row_half_mirror
    if constexpr (kLanes >= 16) v = op(v, dpp<0x140>(v));  // row_mirror
    if constexpr (kLanes >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(s[0], s[1]);
    }
    if constexpr (kLanes >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(s[0], s[1]);
    }
    return v;
}

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
    return __uint_as_float(lanes_reduce<kLanes>(__float_as_uint(v), [](unsigned a, unsigned b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// Largest of the bit patterns: of magnitudes, the largest, with infinities above every
// finite one and NaN above those.
template <int kLanes>
__device__ __forceinline__ unsigned lanes_max(unsigned v) {
    return lanes_reduce<kLanes>(v, [](unsigned a, unsigned b) { return a > b ? a : b; });
}

}  // namespace muon

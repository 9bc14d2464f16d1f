// Quantising a matrix to 8 bits with a power of two for every 128 elements, and reading it
// back (blocks8.hpp has the rule).
#include "blocks8.hpp"
#include "rows.hpp"

namespace muon {
namespace {

// Magnitudes as unsigned integers, 16 bits each for the 16-bit types: `kWords` dwords for 8
// elements, with 0 in the place of an infinity or NaN (the sum of such a magnitude and the
// distance of the infinity from 2^15 or 2^31 has its top bit set).
template <int T>
struct Magnitudes {
    static constexpr int kWords = T == kF32 ? 8 : 4;
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    typedef short i16x2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ unsigned of(unsigned w) {
        if constexpr (T == kF32) {
            const unsigned m = w & 0x7FFFFFFFu;
            return m & ~(unsigned)((int)(m + 0x00800000u) >> 31);
        } else {
            const unsigned m = w & 0x7FFF7FFFu;
            const unsigned short gap = T == kBF16 ? 0x0080 : 0x0400;
            const u16x2 past = __builtin_bit_cast(u16x2, m) + (u16x2){gap, gap};
            return m & ~__builtin_bit_cast(unsigned, __builtin_bit_cast(i16x2, past) >> (i16x2){15, 15});
        }
    }
    static __device__ __forceinline__ unsigned most(unsigned a, unsigned b) {
        if constexpr (T == kF32) return max(a, b);
        else return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
    }
    // the larger half of a dword of two, in fp32's bits
    static __device__ __forceinline__ unsigned half_bits(unsigned m) {
        if constexpr (T == kF32) return m;
        else if constexpr (T == kBF16) return m << 16;
        else return __float_as_uint((float)__builtin_bit_cast(_Float16, (unsigned short)m));
    }
    static __device__ __forceinline__ unsigned bits(unsigned m) {
        if constexpr (T == kF32) return m;
        else return half_bits(max(m & 0xFFFFu, m >> 16));
    }
    // element e's magnitude of `kWords` dwords, in fp32's bits
    static __device__ __forceinline__ unsigned element(const unsigned* w, int e) {
        if constexpr (T == kF32) return w[e];
        else return half_bits((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
    }
};

__device__ __forceinline__ void put_power(uint8_t* row, int at, int blocks, unsigned byte) {
    row[at] = (uint8_t)byte;
    if (at == blocks - 1)  // the rest of the last four, which products read and do not use
        for (int i = blocks; i & 3; ++i) row[i] = 0;
}

// A block of 256 threads takes 128 x 128 elements, a thread 8 x 8 of them in registers: 16
// threads share a row (its largest magnitude is a reduction over 16 lanes, its codes leave as
// 128 contiguous bytes), and the 8 rows of a thread are 8 contiguous bytes of the transposed
// matrix, which is put together in 16 KB of LDS. So both forms cost one read of x.
// HBM-bound: [8192, 5120] bf16 into both forms 34 us (5.0 TB/s), [15360, 5120] fp32 in 128 x 128
// blocks into both 78 us (6.1 TB/s).
template <int T, bool kTiles, bool kDirect, bool kTransposed>
__global__ __launch_bounds__(256) void k_quantise8(Quant8Args a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    __shared__ unsigned tops[4][kBlock8];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kTransposed ? kBlock8 * kBlock8 : 16];
    const int br = blockIdx.x / a.col_blocks, bc = blockIdx.x - br * a.col_blocks;
    const int row_blocks = (a.rows + kBlock8 - 1) / kBlock8;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int row0 = br * kBlock8 + rg * 8, col0 = bc * kBlock8 + cg * 8;
    typedef Magnitudes<T> M;
    constexpr int kParts = 8 / E::kVec, kWords = M::kWords;
    auto most = [](unsigned x, unsigned y) { return M::most(x, y); };
    u32x4 raw[8][kParts];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const elem* x = reinterpret_cast<const elem*>(a.x) + (int64_t)(row0 + p) * a.stride + col0;
        if (row0 + p < a.rows && col0 + 8 <= a.cols) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) raw[p][q] = load16(x + q * E::kVec);
        } else {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = row0 + p < a.rows && col0 + e < a.cols ? (float)x[e] : 0.f;
#pragma unroll
            for (int q = 0; q < kParts; ++q) raw[p][q] = E::pack(f + q * E::kVec);
        }
    }
    unsigned row_top[8], cols_top[kWords], col_top[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const unsigned m = M::of(raw[p][i >> 2][i & 3]);
            row_top[p] = i ? most(row_top[p], m) : m;
            cols_top[i] = p ? most(cols_top[i], m) : m;
        }
    if constexpr (kTiles) {
        unsigned top = row_top[0];
#pragma unroll
        for (int p = 1; p < 8; ++p) top = most(top, row_top[p]);
        top = lanes_max<64>(M::bits(top));
        if ((threadIdx.x & 63) == 0) tops[wave][0] = top;
        __syncthreads();
        top = max(max(tops[0][0], tops[1][0]), max(tops[2][0], tops[3][0]));
#pragma unroll
        for (int e = 0; e < 8; ++e) row_top[e] = col_top[e] = top;
    } else {
        if constexpr (kDirect) {
#pragma unroll
            for (int p = 0; p < 8; ++p) row_top[p] = M::bits(lanes_reduce<16>(row_top[p], most));
        }
        if constexpr (kTransposed) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {  // over the four 16-lane rows of the wave
                auto s = __builtin_amdgcn_permlane16_swap(cols_top[i], cols_top[i], false, false);
                const unsigned m = most(s[0], s[1]);
                s = __builtin_amdgcn_permlane32_swap(m, m, false, false);
                cols_top[i] = most(s[0], s[1]);
            }
            if ((threadIdx.x & 48) == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) tops[wave][cg * 8 + e] = M::element(cols_top, e);
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = cg * 8 + e;
                col_top[e] = max(max(tops[0][c], tops[1][c]), max(tops[2][c], tops[3][c]));
            }
        }
    }
    auto row_of = [&](int p, float (&v)[8]) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) E::unpack(raw[p][q], v + q * E::kVec);
    };
    if constexpr (kDirect) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (row0 + p >= a.rows) break;
            const unsigned byte = block_power(row_top[p]);
            const float s = power_inverse(byte);
            float v[8];
            row_of(p, v);
            u32x2 w;
            w.x = pack_codes(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
            w.y = pack_codes(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
            *reinterpret_cast<u32x2*>(a.direct.codes + (int64_t)(row0 + p) * a.direct.ld + col0) = w;
            if (cg == 0 && (!kTiles || (rg == 0 && p == 0)))
                put_power(a.direct.scales + (int64_t)(kTiles ? br : row0 + p) * a.direct.scale_ld, bc, a.col_blocks, byte);
        }
    }
    if constexpr (kTransposed) {
        // eight rows of a column are an 8-byte slot of the turned tile's row; slot g of row c
        // sits at g ^ (c / 8), so that the 16 column groups of a write meet 16 slots
        float v[8][8];
#pragma unroll
        for (int p = 0; p < 8; ++p) row_of(p, v[p]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = power_inverse(block_power(col_top[e]));
            u32x2 w;
            w.x = pack_codes(v[0][e] * s, v[1][e] * s, v[2][e] * s, v[3][e] * s);
            w.y = pack_codes(v[4][e] * s, v[5][e] * s, v[6][e] * s, v[7][e] * s);
            *reinterpret_cast<u32x2*>(turned + (cg * 8 + e) * kBlock8 + ((rg ^ cg) & 15) * 8) = w;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = q * 32 + (threadIdx.x >> 3), j = threadIdx.x & 7, g = c >> 3;
            const u32x4 r = *reinterpret_cast<const u32x4*>(turned + c * kBlock8 + ((j ^ (g >> 1)) & 7) * 16);
            const u32x4 w = g & 1 ? u32x4{r.z, r.w, r.x, r.y} : r;
            if (bc * kBlock8 + c < a.cols)
                *reinterpret_cast<u32x4*>(a.transposed.codes + (int64_t)(bc * kBlock8 + c) * a.transposed.ld + br * kBlock8 +
                                          j * 16) = w;
        }
        if constexpr (kTiles) {
            if (threadIdx.x == 0)
                put_power(a.transposed.scales + (int64_t)bc * a.transposed.scale_ld, br, row_blocks, block_power(col_top[0]));
        } else if (threadIdx.x < kBlock8 && bc * kBlock8 + (int)threadIdx.x < a.cols) {
            const int c = threadIdx.x;
            const unsigned top = max(max(tops[0][c], tops[1][c]), max(tops[2][c], tops[3][c]));
            put_power(a.transposed.scales + (int64_t)(bc * kBlock8 + c) * a.transposed.scale_ld, br, row_blocks,
                      block_power(top));
        }
    }
}

// A lane's store is 16 bytes next to its neighbours', kChunks of them a thread, all asked for before
// the first is written. HBM-bound: [8192, 5120] into bf16 18.5 us (two stores of a lane next to
// each other, half of what its neighbours fill, took 26).
constexpr int kChunks = 2;
template <int T, bool kStream>
__global__ __launch_bounds__(256) void k_dequantise8(Dequant8Args a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    constexpr int kVec = E::kVec, kWords = kVec / 4;
    unsigned w[kChunks][kWords], row[kChunks];
    float s[kChunks];
    int col[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        const unsigned i = blockIdx.x * (256u * kChunks) + k * 256u + threadIdx.x;
        row[k] = i;
        if (a.per_row > 1) row[k] = (unsigned)(((uint64_t)__umulhi(i, a.mul) + i) >> a.shift);
        col[k] = i < a.total ? (int)(i - row[k] * a.per_row) * kVec : a.cols;
        if (i < a.total) {
            const unsigned* p = reinterpret_cast<const unsigned*>(a.q.codes + (int64_t)row[k] * a.q.ld + col[k]);
            if constexpr (kWords == 2) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(p);
                w[k][0] = v.x;
                w[k][1] = v.y;
            } else {
                w[k][0] = *p;
            }
            s[k] = power_value(a.q.scales[(int64_t)(row[k] >> a.row_shift) * a.q.scale_ld + col[k] / kBlock8]);
        }
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        if (col[k] >= a.cols) break;
        float f[kVec];
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k][q], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k][q], true);
            f[4 * q] = lo[0] * s[k];
            f[4 * q + 1] = lo[1] * s[k];
            f[4 * q + 2] = hi[0] * s[k];
            f[4 * q + 3] = hi[1] * s[k];
        }
        elem* y = reinterpret_cast<elem*>(a.y) + (int64_t)row[k] * a.stride + col[k];
        if (col[k] + kVec <= a.cols) {
            if constexpr (kStream) put_stream16(y, E::pack(f));
            else store16(y, E::pack(f));
        } else {
#pragma unroll
            for (int q = 0; q < kVec; ++q)
                if (col[k] + q < a.cols) y[q] = (elem)f[q];
        }
    }
}

template <int T, bool kTiles>
hipError_t launch_sides(const Quant8Args& a, hipStream_t s) {
    const int64_t blocks = int64_t((a.rows + kBlock8 - 1) / kBlock8) * a.col_blocks;
    const dim3 grid((unsigned)blocks), block(256);
    if (a.direct.codes && a.transposed.codes) hipLaunchKernelGGL((k_quantise8<T, kTiles, true, true>), grid, block, 0, s, a);
    else if (a.direct.codes) hipLaunchKernelGGL((k_quantise8<T, kTiles, true, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_quantise8<T, kTiles, false, true>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantise8(int dtype, bool tiles, const Quant8Args& a, hipStream_t s) {
    if (dtype == kF32) return tiles ? launch_sides<kF32, true>(a, s) : launch_sides<kF32, false>(a, s);
    if (dtype == kBF16) return tiles ? launch_sides<kBF16, true>(a, s) : launch_sides<kBF16, false>(a, s);
    return tiles ? launch_sides<kF16, true>(a, s) : launch_sides<kF16, false>(a, s);
}

template <int T>
static hipError_t launch_back(const Dequant8Args& a, hipStream_t s) {
    const dim3 grid((a.total + (256 * kChunks - 1)) / (256 * kChunks)), block(256);
    // streaming stores where they fill whole pieces of 64 bytes
    const int64_t size = sizeof(typename Elem<T>::type);
    if (((reinterpret_cast<uintptr_t>(a.y) | uintptr_t((a.stride | a.cols) * size)) & 63) == 0)
        hipLaunchKernelGGL((k_dequantise8<T, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_dequantise8<T, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dequantise8(const Dequant8Args& a, hipStream_t s) {
    return a.dtype == kF32 ? launch_back<kF32>(a, s) : a.dtype == kBF16 ? launch_back<kBF16>(a, s) : launch_back<kF16>(a, s);
}

}  // namespace muon

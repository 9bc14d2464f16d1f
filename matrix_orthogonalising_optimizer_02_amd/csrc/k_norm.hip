// Normalisation layers and their gradients. For a row x of H columns in group g:
//   mean = (1/H) sum x (0 for the rms form), rstd = 1 / sqrt((1/H) sum (x - mean)^2 + eps)
//   h = (x - mean) rstd,   y = h (offset + w[g]) + b[g]
// and from dy, with a = dy (offset + w[g]):
//   dx = rstd (a - (1/H) sum a - h (1/H) sum a h)     (rms: without the first sum)
//   dw[g] = sum over the group's rows of dy h,   db[g] = sum of dy
//
// Both passes are HBM-bound: forward reads x and writes y, backward reads x and dy and
// writes dx, and a row stays in registers between its statistics and its output, so every
// element moves once. A row is shared by 8 to 64 lanes of a wave or by the waves of a
// block, 16 bytes a lane and load; a block walks through consecutive rows of one group
// with that group's weights in registers, and asks for the next row before it reduces the
// present one. Statistics are two-pass over the registers (the mean first, then the
// squares of the differences), all sums in fp32 in a fixed order.
#include "lanes.hpp"
#include "train.hpp"

#include <algorithm>

namespace muon {
namespace {

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

// The vector at p, of which the first `valid` elements exist; zeros in the others.
template <int T>
__device__ __forceinline__ u32x4 load_raw(const typename Elem<T>::type* p, int valid) {
    constexpr int kVec = Elem<T>::kVec;
    u32x4 r = {0u, 0u, 0u, 0u};
    if (valid >= kVec) {
        r = load16(p);
    } else if (valid > 0) {
        if constexpr (T == kF32) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid) r[e] = __float_as_uint(p[e]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid)
                    r[e / 2] |= (unsigned)reinterpret_cast<const unsigned short*>(p)[e] << (16 * (e & 1));
        }
    }
    return r;
}

template <int T>
__device__ __forceinline__ void store_raw(typename Elem<T>::type* p, u32x4 r, int valid) {
    constexpr int kVec = Elem<T>::kVec;
    if (valid >= kVec) {
        store16(p, r);
    } else if (valid > 0) {
        if constexpr (T == kF32) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid) p[e] = __uint_as_float(r[e]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid)
                    reinterpret_cast<unsigned short*>(p)[e] = (unsigned short)(r[e / 2] >> (16 * (e & 1)));
        }
    }
}

// `kVec` weights (or biases) starting at element `at` of a row of type `wdtype`, in fp32.
template <int kVec>
__device__ __forceinline__ void load_params(const void* base, int64_t at, int wdtype, int valid, float* f) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) f[e] = 0.f;
    if (wdtype == kF32) {
        const float* p = reinterpret_cast<const float*>(base) + at;
#pragma unroll
        for (int q = 0; q < kVec / 4; ++q) Elem<kF32>::unpack(load_raw<kF32>(p + 4 * q, valid - 4 * q), f + 4 * q);
    } else {
        // the two 16-bit types differ in the conversion alone; a 4-element vector (fp32 rows)
        // is the first half of an 8-element one
        const __bf16* p = reinterpret_cast<const __bf16*>(base) + at;
        const u32x4 r = load_raw<kBF16>(p, min(valid, kVec));
        float t[8];
        if (wdtype == kBF16) Elem<kBF16>::unpack(r, t);
        else Elem<kF16>::unpack(r, t);
#pragma unroll
        for (int e = 0; e < kVec; ++e) f[e] = t[e];
    }
}

__device__ __forceinline__ void store_param(void* base, int64_t at, int wdtype, float f) {
    if (wdtype == kF32) reinterpret_cast<float*>(base)[at] = f;
    else if (wdtype == kBF16) reinterpret_cast<unsigned short*>(base)[at] = f2bf(f);
    else reinterpret_cast<_Float16*>(base)[at] = (_Float16)f;
}

__device__ __forceinline__ int64_t row_offset(const NormArgs& a, const RowsPtr& p, unsigned r) {
    if (a.inner == 1) return (int64_t)r * p.s0;
    const unsigned t = __umulhi(r, a.inner_mul);
    const unsigned q = (unsigned)(((uint64_t)t + r) >> a.inner_shift);
    return (int64_t)q * p.s0 + (int64_t)(r - q * (unsigned)a.inner) * p.s1;
}

// kLanes: lanes of a row within a wave, or 0 where the whole block shares a row.
template <int kLanes>
struct RowTeam {
    static __device__ __forceinline__ int lane() { return kLanes ? threadIdx.x & (kLanes - 1) : threadIdx.x; }
    static __device__ __forceinline__ int team() { return kLanes ? threadIdx.x / (kLanes ? kLanes : 1) : 0; }
    static __device__ __forceinline__ int lanes() { return kLanes ? kLanes : blockDim.x; }
    static __device__ __forceinline__ int teams() { return kLanes ? blockDim.x / (kLanes ? kLanes : 1) : 1; }
};

constexpr int kMaxWaves = 16;

// Sum over the row's lanes. Whole-block rows go through `red` (one slot a wave): the
// caller alternates between two buffers, so that the one barrier of the next sum stands
// between a buffer's reads and its next writes.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* red) {
    if constexpr (kLanes) {
        return lanes_sum<kLanes>(v);
    } else {
        v = lanes_sum<64>(v);
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        const int nw = blockDim.x >> 6;
        float s = red[0];
        for (int i = 1; i < nw; ++i) s += red[i];
        return s;
    }
}

template <int T, bool kRms, int kLanes, int kN>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_norm_forward(NormArgs a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    typedef RowTeam<kLanes> Team;
    constexpr int kVec = E::kVec;
    __shared__ float red[2][kMaxWaves];
    const int group = blockIdx.x / a.chunks, chunk = blockIdx.x - group * a.chunks;
    const unsigned row0 = (unsigned)group * a.rows_per_group;
    const int begin = chunk * a.chunk_rows;
    const int end = min(begin + a.chunk_rows, a.rows_per_group);
    int col[kN], valid[kN];
    float w[kN][kVec], b[kN][kVec];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        col[k] = (k * Team::lanes() + Team::lane()) * kVec;
        valid[k] = a.cols - col[k];
        if (a.w) {
            load_params<kVec>(a.w, (int64_t)group * a.w_stride + col[k], a.wdtype, valid[k], w[k]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[k][e] += a.offset;
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[k][e] = 1.f;
        }
        if (a.b) {
            load_params<kVec>(a.b, (int64_t)group * a.b_stride + col[k], a.wdtype, valid[k], b[k]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) b[k][e] = 0.f;
        }
    }
    const int step = Team::teams();
    // every lane of a wave takes part in every sum: a team past the end repeats the last
    // row and writes nothing
    u32x4 next[kN];
    {
        const unsigned r = row0 + min(begin + Team::team(), end - 1);
        const elem* p = reinterpret_cast<const elem*>(a.x.data) + row_offset(a, a.x, r);
#pragma unroll
        for (int k = 0; k < kN; ++k) next[k] = load_raw<T>(p + col[k], valid[k]);
    }
    for (int at = begin; at < end; at += step) {
        const unsigned r = row0 + min(at + Team::team(), end - 1);
        const bool mine = at + Team::team() < end;
        float x[kN][kVec];
#pragma unroll
        for (int k = 0; k < kN; ++k) E::unpack(next[k], x[k]);
        if (at + step < end) {
            const unsigned rn = row0 + min(at + step + Team::team(), end - 1);
            const elem* p = reinterpret_cast<const elem*>(a.x.data) + row_offset(a, a.x, rn);
#pragma unroll
            for (int k = 0; k < kN; ++k) next[k] = load_raw<T>(p + col[k], valid[k]);
        }
        float mean = 0.f;
        if constexpr (!kRms) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kN; ++k)
#pragma unroll
                for (int e = 0; e < kVec; ++e) s += x[k][e];
            mean = row_sum<kLanes>(s, red[0]) * a.inv_cols;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                if (valid[k] >= kVec) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) x[k][e] -= mean;
                } else {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) x[k][e] = e < valid[k] ? x[k][e] - mean : 0.f;
                }
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < kN; ++k)
#pragma unroll
            for (int e = 0; e < kVec; ++e) sq = fmaf(x[k][e], x[k][e], sq);
        // the rms form has one sum a row, and alternates over the rows
        const int buf = kRms ? ((at - begin) & 1) : 1;
        const float rstd = 1.f / sqrtf(fmaf(row_sum<kLanes>(sq, red[buf]), a.inv_cols, a.eps));
        if (mine) {
            if (Team::lane() == 0) {
                if (!kRms && a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
            elem* q = reinterpret_cast<elem*>(a.y.data) + row_offset(a, a.y, r);
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                float y[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = fmaf(x[k][e] * rstd, w[k][e], b[k][e]);
                store_raw<T>(q + col[k], E::pack(y), valid[k]);
            }
        }
    }
}

template <int T, bool kRms, int kLanes, int kN>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_norm_backward(NormArgs a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    typedef RowTeam<kLanes> Team;
    constexpr int kVec = E::kVec;
    __shared__ float red[2][2][kMaxWaves];
    const int group = blockIdx.x / a.chunks, chunk = blockIdx.x - group * a.chunks;
    const unsigned row0 = (unsigned)group * a.rows_per_group;
    const int begin = chunk * a.chunk_rows;
    const int end = min(begin + a.chunk_rows, a.rows_per_group);
    int col[kN], valid[kN];
    float w[kN][kVec], dw[kN][kVec], db[kN][kVec];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        col[k] = (k * Team::lanes() + Team::lane()) * kVec;
        valid[k] = a.cols - col[k];
        if (a.w) {
            load_params<kVec>(a.w, (int64_t)group * a.w_stride + col[k], a.wdtype, valid[k], w[k]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[k][e] += a.offset;
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[k][e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) dw[k][e] = db[k][e] = 0.f;
    }
    const int step = Team::teams();
    u32x4 xn[kN], gn[kN];
    float mean_n = 0.f, rstd_n = 0.f;
    auto fetch = [&](int at) {
        const unsigned r = row0 + min(at + Team::team(), end - 1);
        const bool mine = at + Team::team() < end;
        const elem* px = reinterpret_cast<const elem*>(a.x.data) + row_offset(a, a.x, r);
        const elem* pg = reinterpret_cast<const elem*>(a.dy.data) + row_offset(a, a.dy, r);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            xn[k] = load_raw<T>(px + col[k], valid[k]);
            // a team past the end adds nothing to the sums over rows
            gn[k] = load_raw<T>(pg + col[k], mine ? valid[k] : 0);
        }
        if constexpr (!kRms) mean_n = a.mean[r];
        rstd_n = a.rstd[r];
    };
    if (begin < end) fetch(begin);
    for (int at = begin; at < end; at += step) {
        const unsigned r = row0 + min(at + Team::team(), end - 1);
        const bool mine = at + Team::team() < end;
        float h[kN][kVec], g[kN][kVec];
        const float mean = mean_n, rstd = rstd_n;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            E::unpack(xn[k], h[k]);
            E::unpack(gn[k], g[k]);
        }
        if (at + step < end) fetch(at + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < kN; ++k)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float hv = kRms ? h[k][e] * rstd : (h[k][e] - mean) * rstd;
                dw[k][e] = fmaf(g[k][e], hv, dw[k][e]);
                db[k][e] += g[k][e];
                const float av = g[k][e] * w[k][e];
                s1 += av;
                s2 = fmaf(av, hv, s2);
                h[k][e] = hv;
                g[k][e] = av;
            }
        if constexpr (kLanes != 0) {
            if constexpr (!kRms) s1 = lanes_sum<kLanes>(s1);
            s2 = lanes_sum<kLanes>(s2);
        } else {
            // both sums behind one barrier; the buffers alternate over the rows
            if constexpr (!kRms) s1 = lanes_sum<64>(s1);
            s2 = lanes_sum<64>(s2);
            float (*buf)[kMaxWaves] = red[(at - begin) & 1];
            if ((threadIdx.x & 63) == 0) {
                buf[0][threadIdx.x >> 6] = s1;
                buf[1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            const int nw = blockDim.x >> 6;
            s1 = buf[0][0];
            s2 = buf[1][0];
            for (int i = 1; i < nw; ++i) {
                s1 += buf[0][i];
                s2 += buf[1][i];
            }
        }
        if (mine) {
            const float c1 = kRms ? 0.f : s1 * a.inv_cols, c2 = s2 * a.inv_cols;
            elem* q = reinterpret_cast<elem*>(a.y.data) + row_offset(a, a.y, r);
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                float d[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) d[e] = rstd * fmaf(-h[k][e], c2, g[k][e] - c1);
                store_raw<T>(q + col[k], E::pack(d), valid[k]);
            }
        }
    }
    if (!a.dw && !a.db) return;
    // the block's sums over its rows: first over its teams (through LDS, in team order)
    if constexpr (kLanes != 0) {
        constexpr int kTeams = 256 / kLanes, kWidth = kLanes * kVec * kN;
        __shared__ float sums[kTeams][kWidth];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kN; ++k)
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    sums[Team::team()][col[k] + e] = which ? db[k][e] : dw[k][e];
            __syncthreads();
            void* out = which ? a.db : a.dw;
            const int64_t stride = which ? a.db_stride : a.dw_stride;
            if (out) {
                for (int c = threadIdx.x; c < a.cols; c += 256) {
                    float s = sums[0][c];
                    for (int t = 1; t < kTeams; ++t) s += sums[t][c];
                    if (a.chunks == 1) store_param(out, (int64_t)group * stride + c, a.wdtype, s);
                    else a.partial[((int64_t)which * a.groups * a.chunks + blockIdx.x) * a.cols + c] = s;
                }
            }
        }
    } else {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            void* out = which ? a.db : a.dw;
            const int64_t stride = which ? a.db_stride : a.dw_stride;
            if (!out) continue;
            float* part = a.partial + ((int64_t)which * a.groups * a.chunks + blockIdx.x) * a.cols;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const float* v = which ? db[k] : dw[k];
                if (a.chunks == 1) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (e < valid[k]) store_param(out, (int64_t)group * stride + col[k] + e, a.wdtype, v[e]);
                } else {
#pragma unroll
                    for (int q = 0; q < kVec / 4; ++q)
                        store_raw<kF32>(part + col[k] + 4 * q, Elem<kF32>::pack(v + 4 * q), valid[k] - 4 * q);
                }
            }
        }
    }
}

// Adds the blocks' partial sums of one group, 64 columns a block: each of 16 waves takes
// every sixteenth partial row, and the waves' sums are added in order.
constexpr int kWgradCols = 64, kWgradWaves = 16;
__global__ __launch_bounds__(kWgradCols * kWgradWaves) void k_norm_wgrad(NormArgs a) {
    __shared__ float sums[kWgradWaves][kWgradCols];
    const int which = blockIdx.z, group = blockIdx.y;
    void* out = which ? a.db : a.dw;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * kWgradCols + lane;
    float s = 0.f;
    if (c < a.cols) {
        const float* p = a.partial + ((int64_t)which * a.groups * a.chunks + (int64_t)group * a.chunks) * a.cols + c;
        for (int i = wave; i < a.chunks; i += kWgradWaves) s += p[(int64_t)i * a.cols];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < a.cols) {
        for (int t = 1; t < kWgradWaves; ++t) s += sums[t][lane];
        store_param(out, (int64_t)group * (which ? a.db_stride : a.dw_stride) + c, a.wdtype, s);
    }
}

template <bool kFwd, int T, bool kRms, int kLanes, int kN>
hipError_t launch(const NormPlan& p, const NormArgs& a, hipStream_t s) {
    const dim3 grid(unsigned(a.groups) * unsigned(p.chunks)), block(p.threads);
    if constexpr (kFwd) hipLaunchKernelGGL((k_norm_forward<T, kRms, kLanes, kN>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_norm_backward<T, kRms, kLanes, kN>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool kFwd, int T, bool kRms>
hipError_t launch_shape(const NormPlan& p, const NormArgs& a, hipStream_t s) {
    if (p.lanes == 8) return launch<kFwd, T, kRms, 8, 1>(p, a, s);
    if (p.lanes == 16) return launch<kFwd, T, kRms, 16, 1>(p, a, s);
    if (p.lanes == 32) return launch<kFwd, T, kRms, 32, 1>(p, a, s);
    if (p.lanes == 64) return launch<kFwd, T, kRms, 64, 1>(p, a, s);
    if (p.vecs == 1) return launch<kFwd, T, kRms, 0, 1>(p, a, s);
    if (p.vecs == 2) return launch<kFwd, T, kRms, 0, 2>(p, a, s);
    if constexpr (T == kF32) {
        if (p.vecs == 4) return launch<kFwd, T, kRms, 0, 4>(p, a, s);
    }
    return hipErrorInvalidValue;
}

template <bool kFwd>
hipError_t launch_type(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s) {
    if (dtype == kF32) return rms ? launch_shape<kFwd, kF32, true>(p, a, s) : launch_shape<kFwd, kF32, false>(p, a, s);
    if (dtype == kBF16)
        return rms ? launch_shape<kFwd, kBF16, true>(p, a, s) : launch_shape<kFwd, kBF16, false>(p, a, s);
    return rms ? launch_shape<kFwd, kF16, true>(p, a, s) : launch_shape<kFwd, kF16, false>(p, a, s);
}

NormPlan plan_shape(int dtype, int64_t cols) {
    const int vec = dtype == kF32 ? 4 : 8;
    const int64_t vectors = (cols + vec - 1) / vec;
    NormPlan p{};
    if (vectors <= 64) {
        p.lanes = vectors <= 8 ? 8 : vectors <= 16 ? 16 : vectors <= 32 ? 32 : 64;
        p.vecs = 1;
        p.threads = 256;
        p.rows_at_once = 256 / p.lanes;
    } else {
        p.vecs = vectors <= 256 ? 1 : vectors <= 2048 ? 2 : 4;
        p.threads = int(((vectors + p.vecs - 1) / p.vecs + 63) / 64 * 64);
        p.lanes = p.threads > 64 ? p.threads : 128;
        p.threads = p.lanes;
        p.rows_at_once = 1;
    }
    return p;
}

void plan_chunks(NormPlan& p, int64_t rows_per_group, int64_t groups, int64_t blocks, int64_t least_rows) {
    const int64_t want = std::max<int64_t>(1, blocks / std::max<int64_t>(groups, 1));
    const int64_t most = std::max<int64_t>(1, (rows_per_group + least_rows - 1) / least_rows);
    int64_t chunks = std::min(want, most);
    int64_t rows = std::max<int64_t>(1, (rows_per_group + chunks - 1) / chunks);
    rows = (rows + p.rows_at_once - 1) / p.rows_at_once * p.rows_at_once;
    p.chunk_rows = int(rows);
    p.chunks = int(std::max<int64_t>(1, (rows_per_group + rows - 1) / rows));
}

}  // namespace

#ifndef MUON_NORM_FWD_BLOCKS
#define MUON_NORM_FWD_BLOCKS 2048
#endif
#ifndef MUON_NORM_BWD_BLOCKS
#define MUON_NORM_BWD_BLOCKS 1024
#endif

NormPlan plan_norm_forward(int dtype, int64_t cols, int64_t rows_per_group, int64_t groups) {
    NormPlan p = plan_shape(dtype, cols);
    plan_chunks(p, rows_per_group, groups, MUON_NORM_FWD_BLOCKS, p.rows_at_once);
    return p;
}

NormPlan plan_norm_backward(int dtype, int64_t cols, int64_t rows_per_group, int64_t groups) {
    NormPlan p = plan_shape(dtype, cols);
    plan_chunks(p, rows_per_group, groups, MUON_NORM_BWD_BLOCKS, 4 * p.rows_at_once);
    return p;
}

hipError_t launch_norm_forward(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s) {
    return launch_type<true>(rms, dtype, p, a, s);
}

hipError_t launch_norm_backward(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s) {
    return launch_type<false>(rms, dtype, p, a, s);
}

hipError_t launch_norm_wgrad(const NormArgs& a, hipStream_t s) {
    const dim3 grid((a.cols + kWgradCols - 1) / kWgradCols, a.groups, 2);
    hipLaunchKernelGGL(k_norm_wgrad, grid, dim3(kWgradCols * kWgradWaves), 0, s, a);
    return hipGetLastError();
}

}  // namespace muon

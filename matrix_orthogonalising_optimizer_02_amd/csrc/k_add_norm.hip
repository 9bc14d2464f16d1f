// The residual's addition with the RMS norm that follows it, and their gradient. For a row:
//   h = x + r, rounded to the residual's type;  rstd = 1 / sqrt((1/H) sum h^2 + eps)
//   y = h rstd (offset + w), in x's type and / or in 8 bits with a power of two for every 128
//   elements (blocks8.hpp), both from the same fp32 values
// and from dy and the gradient dh that comes down the residual stream, with n = h rstd and
// a = dy (offset + w):
//   d = dh + rstd (a - n (1/H) sum a n), the gradient of x and of r;   dw = sum over rows of dy n
//
// HBM-bound: forward reads x and r and writes h and y once, backward reads dy, dh and h and
// writes d. A row stays in registers between its sum and its output, spread over lanes as the
// norms of k_norm.hip spread it (rows.hpp), and the next rows are asked for before the present
// one is reduced. A block of 128 elements is 16 lanes of 16-bit elements (32 of fp32), so its
// largest magnitude is a few lane exchanges and its codes leave as one contiguous piece.
#include "blocks8.hpp"
#include "rows.hpp"

#include <algorithm>

namespace muon {
namespace {

// A lane's kVec elements of type TY in 16-byte pieces.
template <int TY, int kVec>
struct Piece {
    typedef Elem<TY> E;
    typedef typename E::type elem;
    static constexpr int kParts = kVec / E::kVec;
    u32x4 raw[kParts];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int q = 0; q < kParts; ++q) raw[q] = u32x4{0u, 0u, 0u, 0u};
    }
    // rows shorter than a lane's vector are read and written element by element
    template <bool kStream>
    __device__ __forceinline__ void load(const elem* p, int col, int cols) {
        if (cols >= kVec) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) raw[q] = kStream ? stream16(p + col + q * E::kVec) : load16(p + col + q * E::kVec);
        } else {
            float f[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = col + e < cols ? (float)p[col + e] : 0.f;
            pack(f);
        }
    }
    __device__ __forceinline__ void store(elem* p, int col, int cols) const {
        if (cols >= kVec) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) put_stream16(p + col + q * E::kVec, raw[q]);
        } else {
            float f[kVec];
            unpack(f);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (col + e < cols) p[col + e] = (elem)f[e];
        }
    }
    __device__ __forceinline__ void pack(const float* f) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) raw[q] = E::pack(f + q * E::kVec);
    }
    __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
        for (int q = 0; q < kParts; ++q) E::unpack(raw[q], f + q * E::kVec);
    }
};

// As Span, for rows of any length: a row shorter than a vector is lane 0's, from its start, with
// zeros behind it.
template <int kVec>
struct Part {
    int col, skip;
    __device__ __forceinline__ Part(int cols, int index) {
        const int c = index * kVec;
        col = max(0, min(c, cols - kVec));
        skip = cols < kVec ? (index ? kVec : 0) : min(c - col, kVec);
    }
};

template <int kVec>
__device__ __forceinline__ void load_weights(const AddNormArgs& a, int col, float* w) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] = 1.f;
    if (!a.w) return;
    if (a.cols >= kVec) {
        load_params<kVec>(a.w, col, a.wdtype, w);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            if (col + e >= a.cols) w[e] = 0.f;
            else if (a.wdtype == kF32) w[e] = reinterpret_cast<const float*>(a.w)[col + e];
            else if (a.wdtype == kBF16) w[e] = bf2f(reinterpret_cast<const unsigned short*>(a.w)[col + e]);
            else w[e] = (float)reinterpret_cast<const _Float16*>(a.w)[col + e];
        }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] += a.offset;
}

// A lane's vector (elements from `skip` on count) of a row's 8-bit form. kGroup lanes share a
// block of 128.
template <int kVec, int kGroup>
__device__ __forceinline__ void put_codes(const AddNormArgs& a, int64_t row, int index, int skip, const float* y, bool mine) {
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) most = fmaxf(most, e >= skip ? fabsf(y[e]) : 0.f);  // passes over NaN
    unsigned top = lanes_max<kGroup>(__float_as_uint(most));
    if (__any(top >= 0x7F800000u)) {  // an infinity: once more over what is finite
        top = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) top = max(top, e >= skip ? finite_bits(y[e]) : 0u);
        top = lanes_max<kGroup>(top);
    }
    const unsigned byte = block_power(top);
    const int at = index * kVec, blocks = (a.cols + kBlock8 - 1) / kBlock8;
    if (!mine || at >= blocks * kBlock8) return;
    const float s = power_inverse(byte);
    uint8_t* codes = a.q.codes + row * a.q.ld + at;
    // the elements that count move to the front, zeros follow: the row's padding
    const int shift = skip * 8;
    if constexpr (kVec == 8) {
        const uint64_t c = pack_codes(y[0] * s, y[1] * s, y[2] * s, y[3] * s) |
                           (uint64_t)pack_codes(y[4] * s, y[5] * s, y[6] * s, y[7] * s) << 32;
        *reinterpret_cast<uint64_t*>(codes) = skip < kVec ? c >> shift : 0;
    } else {
        const unsigned c = pack_codes(y[0] * s, y[1] * s, y[2] * s, y[3] * s);
        *reinterpret_cast<unsigned*>(codes) = skip < kVec ? c >> shift : 0u;
    }
    if (at % kBlock8 == 0) {
        uint8_t* scales = a.q.scales + row * a.q.scale_ld;
        const int b = at / kBlock8;
        scales[b] = (uint8_t)byte;
        if (b == blocks - 1)
            for (int i = blocks; i & 3; ++i) scales[i] = 0;
    }
}

template <int T, bool kRes32, int kLanes, int kN>
__global__ __launch_bounds__(kLanes ? kSubThreads : 1024) void k_add_norm_forward(AddNormArgs a) {
    constexpr int kVec = Elem<T>::kVec, R = kRes32 ? kF32 : T;
    constexpr int kBlockLanes = kBlock8 / kVec, kGroup = kLanes && kLanes < kBlockLanes ? kLanes : kBlockLanes;
    typedef typename Elem<T>::type elem;
    typedef typename Elem<R>::type relem;
    __shared__ float red[2][kMaxWaves][1];
    const Team<kLanes> t(a.team_waves, a.teams);
    Piece<T, kVec> nx[kN];
    Piece<R, kVec> nr[kN];
    // A team past the last row has zeros and takes part in the sums.
    auto fetch = [&](int at) {
        const int64_t row = at + t.team;
        const bool mine = row < a.rows;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            nx[k].clear();
            nr[k].clear();
            const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
            if (mine) {
                nx[k].template load<false>(reinterpret_cast<const elem*>(a.x) + row * a.x_stride, sp.col, a.cols);
                if (a.r) nr[k].template load<false>(reinterpret_cast<const relem*>(a.r) + row * a.r_stride, sp.col, a.cols);
            }
        }
    };
    const int step = a.chunks * t.teams;
    int at = blockIdx.x * t.teams;
    if (at < a.rows) fetch(at);
    float w[kN][kVec];
#pragma unroll
    for (int k = 0; k < kN; ++k) load_weights<kVec>(a, Part<kVec>(a.cols, k * t.lanes + t.lane).col, w[k]);
    int flip = 0;
    for (; at < a.rows; at += step) {
        const int64_t row = at + t.team;
        const bool mine = row < a.rows;
        float f[kN][kVec];
        Piece<R, kVec> h[kN];
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            nx[k].unpack(f[k]);
            if (a.r) {
                float r[kVec];
                nr[k].unpack(r);
#pragma unroll
                for (int e = 0; e < kVec; ++e) f[k][e] += r[e];
                h[k].pack(f[k]);
                h[k].unpack(f[k]);  // the norm is that of h as it is stored
            }
        }
        if (at + step < a.rows) fetch(at + step);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float c = k < kN - 1 || e >= sp.skip ? f[k][e] : 0.f;
                sq = fmaf(c, c, sq);
            }
        }
        float sum[1] = {sq};
        row_sums<kLanes, 1>(sum, red[flip], t, a.team_waves);
        flip ^= 1;
        // rstd as the sum of two floats (one Newton step in fp64 from the fp32 root)
        const double var = (double)sum[0] * a.inv_cols + a.eps;
        double rd = 1.f / sqrtf((float)var);
        if (rd > 0.0) rd *= 1.5 - 0.5 * var * rd * rd;  // 0 where the sum is infinite
        const float rstd = (float)rd, rest = (float)(rd - rstd);
        if (mine && t.lane == 0 && a.rstd) a.rstd[row] = rstd;
        // All of the row was read before the sum above: h may lie where r or x lay.
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const int index = k * t.lanes + t.lane;
            const Part<kVec> sp(a.cols, index);
            const bool any = k < kN - 1 || sp.skip < kVec;
            if (a.r && mine && any) h[k].store(reinterpret_cast<relem*>(a.h) + row * a.h_stride, sp.col, a.cols);
            float y[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                // rstd w with what its rounding lost: y is then off by little more than its own
                // half step, and fewer codes fall to the other side of a border
                const float p = rstd * w[k][e];
                const float lost = fmaf(rstd, w[k][e], -p) + rest * w[k][e];
                y[e] = fmaf(f[k][e], p, f[k][e] * lost);
            }
            if (a.y && mine && any) {
                Piece<T, kVec> o;
                o.pack(y);
                o.store(reinterpret_cast<elem*>(a.y) + row * a.y_stride, sp.col, a.cols);
            }
            if (a.q.codes) {
                if constexpr (kLanes == 8) {
                    if (a.cols < kVec)  // behind the end of a row that is shorter than a vector: 0 times a NaN rstd
#pragma unroll
                        for (int e = 0; e < kVec; ++e) y[e] = e < a.cols ? y[e] : 0.f;
                }
                put_codes<kVec, kGroup>(a, row, index, sp.skip, y, mine);
            }
        }
        if (a.q.codes && mine)  // rows shorter than their team's lanes: the rest of the last block
            for (int c = (kN * t.lanes + t.lane) * kVec; c < (a.cols + kBlock8 - 1) / kBlock8 * kBlock8; c += t.lanes * kVec)
#pragma unroll
                for (int e = 0; e < kVec; e += 4) *reinterpret_cast<unsigned*>(a.q.codes + row * a.q.ld + c + e) = 0u;
    }
}

template <int T, bool kRes32, int kLanes, int kN, bool kStream>
__global__ __launch_bounds__(kLanes ? kSubThreads : 1024) void k_add_norm_backward(AddNormArgs a) {
    constexpr int kVec = Elem<T>::kVec, R = kRes32 ? kF32 : T;
    typedef typename Elem<T>::type elem;
    typedef typename Elem<R>::type relem;
    __shared__ float red[2][kMaxWaves][1];
    const Team<kLanes> t(a.team_waves, a.teams);
    constexpr int kAhead = kN * kVec <= 8 ? 2 : 0;  // rows asked for in advance; 16 elements a lane leave no registers
    struct Row {
        Piece<T, kVec> g[kN];
        Piece<R, kVec> h[kN], dh[kN];
        float rstd;
    };
    Row ahead[kAhead ? kAhead : 1];
    auto fetch = [&](Row& o, int at) {
        const int64_t row = at + t.team;
        const bool mine = row < a.rows;
        o.rstd = 0.f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            o.g[k].clear();
            o.h[k].clear();
            o.dh[k].clear();
        }
        if (mine) {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
                o.g[k].template load<kStream>(reinterpret_cast<const elem*>(a.x) + row * a.x_stride, sp.col, a.cols);
                o.h[k].template load<kStream>(reinterpret_cast<const relem*>(a.h) + row * a.h_stride, sp.col, a.cols);
                if (a.r) o.dh[k].template load<kStream>(reinterpret_cast<const relem*>(a.r) + row * a.r_stride, sp.col, a.cols);
            }
            o.rstd = a.rstd[row];
        }
    };
    const int step = a.chunks * t.teams;
    int at = blockIdx.x * t.teams;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (at + i * step < a.rows) fetch(ahead[i], at + i * step);
    float w[kN][kVec], dw[kN][kVec];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        load_weights<kVec>(a, Part<kVec>(a.cols, k * t.lanes + t.lane).col, w[k]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) dw[k][e] = 0.f;
    }
    int flip = 0;
    auto process = [&](Row& o) {
        const int64_t row = at + t.team;
        const bool mine = row < a.rows;
        if constexpr (kAhead == 0) fetch(o, at);
        const float rstd = o.rstd;
        float n[kN][kVec], g[kN][kVec];
        Piece<R, kVec> dh[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            o.h[k].unpack(n[k]);
            o.g[k].unpack(g[k]);
            dh[k] = o.dh[k];
        }
        if (kAhead && at + kAhead * step < a.rows) fetch(o, at + kAhead * step);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                n[k][e] *= rstd;
                // elements that do not count are added too: their lane does not write them
                dw[k][e] = fmaf(g[k][e], n[k][e], dw[k][e]);
                g[k][e] *= w[k][e];
                const float c = k < kN - 1 || e >= sp.skip ? g[k][e] : 0.f;
                s = fmaf(c, n[k][e], s);
            }
        }
        float sum[1] = {s};
        // In place over dh the last vector's lane reads what the lane before it writes, which may be
        // another wave's. dh is in no sum, and the barrier inside row_sums waits for LDS alone: so dh
        // is brought to its registers here ([8192, 5120] fp32 141 to 131 us with that, 16-bit rows the
        // same: it was asked for with the rest of the row).
        if constexpr (kLanes == 0) {
#pragma unroll
            for (int k = 0; k < kN; ++k)
#pragma unroll
                for (int q = 0; q < Piece<R, kVec>::kParts; ++q) asm volatile("" ::"v"(dh[k].raw[q]));
        }
        row_sums<kLanes, 1>(sum, red[flip], t, a.team_waves);
        flip ^= 1;
        if (!mine) return;
        const float c2 = sum[0] * (float)a.inv_cols * rstd;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
            if (k == kN - 1 && sp.skip >= kVec) continue;
            float d[kVec], base[kVec];
            dh[k].unpack(base);
#pragma unroll
            for (int e = 0; e < kVec; ++e) d[e] = base[e] + fmaf(g[k][e], rstd, -n[k][e] * c2);
            Piece<R, kVec> od;
            od.pack(d);
            od.store(reinterpret_cast<relem*>(a.d) + row * a.d_stride, sp.col, a.cols);
            if (a.y) {
                Piece<T, kVec> oy;
                oy.pack(d);
                oy.store(reinterpret_cast<elem*>(a.y) + row * a.y_stride, sp.col, a.cols);
            }
        }
    };
    while (at < a.rows) {
#pragma unroll
        for (int i = 0; i < (kAhead ? kAhead : 1); ++i) {
            if (at >= a.rows) break;
            process(ahead[i]);
            at += step;
        }
    }
    if (!a.dw) return;
    // the block's sums over its rows: over its teams through LDS, in team order, then to the
    // gradient or to the block's partial sums
    extern __shared__ float part[];
    float* partial = a.partial + (int64_t)blockIdx.x * a.cols;
    auto put = [&](int c, float v) {
        if (a.chunks == 1) store_param(a.dw, c, a.wdtype, v);
        else partial[c] = v;
    };
    if (t.teams == 1) {  // every column is one thread's
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e >= sp.skip && sp.col + e < a.cols) put(sp.col + e, dw[k][e]);
        }
    } else if constexpr (kLanes != 0) {
        constexpr int kWidth = kLanes * kVec;
        const Part<kVec> sp(a.cols, t.lane);
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e >= sp.skip) part[t.team * kWidth + sp.col + e] = dw[0][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float v = part[c];
            for (int i = 1; i < t.teams; ++i) v += part[i * kWidth + c];
            put(c, v);
        }
    } else {
        for (int i = 0; i < t.teams; ++i) {
            __syncthreads();
            if (t.team != i) continue;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Part<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e >= sp.skip) part[sp.col + e] = i ? part[sp.col + e] + dw[k][e] : dw[k][e];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) put(c, part[c]);
    }
}

template <bool kFwd, int T, bool kRes32, int kLanes, int kN>
hipError_t launch(const NormPlan& p, const AddNormArgs& a, hipStream_t s) {
    const dim3 grid(unsigned(p.chunks)), block(p.threads);
    if constexpr (kFwd) {
        hipLaunchKernelGGL((k_add_norm_forward<T, kRes32, kLanes, kN>), grid, block, 0, s, a);
    } else {
        const size_t lds = a.dw && p.teams > 1 ? size_t(4) * (kLanes ? p.threads * Elem<T>::kVec : a.cols) : 0;
        if (p.stream) hipLaunchKernelGGL((k_add_norm_backward<T, kRes32, kLanes, kN, true>), grid, block, lds, s, a);
        else hipLaunchKernelGGL((k_add_norm_backward<T, kRes32, kLanes, kN, false>), grid, block, lds, s, a);
    }
    return hipGetLastError();
}

template <bool kFwd, int T, bool kRes32>
hipError_t launch_shape(const NormPlan& p, const AddNormArgs& a, hipStream_t s) {
    if (p.lanes == 8) return launch<kFwd, T, kRes32, 8, 1>(p, a, s);
    if (p.lanes == 16) return launch<kFwd, T, kRes32, 16, 1>(p, a, s);
    if (p.lanes == 32) return launch<kFwd, T, kRes32, 32, 1>(p, a, s);
    if (p.lanes == 64) return launch<kFwd, T, kRes32, 64, 1>(p, a, s);
    if (p.vecs == 1) return launch<kFwd, T, kRes32, 0, 1>(p, a, s);
    if (p.vecs == 2) return launch<kFwd, T, kRes32, 0, 2>(p, a, s);
    if constexpr (T == kF32) {
        if (p.vecs == 4) return launch<kFwd, T, kRes32, 0, 4>(p, a, s);
    }
    return hipErrorInvalidValue;
}

template <bool kFwd>
hipError_t launch_type(int dtype, bool res32, const NormPlan& p, const AddNormArgs& a, hipStream_t s) {
    if (dtype == kF32) return launch_shape<kFwd, kF32, true>(p, a, s);
    if (dtype == kBF16) return res32 ? launch_shape<kFwd, kBF16, true>(p, a, s) : launch_shape<kFwd, kBF16, false>(p, a, s);
    return res32 ? launch_shape<kFwd, kF16, true>(p, a, s) : launch_shape<kFwd, kF16, false>(p, a, s);
}

}  // namespace

NormPlan plan_add_norm(bool forward, int dtype, int64_t cols, int64_t rows) {
    // rows shorter than a vector are spread as those of one vector
    const int64_t least = dtype == kF32 ? 4 : 8;
    if (forward) return plan_norm_forward(dtype, std::max(cols, least), rows, 1);
    NormPlan p = plan_norm_backward(dtype, std::max(cols, least), rows, 1);
    // Backward asks for more waves of fp32 rows on a compute unit than the norms' rule, which cuts
    // its 10 to whole blocks: one block of 7 or 8 waves takes [21897, 1629] in 151 us and [8000, 2000]
    // in 64, two take 107 and 53. Over 40 million elements two blocks take 0.62 (16 columns) to 0.79
    // (4096) of one's time at every width up to 4096, floor 102 us: 64 columns 155 and 108 us, 200 190
    // and 123, 512 156 and 111, 1024 142 and 109, 4096 139 and 110. Wider rows' blocks and inputs of 4
    // million elements are cut alike by both. 20 waves take 108 us at 200 and 384 columns, but 123 at
    // 1024 and 140 at 1629. 16-bit rows, of twice the elements a lane, lose: [20000, 2048] bf16 57 us,
    // with 14 waves 61 (with an fp32 residual 123 and 127).
    if (dtype == kF32) {
        constexpr int64_t kUnits = 256, kWaves = 14;
        const int64_t blocks = kUnits * std::max<int64_t>(1, (kWaves * 64 + p.threads / 2) / p.threads);
        p.chunks = int(std::max<int64_t>(p.chunks, std::min<int64_t>(blocks, rows / (4 * p.teams))));
        p.chunk_rows = int((rows + p.chunks - 1) / p.chunks);
    }
    return p;
}

hipError_t launch_add_norm_forward(int dtype, bool res32, const NormPlan& p, const AddNormArgs& a, hipStream_t s) {
    return launch_type<true>(dtype, res32, p, a, s);
}

hipError_t launch_add_norm_backward(int dtype, bool res32, const NormPlan& p, const AddNormArgs& a, hipStream_t s) {
    return launch_type<false>(dtype, res32, p, a, s);
}

}  // namespace muon

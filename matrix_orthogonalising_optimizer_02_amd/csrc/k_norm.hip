// Normalisation layers and their gradients. For a row x of H columns in group g:
//   mean = (1/H) sum x (0 for the rms form), rstd = 1 / sqrt((1/H) sum (x - mean)^2 + eps)
//   h = (x - mean) rstd,   y = h (offset + w[g]) + b[g]
// and from dy, with a = dy (offset + w[g]):
//   dx = rstd (a - (1/H) sum a - h (1/H) sum a h)     (rms: without the first sum)
//   dw[g] = sum over the group's rows of dy h,   db[g] = sum of dy
//
// Both passes are HBM-bound: forward reads x and writes y, backward reads x and dy and
// writes dx, and a row stays in registers between its statistics and its output, so every
// element moves once. A row is shared by 8 to 64 lanes of a wave or by 2 to 16 whole waves
// (a "team"), 16 bytes a lane and load, with the group's weights and the sums for their
// gradients in registers. The blocks of a group take its rows in turn, so that all blocks
// together read one stretch of memory at a time ([8192, 4096] fp32 backward 76 us; 84 us
// where each block has a stretch of its own), and ask for the next rows before they reduce
// the present one. Statistics are two-pass over the registers (the mean first, then the
// squares of the differences), all sums in fp32 in a fixed order. Outputs are stored with
// the non-temporal hint ([32768, 1024] bf16 forward 25 us; 31 us without), inputs are read
// without it (a preceding kernel may have left them in the cache).
// Measured: [8192, 5120] bf16 in 8 groups, forward 28 to 29 us (5.9 TB/s), backward 53 us
// (4.7 TB/s with the weights' gradients, 5.6 TB/s without); [65536, 5120] backward 374 us
// (5.4 TB/s); a copy reaches 6.25 TB/s. The vector units are busy 43% of the forward pass
// and 48% of the backward pass.
#include "rows.hpp"

#include <algorithm>

namespace muon {
namespace {

__device__ __forceinline__ int64_t row_offset(const NormArgs& a, const RowsPtr& p, unsigned r) {
    if (a.inner == 1) return (int64_t)r * p.s0;
    const unsigned t = __umulhi(r, a.inner_mul);
    const unsigned q = (unsigned)(((uint64_t)t + r) >> a.inner_shift);
    return (int64_t)q * p.s0 + (int64_t)(r - q * (unsigned)a.inner) * p.s1;
}

// The rows of a block: every group's rows in turn, t.teams at a time. The groups start at
// different places, so that blocks of different groups do not walk through memory in step:
// groups of 1024 rows of 10 KiB are a multiple of 1 MiB apart, and meet in the same channels
// ([65536, 5120] bf16 in 64 groups, backward 380 us; 392 us from the same row on).
struct Turn {
    int begin, step, count, phase;
    __device__ __forceinline__ Turn(const NormArgs& a, int group, int chunk, int teams) {
        begin = chunk * teams;
        step = a.chunks * teams;
        count = begin < a.rows_per_group ? (a.rows_per_group - begin + step - 1) / step : 0;
        phase = (int)((int64_t)group * count / a.groups);
    }
    __device__ __forceinline__ int row(int i) const {
        const int j = i + phase;
        return begin + (j < count ? j : j - count) * step;
    }
};

template <int T, bool kRms, int kLanes, int kN, bool kExact>
__global__ __launch_bounds__(kLanes ? kSubThreads : 1024) void k_norm_forward(NormArgs a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    constexpr int kVec = E::kVec;
    __shared__ float red[2][kMaxWaves][1];
    const Team<kLanes> t(a.team_waves, a.teams);
    const int group = blockIdx.x / a.chunks, chunk = blockIdx.x - group * a.chunks;
    const unsigned row0 = (unsigned)group * a.rows_per_group;
    const Turn turn(a, group, chunk, t.teams);
    const int end = a.rows_per_group;
    // Every lane of a wave takes part in every sum: a team past the end has zeros and writes
    // nothing. It reads nothing either, as other rows may be written over by then (y is x).
    u32x4 next[kN];
    auto fetch = [&](int at) {
        const bool mine = at + t.team < end;
        const elem* p = reinterpret_cast<const elem*>(a.x.data) + row_offset(a, a.x, row0 + (mine ? at + t.team : at));
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            next[k] = u32x4{0u, 0u, 0u, 0u};
            if (mine) next[k] = load16(p + Span<kVec>(a.cols, k * t.lanes + t.lane).col);
        }
    };
    if (turn.count) fetch(turn.row(0));
    float w[kN][kVec], b[kN][kVec];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            w[k][e] = 1.f;
            b[k][e] = 0.f;
        }
        if (a.w) {
            load_params<kVec>(a.w, (int64_t)group * a.w_stride + sp.col, a.wdtype, w[k]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[k][e] += a.offset;
        }
        if (a.b) load_params<kVec>(a.b, (int64_t)group * a.b_stride + sp.col, a.wdtype, b[k]);
    }
    int flip = 0;
    for (int i = 0; i < turn.count; ++i) {
        const int at = turn.row(i);
        const bool mine = at + t.team < end;
        const unsigned r = row0 + at + t.team;
        float x[kN][kVec];
#pragma unroll
        for (int k = 0; k < kN; ++k) E::unpack(next[k], x[k]);
        if (i + 1 < turn.count) fetch(turn.row(i + 1));
        float mean = 0.f;
        if constexpr (!kRms) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
                for (int e = 0; e < kVec; ++e) s += k < kN - 1 ? x[k][e] : counted<kExact>(sp, e, x[k][e]);
            }
            float sum[1] = {s};
            row_sums<kLanes, 1>(sum, red[0], t, a.team_waves);
            mean = sum[0] * a.inv_cols;
        }
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                if constexpr (!kRms) x[k][e] -= mean;
                const float d = k < kN - 1 ? x[k][e] : counted<kExact>(sp, e, x[k][e]);
                sq = fmaf(d, d, sq);
            }
        }
        // the rms form has one sum a row, and alternates over the rows
        float sum[1] = {sq};
        row_sums<kLanes, 1>(sum, red[kRms ? flip : 1], t, a.team_waves);
        flip ^= 1;
        const float rstd = 1.f / sqrtf(fmaf(sum[0], a.inv_cols, a.eps));
        if (mine) {
            if (t.lane == 0) {
                if (!kRms && a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
            elem* q = reinterpret_cast<elem*>(a.y.data) + row_offset(a, a.y, r);
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
                float y[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = fmaf(x[k][e] * rstd, w[k][e], b[k][e]);
                if (kExact || k < kN - 1 || sp.skip < kVec) put_stream16(q + sp.col, E::pack(y));
            }
        }
    }
}

// kStream: x and dy are read with the non-temporal hint.
template <int T, bool kRms, int kLanes, int kN, bool kExact, bool kStream>
__global__ __launch_bounds__(kLanes ? kSubThreads : 1024) void k_norm_backward(NormArgs a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    constexpr int kVec = E::kVec;
    __shared__ float red[2][kMaxWaves][2];
    const Team<kLanes> t(a.team_waves, a.teams);
    const int group = blockIdx.x / a.chunks, chunk = blockIdx.x - group * a.chunks;
    const unsigned row0 = (unsigned)group * a.rows_per_group;
    const Turn turn(a, group, chunk, t.teams);
    const int end = a.rows_per_group;
    // Rows asked for in advance: two where a lane holds 8 elements. 16 elements leave no
    // registers for that ([1024, 16384] fp32: 53 us without, 76 us with one row and spills).
    constexpr int kAhead = kN * kVec <= 8 ? 2 : 0;
    struct Row {
        u32x4 x[kN], g[kN];
        float mean, rstd;
    };
    Row ahead[kAhead ? kAhead : 1];
    // as in the forward pass, a team past the end has zeros
    auto fetch = [&](Row& row, int at) {
        const bool mine = at + t.team < end;
        const unsigned r = row0 + (mine ? at + t.team : at);
        const elem* px = reinterpret_cast<const elem*>(a.x.data) + row_offset(a, a.x, r);
        const elem* pg = reinterpret_cast<const elem*>(a.dy.data) + row_offset(a, a.dy, r);
#pragma unroll
        for (int k = 0; k < kN; ++k) row.x[k] = row.g[k] = u32x4{0u, 0u, 0u, 0u};
        row.mean = row.rstd = 0.f;
        if (mine) {
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
                row.x[k] = kStream ? stream16(px + sp.col) : load16(px + sp.col);
                row.g[k] = kStream ? stream16(pg + sp.col) : load16(pg + sp.col);
            }
            if constexpr (!kRms) row.mean = a.mean[r];
            row.rstd = a.rstd[r];
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < turn.count) fetch(ahead[i], turn.row(i));
    float w[kN][kVec], dw[kN][kVec], db[kN][kVec];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            w[k][e] = 1.f;
            dw[k][e] = db[k][e] = 0.f;
        }
        if (a.w) {
            load_params<kVec>(a.w, (int64_t)group * a.w_stride + sp.col, a.wdtype, w[k]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[k][e] += a.offset;
        }
    }
    int flip = 0;
    auto process = [&](Row& row, int i) {
        const int at = turn.row(i);
        const bool mine = at + t.team < end;  // a team past the end adds and writes nothing
        if constexpr (kAhead == 0) fetch(row, at);
        const float mean = row.mean, rstd = row.rstd;
        float h[kN][kVec], g[kN][kVec];
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            E::unpack(row.x[k], h[k]);
            E::unpack(row.g[k], g[k]);
        }
        if (kAhead && i + kAhead < turn.count) fetch(row, turn.row(i + kAhead));
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float hv = kRms ? h[k][e] * rstd : (h[k][e] - mean) * rstd;
                // the weights' sums take an element that does not count too: its lane
                // does not write them
                dw[k][e] = fmaf(g[k][e], hv, dw[k][e]);
                db[k][e] += g[k][e];
                const float av = g[k][e] * w[k][e];
                const float ac = k < kN - 1 ? av : counted<kExact>(sp, e, av);
                sums[0] += ac;
                sums[1] = fmaf(ac, hv, sums[1]);
                h[k][e] = hv;
                g[k][e] = av;
            }
        }
        row_sums<kLanes, 2>(sums, red[flip], t, a.team_waves);
        flip ^= 1;
        if (mine) {
            // rstd (a - c1 - h c2) as two fused steps
            const float c1 = kRms ? 0.f : sums[0] * a.inv_cols * rstd, c2 = sums[1] * a.inv_cols * rstd;
            elem* q = reinterpret_cast<elem*>(a.y.data) + row_offset(a, a.y, row0 + at + t.team);
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
                float d[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) d[e] = fmaf(g[k][e], rstd, -fmaf(h[k][e], c2, c1));
                if (kExact || k < kN - 1 || sp.skip < kVec) put_stream16(q + sp.col, E::pack(d));
            }
        }
    };
    for (int i = 0; i < turn.count;) {
#pragma unroll
        for (int k = 0; k < (kAhead ? kAhead : 1); ++k) {
            process(ahead[k], i);
            if (++i >= turn.count) break;
        }
    }
    if (!a.dw && !a.db) return;
    // The block's sums over its rows: over its teams through LDS, in team order, then to
    // the gradients or to the block's partial sums.
    extern __shared__ float part[];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        void* out = which ? a.db : a.dw;
        if (!out) continue;
        const int64_t to = (int64_t)group * (which ? a.db_stride : a.dw_stride);
        float* partial = a.partial + ((int64_t)which * a.groups * a.chunks + blockIdx.x) * a.cols;
        if constexpr (kLanes != 0) {
            // [team][column], each team's row of LDS
            const Span<kVec> sp(a.cols, t.lane);
            constexpr int kWidth = kLanes * kVec;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e >= sp.skip) part[t.team * kWidth + sp.col + e] = which ? db[0][e] : dw[0][e];
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
                float s = part[c];
                for (int i = 1; i < t.teams; ++i) s += part[i * kWidth + c];
                if (a.chunks == 1) store_param(out, to + c, a.wdtype, s);
                else partial[c] = s;
            }
        } else if (t.teams == 1) {  // every column is one thread's
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
                const float* v = which ? db[k] : dw[k];
                if (a.chunks > 1 && sp.skip == 0) {
#pragma unroll
                    for (int q = 0; q < kVec / 4; ++q) store16(partial + sp.col + 4 * q, Elem<kF32>::pack(v + 4 * q));
                } else {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        if (e < sp.skip) continue;
                        if (a.chunks > 1) partial[sp.col + e] = v[e];
                        else store_param(out, to + sp.col + e, a.wdtype, v[e]);
                    }
                }
            }
        } else {
            for (int i = 0; i < t.teams; ++i) {
                __syncthreads();
                if (t.team != i) continue;
#pragma unroll
                for (int k = 0; k < kN; ++k) {
                    const Span<kVec> sp(a.cols, k * t.lanes + t.lane);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        if (e < sp.skip) continue;
                        const float v = which ? db[k][e] : dw[k][e];
                        part[sp.col + e] = i ? part[sp.col + e] + v : v;
                    }
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
                if (a.chunks == 1) store_param(out, to + c, a.wdtype, part[c]);
                else partial[c] = part[c];
            }
        }
    }
}

// Rows shorter than a vector: a thread a row.
constexpr int kTinyCols = 8;
template <int T>
__device__ __forceinline__ float load_elem(const void* base, int64_t i) {
    if constexpr (T == kF32) return reinterpret_cast<const float*>(base)[i];
    else if constexpr (T == kBF16) return bf2f(reinterpret_cast<const unsigned short*>(base)[i]);
    else return (float)reinterpret_cast<const _Float16*>(base)[i];
}

__device__ __forceinline__ float load_param(const void* base, int64_t i, int wdtype) {
    return wdtype == kF32 ? load_elem<kF32>(base, i) : wdtype == kBF16 ? load_elem<kBF16>(base, i) : load_elem<kF16>(base, i);
}

template <int T, bool kRms>
__global__ __launch_bounds__(256) void k_norm_forward_tiny(NormArgs a) {
    const int group = blockIdx.x / a.chunks, chunk = blockIdx.x - group * a.chunks;
    const int at = chunk * a.chunk_rows + threadIdx.x;
    if (threadIdx.x >= a.chunk_rows || at >= a.rows_per_group) return;
    const unsigned r = (unsigned)group * a.rows_per_group + at;
    const int64_t px = row_offset(a, a.x, r), py = row_offset(a, a.y, r);
    float x[kTinyCols], mean = 0.f, sq = 0.f;
#pragma unroll
    for (int e = 0; e < kTinyCols; ++e) {
        x[e] = e < a.cols ? load_elem<T>(a.x.data, px + e) : 0.f;
        mean += x[e];
    }
    mean = kRms ? 0.f : mean * a.inv_cols;
#pragma unroll
    for (int e = 0; e < kTinyCols; ++e) {
        x[e] = e < a.cols ? x[e] - mean : 0.f;
        sq = fmaf(x[e], x[e], sq);
    }
    const float rstd = 1.f / sqrtf(fmaf(sq, a.inv_cols, a.eps));
    if (!kRms && a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
#pragma unroll
    for (int e = 0; e < kTinyCols; ++e) {
        if (e >= a.cols) break;
        const float w = a.w ? a.offset + load_param(a.w, (int64_t)group * a.w_stride + e, a.wdtype) : 1.f;
        const float b = a.b ? load_param(a.b, (int64_t)group * a.b_stride + e, a.wdtype) : 0.f;
        store_param(a.y.data, py + e, T, fmaf(x[e] * rstd, w, b));
    }
}

template <int T, bool kRms>
__global__ __launch_bounds__(256) void k_norm_backward_tiny(NormArgs a) {
    __shared__ float red[4];
    const int group = blockIdx.x / a.chunks, chunk = blockIdx.x - group * a.chunks;
    const int begin = chunk * a.chunk_rows, end = min(begin + a.chunk_rows, a.rows_per_group);
    float w[kTinyCols], dw[kTinyCols], db[kTinyCols];
#pragma unroll
    for (int e = 0; e < kTinyCols; ++e) {
        w[e] = a.w && e < a.cols ? a.offset + load_param(a.w, (int64_t)group * a.w_stride + e, a.wdtype) : 1.f;
        dw[e] = db[e] = 0.f;
    }
    for (int at = begin + threadIdx.x; at < end; at += 256) {
        const unsigned r = (unsigned)group * a.rows_per_group + at;
        const int64_t px = row_offset(a, a.x, r), pg = row_offset(a, a.dy, r), pd = row_offset(a, a.y, r);
        const float mean = kRms ? 0.f : a.mean[r], rstd = a.rstd[r];
        float h[kTinyCols], g[kTinyCols], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int e = 0; e < kTinyCols; ++e) {
            const bool in = e < a.cols;
            h[e] = in ? (load_elem<T>(a.x.data, px + e) - mean) * rstd : 0.f;
            g[e] = in ? load_elem<T>(a.dy.data, pg + e) : 0.f;
            dw[e] = fmaf(g[e], h[e], dw[e]);
            db[e] += g[e];
            g[e] *= w[e];
            s1 += g[e];
            s2 = fmaf(g[e], h[e], s2);
        }
        const float c1 = kRms ? 0.f : s1 * a.inv_cols, c2 = s2 * a.inv_cols;
#pragma unroll
        for (int e = 0; e < kTinyCols; ++e)
            if (e < a.cols) store_param(a.y.data, pd + e, T, rstd * fmaf(-h[e], c2, g[e] - c1));
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        void* out = which ? a.db : a.dw;
        if (!out) continue;
#pragma unroll
        for (int e = 0; e < kTinyCols; ++e) {
            const float s = block_sum_256(which ? db[e] : dw[e], red);
            if (threadIdx.x != 0 || e >= a.cols) continue;
            if (a.chunks == 1) store_param(out, (int64_t)group * (which ? a.db_stride : a.dw_stride) + e, a.wdtype, s);
            else a.partial[((int64_t)which * a.groups * a.chunks + blockIdx.x) * a.cols + e] = s;
        }
    }
}

// Adds the blocks' partial sums of one group. The threads of a block are `slices` rows of
// columns: each takes every slices-th partial row, eight loads at a time, and the slices'
// sums are added in order.
constexpr int kWgradThreads = 512;
__global__ __launch_bounds__(kWgradThreads) void k_norm_wgrad(NormArgs a, int slices) {
    __shared__ float sums[kWgradThreads];
    const int which = a.dw ? blockIdx.z : 1, group = blockIdx.y;
    const int width = kWgradThreads / slices;  // both powers of two
    const int lane = threadIdx.x & (width - 1), slice = threadIdx.x / width;
    const int c = blockIdx.x * width + lane;
    constexpr int kUnroll = 8;
    float s[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) s[k] = 0.f;
    if (c < a.cols) {
        const float* p = a.partial + ((int64_t)which * a.groups * a.chunks + (int64_t)group * a.chunks) * a.cols + c;
        int i = slice;
        for (; i + (kUnroll - 1) * slices < a.chunks; i += kUnroll * slices)
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) s[k] += p[(int64_t)(i + k * slices) * a.cols];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (i + k * slices < a.chunks) s[k] += p[(int64_t)(i + k * slices) * a.cols];
    }
    float t = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    sums[threadIdx.x] = t;
    __syncthreads();
    if (slice == 0 && c < a.cols) {
        for (int k = 1; k < slices; ++k) t += sums[k * width + lane];
        store_param(which ? a.db : a.dw, (int64_t)group * (which ? a.db_stride : a.dw_stride) + c, a.wdtype, t);
    }
}

template <bool kFwd, int T, bool kRms, int kLanes, int kN, bool kExact>
hipError_t launch(const NormPlan& p, const NormArgs& a, hipStream_t s) {
    const dim3 grid(unsigned(a.groups) * unsigned(p.chunks)), block(p.threads);
    if constexpr (kFwd) {
        hipLaunchKernelGGL((k_norm_forward<T, kRms, kLanes, kN, kExact>), grid, block, 0, s, a);
    } else {
        // a team's sums for all columns, or the block's: at most 16 KiB and 8 KiB
        const bool shared = (a.dw || a.db) && p.teams > 1;
        const size_t lds = shared ? size_t(4) * (kLanes ? p.threads * Elem<T>::kVec : a.cols) : 0;
        if (p.stream) hipLaunchKernelGGL((k_norm_backward<T, kRms, kLanes, kN, kExact, true>), grid, block, lds, s, a);
        else hipLaunchKernelGGL((k_norm_backward<T, kRms, kLanes, kN, kExact, false>), grid, block, lds, s, a);
    }
    return hipGetLastError();
}

template <bool kFwd, int T, bool kRms, int kLanes>
hipError_t launch_lanes(const NormPlan& p, const NormArgs& a, hipStream_t s) {
    if (a.cols == kLanes * Elem<T>::kVec) return launch<kFwd, T, kRms, kLanes, 1, true>(p, a, s);
    return launch<kFwd, T, kRms, kLanes, 1, false>(p, a, s);
}

template <bool kFwd, int T, bool kRms>
hipError_t launch_shape(const NormPlan& p, const NormArgs& a, hipStream_t s) {
    if (p.lanes == 1) {
        const dim3 grid(unsigned(a.groups) * unsigned(p.chunks)), block(256);
        if constexpr (kFwd) hipLaunchKernelGGL((k_norm_forward_tiny<T, kRms>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_norm_backward_tiny<T, kRms>), grid, block, 0, s, a);
        return hipGetLastError();
    }
    if (p.lanes == 8) return launch_lanes<kFwd, T, kRms, 8>(p, a, s);
    if (p.lanes == 16) return launch_lanes<kFwd, T, kRms, 16>(p, a, s);
    if (p.lanes == 32) return launch_lanes<kFwd, T, kRms, 32>(p, a, s);
    if (p.lanes == 64) return launch_lanes<kFwd, T, kRms, 64>(p, a, s);
    if (p.vecs == 1) return launch<kFwd, T, kRms, 0, 1, false>(p, a, s);
    if (p.vecs == 2) return launch<kFwd, T, kRms, 0, 2, false>(p, a, s);
    if constexpr (T == kF32) {
        if (p.vecs == 4) return launch<kFwd, T, kRms, 0, 4, false>(p, a, s);
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

// Shapes, measured on MI355X. Forward: a lane holds one vector up to 256 vectors a row, two
// beyond, in blocks of 4 waves, 24 waves a compute unit in all ([8192, 5120] bf16 29.4 us;
// 42 us with one vector a lane and 10 waves a row, 31 us with 40 waves a unit). Backward: one
// vector of 16-bit elements up to 1024 vectors a row (so that a lane's eight columns leave
// registers for two rows in advance), two of fp32 from 129 vectors on, blocks of 8 waves or
// one row, and as many whole blocks a unit as 10 waves hold, one at least: 10 waves where a
// row takes 10, 8 for rows that share a block of 8, 6 for rows of 6 (fp32 of 1153 columns).
// Every block's partial sums are written and read once more, so that fewer blocks win
// ([8192, 5120] bf16 52.9 us; 58 us with 20 waves, 66 us with 30; other widths were not
// measured with more).
constexpr int kForwardVectors = 256, kForwardBlockWaves = 4, kForwardWaves = 24;
constexpr int kBackwardVectors = 1024, kBackwardVectors32 = 128, kBackwardBlockWaves = 8, kBackwardWaves = 10;
constexpr int kComputeUnits = 256;
// x and dy of this many bytes are read with the non-temporal hint in the backward pass: they
// leave the 256 MB memory-side cache before they could be of use ([8192, 4096] fp32, 268 MB,
// 71.6 us; 76.0 without the hint. [131072, 128] bf16, 67 MB, 23.1 us; 21.6 without).
constexpr int64_t kStreamBytes = int64_t(128) << 20;

// one_vec: rows of up to this many vectors are spread over enough waves that a lane holds one.
NormPlan plan_shape(int dtype, int64_t cols, int64_t one_vec, int block_waves) {
    const int vec = dtype == kF32 ? 4 : 8;
    const int64_t vectors = (cols + vec - 1) / vec;
    NormPlan p{};
    p.vecs = 1;
    p.teams = 1;
    p.threads = 256;
    if (cols < vec) {
        p.lanes = 1;
        p.teams = 256;
    } else if (vectors <= 64) {
        p.lanes = vectors <= 8 ? 8 : vectors <= 16 ? 16 : vectors <= 32 ? 32 : 64;
        p.threads = std::min(block_waves * 64, kSubThreads);
        p.teams = p.threads / p.lanes;
    } else {
        // only the last of a lane's vectors may lie past the row's end
        p.vecs = vectors <= one_vec ? 1 : vectors <= 2048 ? 2 : 4;
        p.lanes = std::max(128, int(((vectors + p.vecs - 1) / p.vecs + 63) / 64 * 64));
        p.teams = std::max(1, block_waves * 64 / p.lanes);
        p.threads = p.teams * p.lanes;
    }
    return p;
}

// Splits every group into blocks: so many that the card's compute units hold `waves` waves
// each, of at least `least` passes of a block.
void plan_chunks(NormPlan& p, int64_t rows_per_group, int64_t groups, int64_t waves, int64_t least) {
    const int64_t blocks = kComputeUnits * std::max<int64_t>(1, waves * 64 / p.threads);
    const int64_t want = std::max<int64_t>(1, (blocks + groups / 2) / std::max<int64_t>(groups, 1));
    const int64_t most = std::max<int64_t>(1, rows_per_group / (least * p.teams));
    p.chunks = int(std::min(want, most));
    p.chunk_rows = int((rows_per_group + p.chunks - 1) / p.chunks);
}

}  // namespace

NormPlan plan_norm_forward(int dtype, int64_t cols, int64_t rows_per_group, int64_t groups) {
    NormPlan p = plan_shape(dtype, cols, kForwardVectors, kForwardBlockWaves);
    if (p.lanes == 1) {  // one pass of a block
        p.chunk_rows = p.teams;
        p.chunks = int((rows_per_group + p.teams - 1) / p.teams);
        return p;
    }
    plan_chunks(p, rows_per_group, groups, kForwardWaves, 1);
    return p;
}

NormPlan plan_norm_backward(int dtype, int64_t cols, int64_t rows_per_group, int64_t groups) {
    NormPlan p = plan_shape(dtype, cols, dtype == kF32 ? kBackwardVectors32 : kBackwardVectors, kBackwardBlockWaves);
    plan_chunks(p, rows_per_group, groups, kBackwardWaves, 4);
    p.stream = 2 * rows_per_group * groups * cols * elem_size(dtype) >= kStreamBytes;
    return p;
}

hipError_t launch_norm_forward(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s) {
    return launch_type<true>(rms, dtype, p, a, s);
}

hipError_t launch_norm_backward(bool rms, int dtype, const NormPlan& p, const NormArgs& a, hipStream_t s) {
    return launch_type<false>(rms, dtype, p, a, s);
}

hipError_t launch_norm_wgrad(const NormArgs& a, hipStream_t s) {
    int slices = 1;
    while (slices < 16 && slices * 16 < a.chunks) slices *= 2;
    const int width = kWgradThreads / slices;
    const dim3 grid((a.cols + width - 1) / width, a.groups, a.dw && a.db ? 2 : 1);
    hipLaunchKernelGGL(k_norm_wgrad, grid, dim3(kWgradThreads), 0, s, a, slices);
    return hipGetLastError();
}

}  // namespace muon

// Rotary positions over several axes. Pair i of a head's elements (p, q) is turned by the angle
// 2 pi pos[axis(i)] freq(i) of its token:
//   p' = p cos - q sin,  q' = p sin + q cos
// and the gradient is the same turned back. The angle's fraction of a turn is worked out in
// fp64 (a position of 2^20 times a frequency leaves fp32 no digits of it) and the sine and
// cosine of that fraction in fp32: once for a token and pair, by a block that then turns all
// heads of its tokens from a table in LDS. So the operator is bound by reading and writing its
// rows once; strides take it to the query and key views of a fused projection, in place too.
#include "rows.hpp"

#include <algorithm>

namespace muon {
namespace {

constexpr int kRotThreads = 256;
constexpr int kHeads = 4;  // heads of a thread whose loads are in flight together

// kPairs pairs a lane: 32 bytes. Halves: pairs (i, i + pairs), two 16-byte vectors; adjacent:
// pairs (2 i, 2 i + 1), one stretch.
template <int T, bool kAdjacent>
__global__ __launch_bounds__(kRotThreads) void k_rotary(RotaryArgs a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    constexpr int kVec = E::kVec;  // elements of 16 bytes, and pairs of a lane
    extern __shared__ float2 table[];
    const uint32_t first = blockIdx.x * (uint32_t)a.block_rows;
    const int rows = (int)min((uint32_t)a.block_rows, a.rows - first);
    for (int i = threadIdx.x; i < rows * a.pairs; i += kRotThreads) {
        const int r = i / a.pairs, p = i - r * a.pairs;
        const uint32_t at = first + r, b = at / a.tokens, t = at - b * a.tokens;
        const int64_t from = (int64_t)b * a.pb + (int64_t)t * a.pt + min((unsigned)a.axis[p], (unsigned)a.axes - 1u);
        const double pos = a.pos_type == 0   ? (double)reinterpret_cast<const int32_t*>(a.pos)[from]
                           : a.pos_type == 1 ? (double)reinterpret_cast<const int64_t*>(a.pos)[from]
                                             : (double)reinterpret_cast<const float*>(a.pos)[from];
        const double turns = pos * a.freq[p];
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        table[i] = make_float2(c, s * a.sign);
    }
    __syncthreads();
    const int lanes = 1 << a.lane_bits, j0 = threadIdx.x & (lanes - 1), step = kRotThreads >> a.lane_bits;
    const int turned = (a.pairs + kVec - 1) / kVec, rest = a.dim - 2 * a.pairs;
    const bool copies = a.x.data != a.y.data;  // in place, what is not turned stays
    const int items = turned + (copies ? (rest + kVec - 1) / kVec : 0);
    struct Head {
        const elem* x;
        elem* y;
        const float2* cs;
    };
    auto head = [&](unsigned i) {
        unsigned r = i;
        if (a.heads > 1) r = (unsigned)(((uint64_t)__umulhi(i, a.heads_mul) + i) >> a.heads_shift);
        const unsigned h = i - r * a.heads;
        const uint32_t at = first + r, b = at / a.tokens, t = at - b * a.tokens;
        return Head{reinterpret_cast<const elem*>(a.x.data) + (int64_t)b * a.x.sb + (int64_t)t * a.x.st + (int64_t)h * a.x.sh,
                    reinterpret_cast<elem*>(a.y.data) + (int64_t)b * a.y.sb + (int64_t)t * a.y.st + (int64_t)h * a.y.sh,
                    table + r * a.pairs};
    };
    const unsigned end = (unsigned)rows * a.heads;
    for (int j = j0; j < items; j += lanes) {
        const int p0 = j * kVec, e0 = kAdjacent ? 2 * p0 : p0, e1 = kAdjacent ? e0 + kVec : a.pairs + p0;
        if (p0 + kVec <= a.pairs) {
            // kHeads heads at a time: their loads are in flight together
            for (unsigned i = threadIdx.x >> a.lane_bits; i < end; i += kHeads * step) {
                Head hd[kHeads];
                u32x4 raw[kHeads][2];
#pragma unroll
                for (int u = 0; u < kHeads; ++u)
                    if (i + u * step < end) {
                        hd[u] = head(i + u * step);
                        raw[u][0] = load16(hd[u].x + e0);
                        raw[u][1] = load16(hd[u].x + e1);
                    }
#pragma unroll
                for (int u = 0; u < kHeads; ++u) {
                    if (i + u * step >= end) break;
                    float f[2][kVec], o[2][kVec];
                    E::unpack(raw[u][0], f[0]);
                    E::unpack(raw[u][1], f[1]);
#pragma unroll
                    for (int k = 0; k < kVec; ++k) {
                        const float2 w = hd[u].cs[p0 + k];
                        if constexpr (kAdjacent) {
                            const int v = 2 * k / kVec, e = 2 * k % kVec;
                            o[v][e] = f[v][e] * w.x - f[v][e + 1] * w.y;
                            o[v][e + 1] = f[v][e] * w.y + f[v][e + 1] * w.x;
                        } else {
                            o[0][k] = f[0][k] * w.x - f[1][k] * w.y;
                            o[1][k] = f[0][k] * w.y + f[1][k] * w.x;
                        }
                    }
                    put_stream16(hd[u].y + e0, E::pack(o[0]));
                    put_stream16(hd[u].y + e1, E::pack(o[1]));
                }
            }
        } else {
            for (unsigned i = threadIdx.x >> a.lane_bits; i < end; i += step) {
                const Head hd = head(i);
                if (j < turned) {  // the pairs that are left over
                    for (int k = 0; p0 + k < a.pairs; ++k) {
                        const float2 w = hd.cs[p0 + k];
                        const int ep = kAdjacent ? e0 + 2 * k : e0 + k, eq = kAdjacent ? ep + 1 : e1 + k;
                        const float p = (float)hd.x[ep], q = (float)hd.x[eq];
                        hd.y[ep] = (elem)(p * w.x - q * w.y);
                        hd.y[eq] = (elem)(p * w.y + q * w.x);
                    }
                } else {
                    const int e = 2 * a.pairs + (j - turned) * kVec;
                    if (e + kVec <= a.dim) put_stream16(hd.y + e, load16(hd.x + e));
                    else
                        for (int k = e; k < a.dim; ++k) hd.y[k] = hd.x[k];
                }
            }
        }
    }
}

template <int T>
hipError_t launch_layout(bool adjacent, const RotaryArgs& a, hipStream_t s) {
    const dim3 grid((a.rows + a.block_rows - 1) / a.block_rows), block(kRotThreads);
    const size_t lds = size_t(a.block_rows) * a.pairs * sizeof(float2);
    if (adjacent) hipLaunchKernelGGL((k_rotary<T, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_rotary<T, false>), grid, block, lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(int dtype, bool adjacent, const RotaryArgs& args, hipStream_t s) {
    RotaryArgs a = args;
    // Tokens of a block: enough blocks for 8 a compute unit, a table of 32 KiB at most.
    const uint32_t room = std::max<uint32_t>(1, 4096u / (uint32_t)std::max(1, a.pairs));
    a.block_rows = (int)std::min(room, std::max<uint32_t>(1, a.rows / 2048));
    const int vec = dtype == kF32 ? 4 : 8;
    const int items = (a.pairs + vec - 1) / vec + (a.x.data != a.y.data ? (a.dim - 2 * a.pairs + vec - 1) / vec : 0);
    a.lane_bits = 0;
    while ((1 << a.lane_bits) < items && a.lane_bits < 8) ++a.lane_bits;
    if (dtype == kF32) return launch_layout<kF32>(adjacent, a, s);
    if (dtype == kBF16) return launch_layout<kBF16>(adjacent, a, s);
    return launch_layout<kF16>(adjacent, a, s);
}

}  // namespace muon

// Rotary positions over several axes. Pair i of a head's elements (p, q) is turned by the angle
// 2 pi pos[axis(i)] freq(i) of its token:
//   p' = p cos - q sin,  q' = p sin + q cos
// and the gradient is the same turned back. The angle's fraction of a turn is worked out in
// fp64 (a position of 2^20 times a frequency leaves fp32 no digits of it), the sine and cosine in
// fp32, of the fraction as fp32 holds it and then of the rest, so that small ones keep their digits
// ([8192, 80, 128] bf16 65 us with and without the rest, [60000, 1, 128] 14; all in fp64 65 and 18).
// That is done once for a token and pair, by a block that then turns all heads of its tokens from
// a table in LDS, the first of them read meanwhile. So the operator is bound by reading and writing
// its rows once ([8192, 80, 128] bf16 in 65 us, 5.2 TB/s) where a token has many heads; with few, by
// the table too ([60000, 8, 128] 51, 4.8 TB/s; [60000, 1, 128] 14, 2.1). Strides take it to the query
// and key views of a fused projection, in place too.
#include "rows.hpp"

#include <algorithm>

namespace muon {
namespace {

constexpr int kRotThreads = 256;

// Items of `count` elements, a vector or two each.
__host__ __device__ constexpr int rotary_items(int count, int vec, bool two) {
    const int vectors = (count + vec - 1) / vec;
    return two ? (vectors + 1) / 2 : vectors;
}

// heads of a thread whose loads are in flight together ([8192, 80, 128] bf16 with 2: 68 us, 4: 66,
// 6: 65; [60000, 8, 128] 55, 53, 58)
constexpr int kHeads = 4;

// The same bits wherever a pair lies: which product is rounded is not left to the compiler.
__device__ __forceinline__ void turn_pair(float p, float q, float2 w, float& po, float& qo) {
    po = fmaf(p, w.x, -(q * w.y));
    qo = fmaf(p, w.y, q * w.x);
}

// A lane's item is two 16-byte vectors of a head, next to its neighbours' in each of the two loads:
// of kVec pairs (i, i + pairs), or of adjacent pairs or of elements that are copied only, the j-th
// vector and the j-th of the second half of them. The last vector of each kind ends where its kind
// ends, over a part of the one before where the count does not fit: both then write the same
// values. That needs a whole vector of that kind and, in place, all lanes of a head in one wave,
// whose loads are done before its stores; else the elements left over go one by one.
// kStream: the result passes L2 by.
template <int T, bool kAdjacent, bool kStream>
__global__ __launch_bounds__(kRotThreads) void k_rotary(RotaryArgs a) {
    typedef Elem<T> E;
    typedef typename E::type elem;
    constexpr int kVec = E::kVec;  // elements of 16 bytes, and pairs of a lane
    extern __shared__ float2 table[];
    const uint32_t first = blockIdx.x * (uint32_t)a.block_rows;
    const int rows = (int)min((uint32_t)a.block_rows, a.rows - first);
    auto batch_of = [&](uint32_t at) { return a.tokens == a.rows ? 0u : at / a.tokens; };
    const int lanes = 1 << a.lane_bits, j0 = threadIdx.x & (lanes - 1), step = kRotThreads >> a.lane_bits;
    const int span = kAdjacent ? 2 * a.pairs : a.pairs, rest = a.dim - 2 * a.pairs;  // elements of a vector's kind
    const bool copies = a.x.data != a.y.data;                                         // in place, what is not turned stays
    const bool over = span >= kVec && (copies || lanes <= 64);
    const int turned = rotary_items(span, kVec, kAdjacent), items = turned + (copies ? rotary_items(rest, kVec, true) : 0);
    struct Head {
        const elem* x;
        elem* y;
        const float2* cs;
    };
    auto head = [&](unsigned i) {
        unsigned r = i;
        if (a.heads > 1) r = (unsigned)(((uint64_t)__umulhi(i, a.heads_mul) + i) >> a.heads_shift);
        const unsigned h = i - r * a.heads;
        const uint32_t at = first + r, b = batch_of(at), t = at - b * a.tokens;
        return Head{reinterpret_cast<const elem*>(a.x.data) + (int64_t)b * a.x.sb + (int64_t)t * a.x.st + (int64_t)h * a.x.sh,
                    reinterpret_cast<elem*>(a.y.data) + (int64_t)b * a.y.sb + (int64_t)t * a.y.st + (int64_t)h * a.y.sh,
                    table + r * a.pairs};
    };
    struct Item {
        int e0, e1;
        bool turn, whole;
    };
    auto item = [&](int j) {
        Item it;
        it.turn = j < turned;
        if (it.turn) {
            it.e0 = j * kVec;
            it.e1 = kAdjacent ? it.e0 + turned * kVec : 0;
            it.whole = over || std::max(it.e0, it.e1) + kVec <= span;
            if (it.whole) {
                it.e0 = min(it.e0, span - kVec);
                it.e1 = min(it.e1, span - kVec);
            }
            if (!kAdjacent) it.e1 = it.e0 + span;
        } else {
            it.e0 = (j - turned) * kVec;
            it.e1 = it.e0 + (items - turned) * kVec;
            it.whole = rest >= kVec;
            if (it.whole) {
                it.e0 = min(it.e0, rest - kVec);
                it.e1 = min(it.e1, rest - kVec);
            }
            it.e0 += 2 * a.pairs;
            it.e1 += 2 * a.pairs;
        }
        return it;
    };
    // kHeads heads at a time: their loads are in flight together
    struct Batch {
        Head hd[kHeads];
        u32x4 raw[kHeads][2];
    };
    const unsigned end = (unsigned)rows * a.heads, i0 = threadIdx.x >> a.lane_bits;
    auto load = [&](Batch& t, const Item& it, unsigned i) {
#pragma unroll
        for (int u = 0; u < kHeads; ++u)
            if (i + u * step < end) {
                t.hd[u] = head(i + u * step);
                t.raw[u][0] = load16(t.hd[u].x + it.e0);
                t.raw[u][1] = load16(t.hd[u].x + it.e1);
            }
    };
    auto put = [&](Batch& t, const Item& it, unsigned i) {
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            if (i + u * step >= end) break;
            if (it.turn) {
                float f[2][kVec], o[2][kVec];
                E::unpack(t.raw[u][0], f[0]);
                E::unpack(t.raw[u][1], f[1]);
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    if constexpr (kAdjacent) {
                        const int v = 2 * k / kVec, e = 2 * k % kVec;
                        const float2 w = t.hd[u].cs[((v ? it.e1 : it.e0) + e) >> 1];
                        turn_pair(f[v][e], f[v][e + 1], w, o[v][e], o[v][e + 1]);
                    } else {
                        const float2 w = t.hd[u].cs[it.e0 + k];
                        turn_pair(f[0][k], f[1][k], w, o[0][k], o[1][k]);
                    }
                }
                t.raw[u][0] = E::pack(o[0]);
                t.raw[u][1] = E::pack(o[1]);
            }
            if constexpr (kStream) {
                put_stream16(t.hd[u].y + it.e0, t.raw[u][0]);
                put_stream16(t.hd[u].y + it.e1, t.raw[u][1]);
            } else {
                store16(t.hd[u].y + it.e0, t.raw[u][0]);
                store16(t.hd[u].y + it.e1, t.raw[u][1]);
            }
        }
    };
    // the first heads are on their way while the table is worked out
    const bool any = j0 < items;
    Item it = item(any ? j0 : 0);
    Batch t;
    const bool early = any && it.whole;
    if (early) load(t, it, i0);
    for (int i = threadIdx.x; i < rows * a.pairs; i += kRotThreads) {
        const int r = i / a.pairs, p = i - r * a.pairs;
        const uint32_t at = first + r, b = batch_of(at), tok = at - b * a.tokens;
        const int64_t from = (int64_t)b * a.pb + (int64_t)tok * a.pt + min((unsigned)a.axis[p], (unsigned)a.axes - 1u);
        const double pos = a.pos_type == 0   ? (double)reinterpret_cast<const int32_t*>(a.pos)[from]
                           : a.pos_type == 1 ? (double)reinterpret_cast<const int64_t*>(a.pos)[from]
                                             : (double)reinterpret_cast<const float*>(a.pos)[from];
        const double turns = pos * a.freq[p];
        float s, c;
        const double half = 2.0 * (turns - rint(turns));
        const float near = (float)half;
        sincospif(near, &s, &c);
        // what the rounding to fp32 left of the angle, by the sine's and cosine's slopes
        const float left = (float)(3.141592653589793 * (half - near)), slope = c;
        c = fmaf(-s, left, c);
        s = fmaf(slope, left, s);
        table[i] = make_float2(c, s * a.sign);
    }
    __syncthreads();
    if (!any) return;
    if (early) {
        put(t, it, i0);
        for (unsigned i = i0 + kHeads * step; i < end; i += kHeads * step) {
            load(t, it, i);
            put(t, it, i);
        }
    }
    for (int j = early ? j0 + lanes : j0; j < items; j += lanes) {
        it = item(j);
        if (it.whole) {
            for (unsigned i = i0; i < end; i += kHeads * step) {
                load(t, it, i);
                put(t, it, i);
            }
            continue;
        }
        for (unsigned i = i0; i < end; i += step) {
            const Head hd = head(i);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int e = v ? it.e1 : it.e0;
                if (!it.turn) {
                    for (int k = e; k < min(e + kVec, a.dim); ++k) hd.y[k] = hd.x[k];
                } else if (kAdjacent || v == 0) {
                    for (int k = e; k < min(e + kVec, span); k += kAdjacent ? 2 : 1) {
                        const float2 w = hd.cs[kAdjacent ? k >> 1 : k];
                        const int other = kAdjacent ? k + 1 : k + span;
                        float p, q;
                        turn_pair((float)hd.x[k], (float)hd.x[other], w, p, q);
                        hd.y[k] = (elem)p;
                        hd.y[other] = (elem)q;
                    }
                }
            }
        }
    }
}

template <int T, bool kAdjacent>
hipError_t launch_layout(bool stream, const RotaryArgs& a, hipStream_t s) {
    const dim3 grid((a.rows + a.block_rows - 1) / a.block_rows), block(kRotThreads);
    const size_t lds = size_t(a.block_rows) * a.pairs * sizeof(float2);
    if (stream) hipLaunchKernelGGL((k_rotary<T, kAdjacent, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_rotary<T, kAdjacent, false>), grid, block, lds, s, a);
    return hipGetLastError();
}

template <int T>
hipError_t launch_type(bool adjacent, bool stream, const RotaryArgs& a, hipStream_t s) {
    return adjacent ? launch_layout<T, true>(stream, a, s) : launch_layout<T, false>(stream, a, s);
}

}  // namespace

hipError_t launch_rotary(int dtype, bool adjacent, const RotaryArgs& args, hipStream_t s) {
    RotaryArgs a = args;
    // Tokens of a block: enough blocks for 8 a compute unit, a table of 32 KiB at most.
    const uint32_t room = std::max<uint32_t>(1, 4096u / (uint32_t)std::max(1, a.pairs));
    a.block_rows = (int)std::min(room, std::max<uint32_t>(1, a.rows / 2048));
    const int vec = dtype == kF32 ? 4 : 8;
    const int items = rotary_items(adjacent ? 2 * a.pairs : a.pairs, vec, adjacent) +
                      (a.x.data != a.y.data ? rotary_items(a.dim - 2 * a.pairs, vec, true) : 0);
    a.lane_bits = 0;
    while ((1 << a.lane_bits) < items && a.lane_bits < 8) ++a.lane_bits;
    // Streaming stores where every head's parts fill whole pieces of 64 bytes ([8192, 80, 128] bf16
    // 66 us, with ordinary stores 70); elsewhere the pieces meet in L2 first ([4999, 24, 90] fp32
    // 17.5 us, with streaming stores 20.7).
    const int64_t size = dtype == kF32 ? 4 : 2;
    const int64_t cuts = (a.x.data == a.y.data ? 0 : int64_t(a.dim)) | a.y.sb | a.y.st | a.y.sh | (adjacent ? 2 * a.pairs : a.pairs);
    const bool stream = ((reinterpret_cast<uintptr_t>(a.y.data) | uintptr_t(cuts * size)) & 63) == 0;
    if (dtype == kF32) return launch_type<kF32>(adjacent, stream, a, s);
    if (dtype == kBF16) return launch_type<kBF16>(adjacent, stream, a, s);
    return launch_type<kF16>(adjacent, stream, a, s);
}

}  // namespace muon

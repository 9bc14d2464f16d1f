// AdamW over many tensors in one launch, with fp32 states or with 8-bit ones:
//   m <- b1 m + (1 - b1) s g,   v <- b2 v + (1 - b2) (s g)^2
//   W <- (1 - lr wd) W - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// and a 16-bit copy of W where the caller wants one.
//
// HBM-bound. Bytes an element, e = 4 or 2 those of a gradient: 32-bit states 24 + e, 8-bit
// states 12 + e + 1/16, 2 more with the copy. A block takes 4096 consecutive elements of
// one tensor, looked up in the table by its block index (two dependent scalar loads, hidden
// by the other blocks of the compute unit). Each wave takes four runs of 256 elements, four
// elements a lane: with 8-bit states a run is one block of a shared scale, so its largest
// magnitudes are two wave reductions in registers. All loads of a wave are issued before
// its first store.
#include "lanes.hpp"
#include "train.hpp"

namespace muon {
namespace {

typedef float float2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf162_t __attribute__((ext_vector_type(2)));

__global__ void k_multi_table(MultiDescArgs a) {
    // a descriptor as 32-bit words, copied by the block's threads
    constexpr int kWords = sizeof(MultiDesc) / 4;
    const unsigned* src = reinterpret_cast<const unsigned*>(&a.d[blockIdx.x]);
    unsigned* dst = reinterpret_cast<unsigned*>(a.table + a.first + blockIdx.x);
    for (int i = threadIdx.x; i < kWords; i += blockDim.x) dst[i] = src[i];
}

// The tensor of each block: the last whose first block is not behind it. Empty tensors
// have their successor's first block, and are passed over.
template <class Desc>
__global__ void k_map(const Desc* table, int count, int32_t* map, int blocks) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= blocks) return;
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (table[mid].blk_begin <= b) lo = mid;
        else hi = mid - 1;
    }
    map[b] = lo;
}

struct Hyper {
    float b1, b2, ob1, ob2, eps, step, inv_sqrt_bc2, decay, gs;
};

// sqrt(v): r = 1/sqrt(v) from the hardware (1 ulp), s = v r, and one Newton step on s
// whose residual is exact; with the factor below twelve operations where sqrtf has about
// sixteen. The same bits as sqrtf on all values below 2^-93 and 3e8 up to 2^127. Nearer to
// 2^-126 the unscaled residual would lose digits, and the hardware's root takes no number
// below it: a v below 2^-96 is multiplied by 2^64 first and its root by 2^-32 after, both
// exact (8-bit states, 177 M elements: 521.7 us; 520 us without).
__device__ __forceinline__ float root(float v) {
    const bool small = v < 0x1p-96f;
    const float x = v * (small ? 0x1p64f : 1.f);
    const float r = __builtin_amdgcn_rsqf(fmaxf(x, 0x1p-126f));  // finite for 0
    const float s = x * r;
    const float u = fmaf(fmaf(-s, s, x), 0.5f * r, s) * (small ? 0x1p-32f : 1.f);
    return v == __builtin_inff() ? v : u;
}

// New m, v and u = sqrt(v), and the new weight. The moments' products are rounded before
// they are added (no fused multiply-add): any fp32 program that follows the formula gets
// the same bits, and so, with 8-bit states, the same stochastic roundings. The division is
// the hardware's reciprocal (1 ulp of the update; eps keeps its argument a normal number).
__device__ __forceinline__ float adam(const Hyper& h, float w, float g, float& m, float& v, float& u) {
    {
#pragma clang fp contract(off)
        g = g * h.gs;
        m = h.b1 * m + h.ob1 * g;
        v = h.b2 * v + h.ob2 * (g * g);
    }
    u = root(v);
    return fmaf(-h.step, m * __builtin_amdgcn_rcpf(fmaf(u, h.inv_sqrt_bc2, h.eps)), w * h.decay);
}

// kType: the gradient's type where it is known at compile time, else -1.
template <int kType>
__device__ __forceinline__ floatx4 load_grad(const void* g, int run_type, int64_t i, int valid) {
    const int type = kType < 0 ? run_type : kType;
    floatx4 r = {0.f, 0.f, 0.f, 0.f};
    if (type == kF32) {
        const float* p = reinterpret_cast<const float*>(g) + i;
        if (valid >= 4) r = ld_stream(p);
        else
            for (int e = 0; e < 4; ++e)
                if (e < valid) r[e] = p[e];
    } else {
        const unsigned short* p = reinterpret_cast<const unsigned short*>(g) + i;
        unsigned lo = 0, hi = 0;
        if (valid >= 4) {
            const u32x2 t = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
            lo = t[0];
            hi = t[1];
        } else {
            if (valid > 0) lo = p[0];
            if (valid > 1) lo |= (unsigned)p[1] << 16;
            if (valid > 2) hi = p[2];
        }
        if (type == kBF16) {
            r[0] = __uint_as_float(lo << 16);
            r[1] = __uint_as_float(lo & 0xFFFF0000u);
            r[2] = __uint_as_float(hi << 16);
            r[3] = __uint_as_float(hi & 0xFFFF0000u);
        } else {
            const half2_t a = __builtin_bit_cast(half2_t, lo), b = __builtin_bit_cast(half2_t, hi);
            r[0] = (float)a[0];
            r[1] = (float)a[1];
            r[2] = (float)b[0];
            r[3] = (float)b[1];
        }
    }
    return r;
}

__device__ __forceinline__ floatx4 load4(const float* p, int valid) {
    floatx4 r = {0.f, 0.f, 0.f, 0.f};
    if (valid >= 4) r = ld_stream(p);
    else
        for (int e = 0; e < 4; ++e)
            if (e < valid) r[e] = p[e];
    return r;
}

__device__ __forceinline__ void store4(float* p, floatx4 v, int valid) {
    if (valid >= 4) st_stream(p, v);
    else
        for (int e = 0; e < 4; ++e)
            if (e < valid) p[e] = v[e];
}

__device__ __forceinline__ unsigned load_codes(const void* base, int64_t i, int valid) {
    const unsigned char* p = reinterpret_cast<const unsigned char*>(base) + i;
    if (valid >= 4) return __builtin_nontemporal_load(reinterpret_cast<const unsigned*>(p));
    unsigned r = 0;
    for (int e = 0; e < 4; ++e)
        if (e < valid) r |= (unsigned)p[e] << (8 * e);
    return r;
}

__device__ __forceinline__ void store_codes(void* base, int64_t i, unsigned v, int valid) {
    unsigned char* p = reinterpret_cast<unsigned char*>(base) + i;
    if (valid >= 4) __builtin_nontemporal_store(v, reinterpret_cast<unsigned*>(p));
    else
        for (int e = 0; e < 4; ++e)
            if (e < valid) p[e] = (unsigned char)(v >> (8 * e));
}

__device__ __forceinline__ void store_copy(void* base, int type, int64_t i, floatx4 w, int valid) {
    const float2_t a = {w[0], w[1]}, b = {w[2], w[3]};
    u32x2 r;
    if (type == kBF16) {
        r[0] = __builtin_bit_cast(unsigned, __builtin_convertvector(a, bf162_t));
        r[1] = __builtin_bit_cast(unsigned, __builtin_convertvector(b, bf162_t));
    } else {
        r[0] = __builtin_bit_cast(unsigned, __builtin_convertvector(a, half2_t));
        r[1] = __builtin_bit_cast(unsigned, __builtin_convertvector(b, half2_t));
    }
    unsigned short* p = reinterpret_cast<unsigned short*>(base) + i;
    if (valid >= 4) __builtin_nontemporal_store(r, reinterpret_cast<u32x2*>(p));
    else
        for (int e = 0; e < 4; ++e)
            if (e < valid) p[e] = (unsigned short)(r[e / 2] >> (16 * (e & 1)));
}

// Four e4m3 codes to fp32 (exact).
__device__ __forceinline__ floatx4 decode(unsigned c) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    return floatx4{a[0], a[1], b[0], b[1]};
}

constexpr float kE4m3Max = 448.f;
constexpr float kLeastMax = 1e-30f;

// Scale and multiplier of a block whose largest magnitude is amax (NaN or infinite where one
// element is).
__device__ __forceinline__ void block_scale(float amax, float& scale, float& mul) {
    // 1 / amax: the hardware's reciprocal (1 ulp) and one Newton step, the nearest number but
    // for rare last bits
    const float r0 = __builtin_amdgcn_rcpf(amax);
    const float r = fmaf(fmaf(-amax, r0, 1.f), r0, r0);
    const bool finite = amax <= 3.402823466e38f, some = amax >= kLeastMax;
    scale = finite ? (some ? amax * (1.f / kE4m3Max) : 0.f) : __builtin_nanf("");
    mul = finite && some ? r * kE4m3Max : 0.f;
}

template <bool kFull, int kType>
__device__ __forceinline__ void step32(const MultiDesc& d, const Hyper& h, int64_t base) {
    constexpr int kRuns = 4;  // loads of a lane
    floatx4 w[kRuns], g[kRuns], m[kRuns], v[kRuns];
    int valid[kRuns];
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        const int64_t i = base + (int64_t)(k * kMultiThreads + threadIdx.x) * 4;
        valid[k] = kFull ? 4 : (int)min((int64_t)4, max((int64_t)0, d.n - i));
        w[k] = load4(d.w + i, valid[k]);
        g[k] = load_grad<kType>(d.g, d.g_type, i, valid[k]);
        m[k] = load4(reinterpret_cast<const float*>(d.m) + i, valid[k]);
        v[k] = load4(reinterpret_cast<const float*>(d.v) + i, valid[k]);
    }
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        const int64_t i = base + (int64_t)(k * kMultiThreads + threadIdx.x) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float mv = m[k][e], vv = v[k][e], u;
            w[k][e] = adam(h, w[k][e], g[k][e], mv, vv, u);
            m[k][e] = mv;
            v[k][e] = vv;
        }
        store4(d.w + i, w[k], valid[k]);
        store4(reinterpret_cast<float*>(d.m) + i, m[k], valid[k]);
        store4(reinterpret_cast<float*>(d.v) + i, v[k], valid[k]);
        if (d.copy) store_copy(d.copy, d.copy_type, i, w[k], valid[k]);
    }
}

// x << 16, in a form that is not turned into one more multiplication by the hash's constant.
__device__ __forceinline__ uint32_t high_half(uint32_t x) { return __builtin_amdgcn_alignbit(x, 0u, 16u); }

// 8-bit states. A wave takes four blocks of 256 elements, 16 lanes a block: lane l of a
// block has elements 64 c + 4 l + e, so that a load of four elements a lane is 256
// contiguous bytes of fp32 a block, and the largest magnitude is found in a lane's 16
// registers and four exchanges within 16 lanes (a block over all 64 lanes takes six
// exchanges for every four elements of a lane, and its scale's arithmetic four times over:
// 90 issue slots an element instead of about 60, and 825 us instead of 742 us for 268 M).
// Stochastic rounding to e4m3 is one instruction: v_cvt_sr_fp8_f32 adds the top 20 bits of
// its random operand to the part of the value that is cut, subnormal codes included (on
// 2^24 pairs of values and bits it gave the same codes as the integer form of the header's
// rule). A product x mul passes 448 by at most three units in the last place, which no
// random bits carry to the next code. The random bits are one hash an element, 16 for
// each moment.
template <bool kFull, int kType>
__device__ __forceinline__ void step8(const MultiDesc& d, const Hyper& h, int64_t base, uint32_t key) {
    constexpr int kRuns = 4;  // loads of a lane
    static_assert(kMultiBlockElems == kMultiThreads / 64 * 4 * kQBlock, "every wave takes four blocks");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t from = base + wave * (4 * kQBlock);
    const int in = (lane >> 4) * kQBlock + (lane & 15) * 4;  // the lane's first element in the wave's 1024
    const int64_t q = from / kQBlock + (lane >> 4);
    if (!kFull && from >= d.n) return;
    floatx4 w[kRuns], g[kRuns];
    unsigned mc[kRuns], vc[kRuns];
    int valid[kRuns];
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        const int64_t i = from + in + k * 64;
        valid[k] = kFull ? 4 : (int)min((int64_t)4, max((int64_t)0, d.n - i));
        w[k] = load4(d.w + i, valid[k]);
        g[k] = load_grad<kType>(d.g, d.g_type, i, valid[k]);
        mc[k] = load_codes(d.m, i, valid[k]);
        vc[k] = load_codes(d.v, i, valid[k]);
    }
    const bool some = kFull || q * kQBlock < d.n;
    const float ms = some ? d.ms[q] : 0.f, vs = some ? d.vs[q] : 0.f;
    float m[kRuns][4], u[kRuns][4], mmax = 0.f, umax = 0.f;
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        const floatx4 md = decode(mc[k]), ud = decode(vc[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            m[k][e] = md[e] * ms;
            const float u0 = ud[e] * vs;
            float v = u0 * u0;
            w[k][e] = adam(h, w[k][e], g[k][e], m[k][e], v, u[k][e]);
            // a maximum that a NaN wins
            mmax = __builtin_elementwise_maximum(mmax, fabsf(m[k][e]));
            umax = __builtin_elementwise_maximum(umax, u[k][e]);
        }
        const int64_t i = from + in + k * 64;
        store4(d.w + i, w[k], valid[k]);
        if (d.copy) store_copy(d.copy, d.copy_type, i, w[k], valid[k]);
    }
    // bit patterns of magnitudes: NaN above infinity above the finite ones
    mmax = __uint_as_float(lanes_max<16>(__float_as_uint(mmax) & 0x7FFFFFFFu));
    umax = __uint_as_float(lanes_max<16>(__float_as_uint(umax) & 0x7FFFFFFFu));
    float msc, mmul, usc, umul;
    block_scale(mmax, msc, mmul);
    block_scale(umax, usc, umul);
    if ((lane & 15) == 0 && some) {
        d.ms[q] = msc;
        d.vs[q] = usc;
    }
    // all of the wave's elements have one high index word: it starts at a multiple of 1024
    const uint32_t first = (uint32_t)from * 0x9E3779B9u + (uint32_t)((uint64_t)from >> 32) * 0x510E527Fu + key;
    const uint32_t mine = first + (uint32_t)in * 0x9E3779B9u;
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
        int mo = 0, uo = 0;
#define MUON_QUANTISE(e)                                                                                     \
    {                                                                                                        \
        const uint32_t bits = mix32(mine + (k * 64 + (e)) * 0x9E3779B9u);                                    \
        /* the median keeps 0 and lifts what lies between 0 and the least code to it */                      \
        const float ua = __builtin_amdgcn_fmed3f(u[k][e] * umul, 0x1p-9f, u[k][e] * 0x1p126f);               \
        mo = __builtin_amdgcn_cvt_sr_fp8_f32(m[k][e] * mmul, (int)(bits << 16), mo, e);                      \
        uo = __builtin_amdgcn_cvt_sr_fp8_f32(ua, (int)(bits & 0xFFFF0000u), uo, e);                          \
    }
        MUON_QUANTISE(0)
        MUON_QUANTISE(1)
        MUON_QUANTISE(2)
        MUON_QUANTISE(3)
#undef MUON_QUANTISE
        const int64_t i = from + in + k * 64;
        store_codes(d.m, i, (unsigned)mo, valid[k]);
        store_codes(d.v, i, (unsigned)uo, valid[k]);
    }
}

// kBits: the states' width where the whole plan has one, 0 where both occur (a kernel of its
// own for each width, as the 32-bit path's registers would halve the other's waves).
template <int kBits>
__global__ __launch_bounds__(kMultiThreads) void k_adamw_multi(MultiArgs a) {
    const MultiDesc& d = a.table[a.tensor_of_block[blockIdx.x]];
    const int64_t base = (int64_t)(blockIdx.x - d.blk_begin) * kMultiBlockElems;
    Hyper h;
    h.b1 = a.beta1;
    h.b2 = a.beta2;
    h.ob1 = a.one_minus_beta1;
    h.ob2 = a.one_minus_beta2;
    h.eps = a.eps;
    const MultiScalars sc = a.scalars ? *a.scalars : a.host;
    h.step = sc.lr_bc1 * d.lr_scale;
    h.inv_sqrt_bc2 = sc.inv_sqrt_bc2;
    h.decay = (float)(1.0 - sc.lr_wd * (double)d.lr_scale * (double)d.wd_scale);
    h.gs = a.grad_scale ? *a.grad_scale : 1.f;
    const bool full = base + kMultiBlockElems <= d.n;
    if (kBits == 8 || (kBits == 0 && d.bits == 8)) {
        const uint32_t key = mix32(sc.key + (uint32_t)d.index * 0x510E527Fu);
        if (!full) step8<false, -1>(d, h, base, key);
        else if (d.g_type == kF32) step8<true, kF32>(d, h, base, key);
        else if (d.g_type == kBF16) step8<true, kBF16>(d, h, base, key);
        else step8<true, kF16>(d, h, base, key);
    } else if constexpr (kBits != 8) {
        if (!full) step32<false, -1>(d, h, base);
        else if (d.g_type == kF32) step32<true, kF32>(d, h, base);
        else if (d.g_type == kBF16) step32<true, kBF16>(d, h, base);
        else step32<true, kF16>(d, h, base);
    }
}

// The scalars of a step whose counter is on the device, and the counter's increase: one
// thread, in double as the host's.
__global__ void k_multi_scalars(MultiScalarArgs a) {
    const int64_t step = *a.counter;
    const double t = (double)step + 1.0, lr = a.lr ? (double)*a.lr : (double)a.lr_host;
    MultiScalars s;
    s.lr_bc1 = (float)(lr / (1.0 - pow((double)a.beta1, t)));
    s.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow((double)a.beta2, t)));
    s.lr_wd = lr * (double)a.weight_decay;
    s.key = mix32(a.seed_key + (uint32_t)step);
    s.pad_ = 0;
    *a.out = s;
    *a.counter = step + 1;
}

__global__ void k_grad_table(GradDescArgs a) {
    const int i = threadIdx.x;
    if (i < a.n) a.table[a.first + i] = a.d[i];
}

}  // namespace

hipError_t launch_multi_table(const MultiDescArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_multi_table, dim3(a.n), dim3(64), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_multi_map(const MultiDesc* table, int count, int32_t* map, int blocks, hipStream_t s) {
    hipLaunchKernelGGL(k_map<MultiDesc>, dim3((unsigned(blocks) + 255) / 256), dim3(256), 0, s, table, count, map, blocks);
    return hipGetLastError();
}

hipError_t launch_multi_scalars(const MultiScalarArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_multi_scalars, dim3(1), dim3(1), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_multi_step(const MultiArgs& a, hipStream_t s) {
    if (a.bits == 8) hipLaunchKernelGGL(k_adamw_multi<8>, dim3(a.blocks), dim3(kMultiThreads), 0, s, a);
    else if (a.bits == 32) hipLaunchKernelGGL(k_adamw_multi<32>, dim3(a.blocks), dim3(kMultiThreads), 0, s, a);
    else hipLaunchKernelGGL(k_adamw_multi<0>, dim3(a.blocks), dim3(kMultiThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_table(const GradDescArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_grad_table, dim3(1), dim3(128), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_map(const GradDesc* table, int count, int32_t* map, int blocks, hipStream_t s) {
    hipLaunchKernelGGL(k_map<GradDesc>, dim3((unsigned(blocks) + 255) / 256), dim3(256), 0, s, table, count, map, blocks);
    return hipGetLastError();
}

}  // namespace muon

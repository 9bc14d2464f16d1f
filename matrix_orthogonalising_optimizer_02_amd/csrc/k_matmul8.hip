// Products of matrices in 8 bits with a power of two for every 128 elements (blocks8.hpp):
//   C[i][j] = sum over blocks of 2^(ea + eb) sum over the block of a[i][k] b[j][k]
// Both operands lie with k along their rows, so that every fragment of a matrix instruction is
// contiguous bytes.
#include "blocks8.hpp"
#include "rows.hpp"

#include <algorithm>

namespace muon {
namespace {

typedef int v8i32 __attribute__((ext_vector_type(8)));
typedef int v4i32 __attribute__((ext_vector_type(4)));
typedef __bf16 bf162 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

template <bool B>
struct BoolC {
    static constexpr bool value = B;
};
template <int N>
struct IntC {
    static constexpr int value = N;
};

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// Without the fence of __syncthreads(), which waits for every load in flight: each wave waits
// for what it needs itself before it comes here.
__device__ __forceinline__ void barrier_no_fence() { asm volatile("s_barrier" ::: "memory"); }

__device__ __forceinline__ void* uniform_ptr(const void* q) {
    const uint64_t v = reinterpret_cast<uint64_t>(q);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* q) {
    return __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(q), (short)0, 0x7FFFFFFF, 0x00020000);
}

// The products of one fragment pair over 64 k. Narrow: one scaled 8-bit instruction. Wide: the
// codes become bf16 (exact, powers included) and go through four bf16 instructions, whose sums
// are as good as a sequence of fp32 additions; the 8-bit instruction rounds inside (the sum of
// 64 products is off by 2^-16 of it on gaussian codes, 2^-12 of the sum of magnitudes at most
// on codes of any size), which a 16-bit result does not show and an fp32 one does.
constexpr int kRaster = 8;  // tile rows that are walked together, so that their B panels meet in L2

struct TileAt {
    int ti, tj, part;
};

// Blocks are dealt round-robin over the 8 XCDs. XCD x takes one contiguous eighth of all tiles
// (of all parts of k, the parts one after another), walked in groups of kRaster tile rows, so
// that what it reads at a time is a compact patch that meets in its L2.
__device__ __forceinline__ bool tile_of(const Mat8Args& a, TileAt& t) {
    const int tiles = a.tiles_m * a.tiles_n, total = tiles * a.splits;
    const int x = blockIdx.x & 7, sl = blockIdx.x >> 3;
    const int lo = (int)(((int64_t)x * total) >> 3), hi = (int)(((int64_t)(x + 1) * total) >> 3);
    if (sl >= hi - lo) return false;
    const int u = lo + sl;
    t.part = u / tiles;
    const int local = u - t.part * tiles;
    const int per = kRaster * a.tiles_n, g = local / per, first = g * kRaster;
    const int rows = min(a.tiles_m - first, kRaster), r = local - g * per;
    t.ti = first + r % rows;
    t.tj = r / rows;
    return true;
}

// c[col .. col + 7] of a row from eight fp32 sums.
__device__ __forceinline__ void put8(const Mat8Args& a, int row, int col, float* f) {
    const int64_t at = (int64_t)row * a.ldc + col;
    if (a.dtype == kF32) {
        float* c = reinterpret_cast<float*>(a.c) + at;
        if (col + 8 <= a.n) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (a.accumulate) {
                    float o[4];
                    Elem<kF32>::unpack(load16(c + 4 * h), o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[4 * h + e] += o[e];
                }
                store16(c + 4 * h, Elem<kF32>::pack(f + 4 * h));
            }
        } else {
            for (int e = 0; e < 8 && col + e < a.n; ++e) c[e] = a.accumulate ? c[e] + f[e] : f[e];
        }
        return;
    }
    unsigned short* c = reinterpret_cast<unsigned short*>(a.c) + at;
    auto old = [&](unsigned short u) { return a.dtype == kBF16 ? bf2f(u) : (float)__builtin_bit_cast(_Float16, u); };
    if (col + 8 <= a.n) {
        if (a.accumulate) {
            const u32x4 r = load16(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += old((unsigned short)(r[e >> 1] >> (16 * (e & 1))));
        }
        store16(c, a.dtype == kBF16 ? Elem<kBF16>::pack(f) : Elem<kF16>::pack(f));
    } else {
        for (int e = 0; e < 8 && col + e < a.n; ++e) {
            const float v = a.accumulate ? f[e] + old(c[e]) : f[e];
            if (a.dtype == kBF16) c[e] = f2bf(v);
            else reinterpret_cast<_Float16*>(c)[e] = (_Float16)v;
        }
    }
}

// A block of four waves (2 x 2) computes kSide x kSide of C, a wave a quarter of it in 32 x 32
// accumulators. A step is 128 of k: both operands' tiles come straight to LDS (a load of 1 KiB
// brings 8 rows of 128 bytes, whole cache lines), two stages. The wave reads a half step's
// fragments (64 of k) while the matrix instructions work on the half before, and once all waves
// hold a step's second half in registers, one barrier a step, its stage is filled again: a load
// has one and a half steps to arrive. Rows of LDS are 128 bytes; chunk c of row r (16 bytes)
// sits at c ^ ((r / 2) & 7), so that 16 lanes that read the same chunk of 16 rows meet all banks.
// Rows past the matrix's end are its last row again, and are not stored.
template <int kSide, bool kWide>
struct Mat8Lds {
    static constexpr int kEpi = 32 * (kSide / 2 + 4) * 4;                       // a wave's 32 staged rows of the result
    static constexpr int kBytes = std::max(2 * 2 * kSide * 128, 4 * kEpi);
};

template <int kSide, bool kWide>
__device__ __forceinline__ void matmul8_tile(const Mat8Args& a, uint8_t* smem) {
    constexpr int kHalf = kSide / 2, T = kHalf / 32;    // a wave's side, and in fragments
    constexpr int kLoads = kSide / 32;                  // 1 KiB loads of a wave, an operand and a step
    constexpr int kTile = kSide * 128, kStage = 2 * kTile;
    constexpr int kRowF = kHalf + 4;                    // floats of a staged row of the result
    constexpr int kEpi = Mat8Lds<kSide, kWide>::kEpi;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    TileAt t;
    if (!tile_of(a, t)) return;
    // this part's steps: cut at multiples of four, whose powers are one dword of a row
    const int fours = (a.steps + 3) >> 2;
    const int s0 = 4 * (int)((int64_t)t.part * fours / a.splits);
    const int s1 = min(a.steps, 4 * (int)((int64_t)(t.part + 1) * fours / a.splits));
    const int nk = s1 - s0;
    const int row0 = t.ti * kSide, col0 = t.tj * kSide;

    const __amdgpu_buffer_rsrc_t ra = resource(a.a + (int64_t)row0 * a.lda + (int64_t)s0 * 128);
    const __amdgpu_buffer_rsrc_t rb = resource(a.b + (int64_t)col0 * a.ldb + (int64_t)s0 * 128);
    const __amdgpu_buffer_rsrc_t rsa = resource(a.as + (int64_t)(row0 >> a.sha) * a.lsa + s0);
    const __amdgpu_buffer_rsrc_t rsb = resource(a.bs + (int64_t)(col0 >> a.shb) * a.lsb + s0);
    uint32_t offa[kLoads], offb[kLoads], offsa[T], offsb[T];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
        const int r = (wave * kLoads + q) * 8 + (lane >> 3);
        const uint32_t chunk = (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) * 16;
        offa[q] = (uint32_t)min(r, a.m - 1 - row0) * (uint32_t)a.lda + chunk;
        offb[q] = (uint32_t)min(r, a.n - 1 - col0) * (uint32_t)a.ldb + chunk;
    }
#pragma unroll
    for (int f = 0; f < T; ++f) {
        const int r = f * 32 + (lane & 31);
        offsa[f] = (uint32_t)((min(row0 + wm * kHalf + r, a.m - 1) >> a.sha) - (row0 >> a.sha)) * (uint32_t)a.lsa;
        offsb[f] = (uint32_t)((min(col0 + wn * kHalf + r, a.n - 1) >> a.shb) - (col0 >> a.shb)) * (uint32_t)a.lsb;
    }
    auto load = [&](int stage, int step, int q) {  // q < 2 kLoads
        uint8_t* to = smem + stage * kStage + (q < kLoads ? 0 : kTile) + (wave * kLoads + q % kLoads) * 1024;
        if (q < kLoads) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)to, 16, offa[q], step * 128, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)to, 16, offb[q - kLoads], step * 128, 0, 0);
    };
    // powers of the present four steps and of the next four, a dword a fragment
    unsigned pa[T], pb[T], na[T], nb[T];
    auto load_powers = [&](int four) {
#pragma unroll
        for (int f = 0; f < T; ++f) {
            na[f] = __builtin_amdgcn_raw_buffer_load_b32(rsa, offsa[f], four * 4, 0);
            nb[f] = __builtin_amdgcn_raw_buffer_load_b32(rsb, offsb[f], four * 4, 0);
        }
    };
    // fragments of a half step: lane l holds row l % 32, 32 bytes: chunks 4 half + 2 (l / 32), + 1
    v4i32 fa[2][T][2], fb[2][T][2];
    const int sw = (lane >> 1) & 7, lrow = (lane & 31) * 128;
    auto frag = [&](int half, int stage, int i) {  // i < 4 T: one 16-byte read
        const int j = i & 1, f = (i >> 1) % T;
        const bool is_b = i >= 2 * T;
        const int chunk = ((half * 4 + (lane >> 5) * 2 + j) ^ sw) * 16;
        const uint8_t* p = smem + stage * kStage + (is_b ? kTile + wn * kHalf * 128 : wm * kHalf * 128) + f * 4096 + lrow + chunk;
        const v4i32 v = *reinterpret_cast<const v4i32*>(p);
        if (is_b) fb[half][f][j] = v;
        else fa[half][f][j] = v;
    };
    floatx16 acc[T][T];  // [n][m]: a lane holds four consecutive columns of one row of C
#pragma unroll
    for (int b = 0; b < T; ++b)
#pragma unroll
        for (int m = 0; m < T; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[b][m][r] = 0.f;

    auto whole = [](const v4i32 (&h)[2]) { return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7); };
    // i-th fragment pair, snake order: two in a row differ in one operand only
    auto pair = [](int i, int& b, int& m) {
        b = i / T;
        m = b & 1 ? T - 1 - i % T : i % T;
    };
    // `between(slot)`, slot < T T: what is issued after the slot's matrix instructions
    auto multiply = [&](int half, auto phase_c, int phase, auto between) {
        constexpr int PH = decltype(phase_c)::value;
        if constexpr (!kWide) {
#pragma unroll
            for (int i = 0; i < T * T; ++i) {
                int b, m;
                pair(i, b, m);
                // PH < 0: the byte was moved down already
                acc[b][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(whole(fb[half][b]), whole(fa[half][m]), acc[b][m], 0, 0,
                                                                           PH < 0 ? 0 : PH, (int)pb[b], PH < 0 ? 0 : PH,
                                                                           (int)pa[m]);
                between(i);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            float sa[T], sb[T];
            const int sh = PH < 0 ? 0 : 8 * PH;
#pragma unroll
            for (int f = 0; f < T; ++f) {
                sa[f] = power_value((pa[f] >> sh) & 255u);
                sb[f] = power_value((pb[f] >> sh) & 255u);
            }
            auto widen = [](unsigned lo, unsigned hi, float s) {
                const bf162 w[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true),
                                    __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true)};
                return bf16x8{w[0][0], w[0][1], w[1][0], w[1][1], w[2][0], w[2][1], w[3][0], w[3][1]};
            };
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                bf16x8 wa[T], wb[T];
#pragma unroll
                for (int f = 0; f < T; ++f) {
                    wa[f] = widen(fa[half][f][s >> 1][2 * (s & 1)], fa[half][f][s >> 1][2 * (s & 1) + 1], sa[f]);
                    wb[f] = widen(fb[half][f][s >> 1][2 * (s & 1)], fb[half][f][s >> 1][2 * (s & 1) + 1], sb[f]);
                }
#pragma unroll
                for (int i = 0; i < T * T; ++i) {
                    int b, m;
                    pair(i, b, m);
                    acc[b][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[b], wa[m], acc[b][m], 0, 0, 0);
                }
                // a quarter of the slots
#pragma unroll
                for (int i = 0; i < (T * T) / 4; ++i) between(s * ((T * T) / 4) + i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    constexpr int kSlots = T * T, kReads = (4 * T + kSlots / 2 - 1) / (kSlots / 2), kPuts = (2 * kLoads + kSlots / 2 - 1) / (kSlots / 2);
    // one step of 128. MORE: step kt + 2 is loaded; NEXT: step kt + 1 exists. PH: kt % 4, -1
    // where it is known at run time only.
    auto step = [&](int kt, auto more_c, auto next_c, auto phase_c) {
        constexpr bool MORE = decltype(more_c)::value, NEXT = decltype(next_c)::value;
        constexpr int PH = decltype(phase_c)::value;
        const int cur = PH >= 0 ? PH & 1 : kt & 1;
        if (PH == 0 || (PH < 0 && (kt & 3) == 0)) {
#pragma unroll
            for (int f = 0; f < T; ++f) {
                pa[f] = na[f];
                pb[f] = nb[f];
            }
            load_powers(min((kt >> 2) + 1, (nk - 1) >> 2));
        }
        // without a phase the dwords move down a byte a step: byte 0 is always this step's
        multiply(0, phase_c, kt, [&](int i) {
#pragma unroll
            for (int q = 0; q < kReads; ++q)
                if (i * kReads + q < 4 * T) frag(1, cur, i * kReads + q);
        });
        if (NEXT) {
            wait_lds();
            wait_loads();
            barrier_no_fence();
        }
        multiply(1, phase_c, kt, [&](int i) {
            if (MORE) {
#pragma unroll
                for (int q = 0; q < kPuts; ++q)
                    if (i * kPuts + q < 2 * kLoads) load(cur, kt + 2, i * kPuts + q);
            }
            if (NEXT) {
#pragma unroll
                for (int q = 0; q < kReads; ++q)
                    if (i * kReads + q < 4 * T) frag(0, cur ^ 1, i * kReads + q);
            }
        });
        if constexpr (PH < 0) {
#pragma unroll
            for (int f = 0; f < T; ++f) {
                pa[f] >>= 8;
                pb[f] >>= 8;
            }
        }
    };
    constexpr BoolC<true> Y{};
    constexpr BoolC<false> N{};
    if (nk > 0) {
        load_powers(0);
#pragma unroll
        for (int q = 0; q < 2 * kLoads; ++q) load(0, 0, q);
        if (nk > 1)
#pragma unroll
            for (int q = 0; q < 2 * kLoads; ++q) load(1, 1, q);
        wait_loads();
        barrier_no_fence();
#pragma unroll
        for (int i = 0; i < 4 * T; ++i) frag(0, 0, i);
        int kt = 0;
        for (; kt + 5 < nk; kt += 4) {
            step(kt, Y, Y, IntC<0>{});
            step(kt + 1, Y, Y, IntC<1>{});
            step(kt + 2, Y, Y, IntC<2>{});
            step(kt + 3, Y, Y, IntC<3>{});
        }
        for (; kt + 2 < nk; ++kt) step(kt, Y, Y, IntC<-1>{});
        if (kt + 1 < nk) step(kt++, N, Y, IntC<-1>{});
        step(kt, N, N, IntC<-1>{});
    }
    wait_loads();
    __syncthreads();

    // A wave's result leaves 32 rows at a time through its own part of LDS, so that every store
    // is 16 bytes of a row: 16 lanes a row in 16 bits.
    float* const st = reinterpret_cast<float*>(smem + wave * kEpi);
    Mat8Args o = a;
    if (a.splits > 1) {
        o.c = a.partial + (int64_t)t.part * a.m * a.n;
        o.ldc = a.n;
        o.dtype = kF32;
        o.accumulate = 0;
    }
    const int rbase = row0 + wm * kHalf, cbase = col0 + wn * kHalf;
#pragma unroll
    for (int m = 0; m < T; ++m) {
#pragma unroll
        for (int b = 0; b < T; ++b)
#pragma unroll
            for (int rg = 0; rg < 4; ++rg) {
                const floatx4 v = {acc[b][m][4 * rg], acc[b][m][4 * rg + 1], acc[b][m][4 * rg + 2], acc[b][m][4 * rg + 3]};
                *reinterpret_cast<floatx4*>(st + (lane & 31) * kRowF + b * 32 + rg * 8 + (lane >> 5) * 4) = v;
            }
        wait_lds();
        constexpr int kPer = kHalf / 8;  // 8 columns a lane
#pragma unroll
        for (int it = 0; it < 32 * kPer / 64; ++it) {
            const int c = it * 64 + lane, r = c / kPer, k = c % kPer;
            float f[8];
            *reinterpret_cast<floatx4*>(f) = *reinterpret_cast<const floatx4*>(st + r * kRowF + k * 8);
            *reinterpret_cast<floatx4*>(f + 4) = *reinterpret_cast<const floatx4*>(st + r * kRowF + k * 8 + 4);
            const int row = rbase + m * 32 + r, col = cbase + k * 8;
            if (row < a.m && col < a.n) put8(o, row, col, f);
        }
        wait_lds();
    }
}

template <int kSide, bool kWide>
__global__ __launch_bounds__(256, kSide == 256 ? 1 : 2) void k_matmul8(Mat8Args a) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Mat8Lds<kSide, kWide>::kBytes];
    matmul8_tile<kSide, kWide>(a, smem);
}

// Adds the parts of k in order.
__global__ __launch_bounds__(256) void k_matmul8_join(Mat8Args a, int chunks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = (int)(i / chunks), col = (int)(i - (int64_t)row * chunks) * 8;
    if (row >= a.m) return;
    const float* p = a.partial + (int64_t)row * a.n + col;
    const int64_t part = (int64_t)a.m * a.n;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
        if (col + 8 <= a.n) {
            float g[8];
            Elem<kF32>::unpack(load16(p + s * part), g);
            Elem<kF32>::unpack(load16(p + s * part + 4), g + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += g[e];
        } else {
            for (int e = 0; e < 8 && col + e < a.n; ++e) f[e] += p[s * part + e];
        }
    }
    put8(a, row, col, f);
}

}  // namespace

Mat8Plan plan_matmul8(int64_t m, int64_t n, int64_t k, bool wide) {
    Mat8Plan p{};
    auto tiles = [&](int64_t side) { return ((m + side - 1) / side) * ((n + side - 1) / side); };
    p.tile = tiles(256) >= 128 ? 256 : 128;
    p.splits = 1;
    const int64_t room = p.tile == 256 ? 256 : 512, fours = (k + 511) / 512;
    if (tiles(p.tile) < room) p.splits = (int)std::max<int64_t>(1, std::min(room / tiles(p.tile), fours / 2));
    if (p.splits > 1) p.partial_bytes = size_t(p.splits) * size_t(m) * size_t(n) * 4;
    return p;
}

hipError_t launch_matmul8(const Mat8Plan& p, bool wide, const Mat8Args& a, hipStream_t s) {
    const int64_t total = int64_t(a.tiles_m) * a.tiles_n * a.splits;
    const dim3 grid((unsigned)(8 * ((total + 7) / 8))), block(256);
    if (p.tile == 256) {
        if (wide) hipLaunchKernelGGL((k_matmul8<256, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_matmul8<256, false>), grid, block, 0, s, a);
    } else {
        if (wide) hipLaunchKernelGGL((k_matmul8<128, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_matmul8<128, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_matmul8_join(const Mat8Args& a, hipStream_t s) {
    const int chunks = (a.n + 7) / 8;
    const dim3 grid((unsigned)((int64_t(a.m) * chunks + 255) / 256)), block(256);
    hipLaunchKernelGGL(k_matmul8_join, grid, block, 0, s, a, chunks);
    return hipGetLastError();
}

}  // namespace muon

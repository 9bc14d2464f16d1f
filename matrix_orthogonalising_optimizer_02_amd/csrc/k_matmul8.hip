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

// Two ways to multiply. Narrow: the scaled 8-bit instructions. They add products in groups of
// eight, in which bits below 2^-13 of the largest product are dropped (found with one large and
// one small product at every pair of places), and the groups in fp32: a sum is off by 2^-16 of
// it, root mean square, on normally distributed values, and by 2^-10 of its magnitudes' sum at
// most. That is the choice for 16-bit results, for twice the rate: on such values it is a 32nd of
// fp16's half step and a 256th of bf16's ([1003, 2011] x [1153, 2011] into fp16 off by 2.09e-4
// relative, with fp32 sums 2.07e-4). The most that it can be is above fp16's half step, and above
// bf16's where a sum is less than a quarter of its magnitudes: who has such sums asks for the wide
// form. Wide: eight codes become bf16, exactly and with their powers, for bf16 instructions at
// half the rate, whose sums are as good as a sequence of fp32 additions; fp32 results take it.
__device__ __forceinline__ bf16x8 widen(unsigned lo, unsigned hi, float power) {
    const bf162_t w[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, false),
                        __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, true),
                        __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, false),
                        __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, true)};
    return bf16x8{w[0][0], w[0][1], w[1][0], w[1][1], w[2][0], w[2][1], w[3][0], w[3][1]};
}

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

// A block computes kSide x kSide of C in 32 x 32 accumulators, a wave a part of it: eight waves
// (2 x 4, two a SIMD, each 128 x 64) for 256 x 256 in the 8-bit instructions, else four (2 x 2). A
// step is 128 of k: both operands' tiles come straight to LDS (a load of 1 KiB brings 8 rows of 128
// bytes, whole cache lines), two stages. The wave reads a half step's fragments (64 of k) while the
// matrix instructions work on the half before, and once all waves hold a step's second half in
// registers, one barrier a step, its stage is filled again. Rows of LDS are 128 bytes; chunk c of
// row r (16 bytes) sits at c ^ ((r / 2) & 7), so that 16 lanes that read the same chunk of 16 rows
// meet all banks. Rows past the matrix's end are its last row again, and are not stored.
// What bounds 256 x 256: a step's matrix instructions take 1.0 us, its LDS reads hide behind them
// in part, and 64 KiB a compute unit and step come from L2 at some 65 lines in flight; asking for
// half of a step's loads a half step later, A's and B's in turn, took [8192, 20480, 5120] from 718
// to 655 us (2.6 PFLOP/s; 3.9 with nothing but matrix instructions). Halves of lines (64 of k a
// stage, four stages) took 759 us, k begun at another place by every block 735 to 939 us, four
// waves of 128 x 128 a block 705 us, blocks that stay for further tiles and load the next one's
// first step while a result leaves 676 us (alike blocks then store at the same time).
template <int kSide, bool kWide>
struct Mat8Cfg {
    static constexpr bool kDense = kSide == 256 && !kWide;                      // two waves a SIMD of 256 registers
    static constexpr int kWavesN = kDense ? 4 : 2, kWaves = 2 * kWavesN;        // 2 waves along m
    static constexpr int kM = kSide / 2, kN = kSide / kWavesN;                  // a wave's part
    static constexpr int kEpi = 32 * (kN + 4) * 4;                              // its 32 staged rows of the result
    static constexpr int kPowers = 2 * kSide * 4;                               // both operands' powers of four steps
    static constexpr int kLds = std::max(2 * 2 * kSide * 128 + 2 * kPowers, kWaves * kEpi);
};

template <int kSide, bool kWide>
__device__ __forceinline__ void matmul8_tile(const Mat8Args& a, uint8_t* smem) {
    typedef Mat8Cfg<kSide, kWide> Cfg;
    constexpr int kM = Cfg::kM, kN = Cfg::kN, TM = kM / 32, TN = kN / 32;  // a wave's part, and in fragments
    constexpr int kLoads = kSide / 8 / Cfg::kWaves;     // 1 KiB loads of a wave, an operand and a step
    // A's two stages, then B's: a wave's reads of both are within an instruction's offset of one address
    constexpr int kTile = kSide * 128;
    constexpr int kRowF = kN + 4;                       // floats of a staged row of the result
    constexpr int kEpi = Cfg::kEpi;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / Cfg::kWavesN, wn = wave % Cfg::kWavesN;
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
    uint32_t offa[kLoads], offb[kLoads];
    // Eight tiles next to each other along m run at the same time on one XCD and read the same rows
    // of B, and four along n the same of A. Each begins with other rows (the wave's loads in another
    // turn): the rows that a block asks for first come from memory, and the other blocks find them in
    // L2 when their turn comes (718 to 680 us by itself; tiles of 128, of few steps, show nothing).
    const int turn_a = kSide == 256 ? t.tj * (kLoads / 4) : 0, turn_b = kSide == 256 ? t.ti * kLoads / 8 : 0;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
        const int r = (wave * kLoads + (q + turn_a) % kLoads) * 8 + (lane >> 3);
        offa[q] = (uint32_t)min(r, a.m - 1 - row0) * (uint32_t)a.lda + (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) * 16;
        const int s = (wave * kLoads + (q + turn_b) % kLoads) * 8 + (lane >> 3);
        offb[q] = (uint32_t)min(s, a.n - 1 - col0) * (uint32_t)a.ldb + (uint32_t)((lane & 7) ^ ((s >> 1) & 7)) * 16;
    }
    // The powers of four steps, a dword a row, come to LDS as well: 64 rows a load, A's 256 (128)
    // first, in two places in turn.
    constexpr int kPowerLoads = 2 * kSide / 64 / Cfg::kWaves;
    uint8_t* const powers = smem + 4 * kTile;
    uint32_t offp[kPowerLoads];
#pragma unroll
    for (int q = 0; q < kPowerLoads; ++q) {
        const int r = (wave * kPowerLoads + q) * 64 % kSide + lane;
        const bool is_b = (wave * kPowerLoads + q) * 64 >= kSide;
        offp[q] = is_b ? (uint32_t)((min(col0 + r, a.n - 1) >> a.shb) - (col0 >> a.shb)) * (uint32_t)a.lsb
                       : (uint32_t)((min(row0 + r, a.m - 1) >> a.sha) - (row0 >> a.sha)) * (uint32_t)a.lsa;
    }
    auto load_powers = [&](int four) {
        const int from = min(four, (nk - 1) >> 2);  // past the end: once more, and not read
#pragma unroll
        for (int q = 0; q < kPowerLoads; ++q) {
            const int at = wave * kPowerLoads + q;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(at * 64 >= kSide ? rsb : rsa, (lds_ptr_t)(powers + (four & 1) * Cfg::kPowers + at * 256),
                                                     4, offp[q], from * 4, 0, 0);
        }
    };
    unsigned pa[TM], pb[TN];
    auto read_powers = [&](int four) {
        const unsigned* p = reinterpret_cast<const unsigned*>(powers + (four & 1) * Cfg::kPowers);
#pragma unroll
        for (int f = 0; f < TM; ++f) pa[f] = p[wm * kM + f * 32 + (lane & 31)];
#pragma unroll
        for (int f = 0; f < TN; ++f) pb[f] = p[kSide + wn * kN + f * 32 + (lane & 31)];
    };
    auto load = [&](int stage, int step, int i) {  // i < 2 kLoads
        const int q = Cfg::kDense ? i >> 1 : i % kLoads;
        if (Cfg::kDense ? i & 1 : i >= kLoads) {
            uint8_t* to = smem + (stage + 2) * kTile + (wave * kLoads + (q + turn_b) % kLoads) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)to, 16, offb[q], step * 128, 0, 0);
        } else {
            uint8_t* to = smem + stage * kTile + (wave * kLoads + (q + turn_a) % kLoads) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)to, 16, offa[q], step * 128, 0, 0);
        }
    };
    // fragments of a half step: lane l holds row l % 32, 32 bytes: chunks 4 half + 2 (l / 32), + 1
    // (Dense: A's have one set of registers, and are read again once both of a fragment's products
    // are under way; a second set does not fit)
    constexpr int kSetsA = Cfg::kDense ? 1 : 2;
    v4i32 fa[kSetsA][TM][2], fb[2][TN][2];
    constexpr int kFrags = 2 * (TM + TN);  // 16-byte reads of a half step
    const int sw = (lane >> 1) & 7, lrow = (lane & 31) * 128;
    auto frag = [&](int half, int stage, int i) {  // i < kFrags
        const bool is_b = i >= 2 * TM;
        const int j = i & 1, f = is_b ? (i >> 1) - TM : i >> 1;
        const int chunk = ((half * 4 + (lane >> 5) * 2 + j) ^ sw) * 16;
        const uint8_t* p = smem + (is_b ? 2 * kTile + wn * kN * 128 : wm * kM * 128) + lrow + chunk + stage * kTile + f * 4096;
        const v4i32 v = *reinterpret_cast<const v4i32*>(p);
        if (is_b) fb[half][f][j] = v;
        else fa[half % kSetsA][f][j] = v;
    };
    floatx16 acc[TN][TM];  // [n][m]: a lane holds four consecutive columns of one row of C
#pragma unroll
    for (int b = 0; b < TN; ++b)
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[b][m][r] = 0.f;

    auto whole = [](const v4i32 (&h)[2]) { return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7); };
    // i-th fragment pair, snake order: two in a row differ in one operand only
    auto pair = [](int i, int& b, int& m) {
        if constexpr (Cfg::kDense) {
            m = i / TN;
            b = m & 1 ? TN - 1 - i % TN : i % TN;
        } else {
            b = i / TM;
            m = b & 1 ? TM - 1 - i % TM : i % TM;
        }
    };
    // `between(slot)`, slot < TM TN: what is issued after the slot's matrix instructions
    auto multiply = [&](int half, auto phase_c, auto between) {
        constexpr int PH = decltype(phase_c)::value;
        if constexpr (!kWide) {
#pragma unroll
            for (int i = 0; i < TM * TN; ++i) {
                int b, m;
                pair(i, b, m);
                // PH < 0: the byte was moved down already
                acc[b][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(whole(fb[half][b]), whole(fa[half % kSetsA][m]), acc[b][m], 0, 0,
                                                                           PH < 0 ? 0 : PH, (int)pb[b], PH < 0 ? 0 : PH,
                                                                           (int)pa[m]);
                between(i);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            float sa[TM], sb[TN];
            const int sh = PH < 0 ? 0 : 8 * PH;
#pragma unroll
            for (int f = 0; f < TM; ++f) sa[f] = power_operand((pa[f] >> sh) & 255u);
#pragma unroll
            for (int f = 0; f < TN; ++f) sb[f] = power_operand((pb[f] >> sh) & 255u);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                bf16x8 wa[TM], wb[TN];
#pragma unroll
                for (int f = 0; f < TM; ++f)
                    wa[f] = widen(fa[half % kSetsA][f][s >> 1][2 * (s & 1)], fa[half % kSetsA][f][s >> 1][2 * (s & 1) + 1], sa[f]);
#pragma unroll
                for (int f = 0; f < TN; ++f)
                    wb[f] = widen(fb[half][f][s >> 1][2 * (s & 1)], fb[half][f][s >> 1][2 * (s & 1) + 1], sb[f]);
#pragma unroll
                for (int i = 0; i < TM * TN; ++i) {
                    int b, m;
                    pair(i, b, m);
                    acc[b][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[b], wa[m], acc[b][m], 0, 0, 0);
                }
                // a quarter of the slots
#pragma unroll
                for (int i = 0; i < (TM * TN) / 4; ++i) between(s * ((TM * TN) / 4) + i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    constexpr int kSlots = TM * TN, kReads = (kFrags + kSlots / 2 - 1) / (kSlots / 2), kPuts = 2;
    // loads of a step that are asked for in the second half of the step two before; the others
    // follow in the first half of the step between
    constexpr int kEarly = kSide == 256 ? kLoads : 2 * kLoads;
    // what slot i reads of the next half: a share of all fragments, or (dense) the one of A whose
    // products are done, and one piece of B's
    auto read = [&](int half, int stage, int i) {
        if constexpr (Cfg::kDense) {
            static_assert(TN == 2 && TM == 4, "two slots a fragment of A, four pieces of B");
            if (i & 1) {
                frag(half, stage, 2 * (i >> 1));
                frag(half, stage, 2 * (i >> 1) + 1);
            } else {
                frag(half, stage, 2 * TM + (i >> 1));
            }
        } else {
#pragma unroll
            for (int q = 0; q < kReads; ++q)
                if (i * kReads + q < kFrags) frag(half, stage, i * kReads + q);
        }
    };
    // one step of 128. MORE: step kt + 2 is loaded; NEXT: step kt + 1 exists. PH: kt % 4, -1
    // where it is known at run time only.
    auto step = [&](int kt, auto more_c, auto next_c, auto phase_c) {
        constexpr bool MORE = decltype(more_c)::value, NEXT = decltype(next_c)::value;
        constexpr int PH = decltype(phase_c)::value;
        const int cur = PH >= 0 ? PH & 1 : kt & 1;
        if (PH == 0 || (PH < 0 && (kt & 3) == 0)) read_powers(kt >> 2);
        // without a phase the dwords move down a byte a step: byte 0 is always this step's
        multiply(0, phase_c, [&](int i) {
            if (NEXT) {
#pragma unroll
                for (int q = 0; q < kPuts; ++q)
                    if (kEarly + i * kPuts + q < 2 * kLoads) load(cur ^ 1, kt + 1, kEarly + i * kPuts + q);
            }
            read(1, cur, i);
        });
        if (NEXT) {
            wait_lds();
            wait_loads();
            barrier_no_fence();
        }
        multiply(1, phase_c, [&](int i) {
            if (i == 0 && MORE && (PH == 0 || (PH < 0 && (kt & 3) == 0))) load_powers((kt >> 2) + 1);
            if (MORE) {
#pragma unroll
                for (int q = 0; q < kPuts; ++q)
                    if (i * kPuts + q < kEarly) load(cur, kt + 2, i * kPuts + q);
            }
            if (NEXT) read(0, cur ^ 1, i);
        });
        if constexpr (PH < 0) {
#pragma unroll
            for (int f = 0; f < TM; ++f) pa[f] >>= 8;
#pragma unroll
            for (int f = 0; f < TN; ++f) pb[f] >>= 8;
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
            for (int q = 0; q < kEarly; ++q) load(1, 1, q);
        wait_loads();
        barrier_no_fence();
#pragma unroll
        for (int i = 0; i < kFrags; ++i) frag(0, 0, i);
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
    const int rbase = row0 + wm * kM, cbase = col0 + wn * kN;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int rg = 0; rg < 4; ++rg) {
                const floatx4 v = {acc[b][m][4 * rg], acc[b][m][4 * rg + 1], acc[b][m][4 * rg + 2], acc[b][m][4 * rg + 3]};
                *reinterpret_cast<floatx4*>(st + (lane & 31) * kRowF + b * 32 + rg * 8 + (lane >> 5) * 4) = v;
            }
        wait_lds();
        constexpr int kPer = kN / 8;  // 8 columns a lane
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
__global__ __launch_bounds__(kSide == 256 && !kWide ? 512 : 256, kSide == 256 && kWide ? 1 : 2) void k_matmul8(Mat8Args a) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Mat8Cfg<kSide, kWide>::kLds];
    matmul8_tile<kSide, kWide>(a, smem);
}

// c[row][col] of one fp32 sum.
__device__ __forceinline__ void put1(const Mat8Args& a, int row, int col, float f) {
    const int64_t at = (int64_t)row * a.ldc + col;
    if (a.dtype == kF32) {
        float* c = reinterpret_cast<float*>(a.c) + at;
        *c = a.accumulate ? *c + f : f;
    } else if (a.dtype == kBF16) {
        unsigned short* c = reinterpret_cast<unsigned short*>(a.c) + at;
        *c = f2bf(a.accumulate ? bf2f(*c) + f : f);
    } else {
        _Float16* c = reinterpret_cast<_Float16*>(a.c) + at;
        *c = (_Float16)(a.accumulate ? (float)*c + f : f);
    }
}

// Few rows of A and a small B: bound by latency, in one launch. A wave takes 16 rows of B with all
// rows of A (kM x 16) and goes along k, kSteps steps of 128 at a time, the next ones asked for
// before the present ones are waited for.
// `share` waves of a block take turns at the steps of the same rows where B has too few rows to
// give every compute unit 8 waves; their sums meet in LDS, in the waves' order. The block's other
// waves take other rows, and find the same pieces of A in the cache. Fragments come straight from
// memory: a lane holds row l % 16, chunks l / 16 and 4 + l / 16 of the 128 bytes (the order of k
// inside a block is free, as a block has one power), so that a load covers 64 contiguous bytes of
// 16 rows.
constexpr int kFewWaves = 8;  // most waves of a block
constexpr int kUnits = 256;   // compute units

template <int kM, bool kWide>
__device__ __forceinline__ void matmul8_few(const Mat8Args& a, float* red) {
    constexpr int kSteps = kM == 1 ? 4 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int share = a.share, own = wave / share, turn = wave - own * share, per_block = waves / share;
    const int col0 = (blockIdx.x * per_block + own) * 16;  // past the end: the last rows again, nothing is stored
    const int s1 = a.steps;
    const uint8_t *pa[kM], *qa[kM];
#pragma unroll
    for (int f = 0; f < kM; ++f) {
        const int r = min(f * 16 + (lane & 15), a.m - 1);
        pa[f] = a.a + (int64_t)r * a.lda + (lane >> 4) * 16;
        qa[f] = a.as + (int64_t)(r >> a.sha) * a.lsa;
    }
    const int rb = min(col0 + (lane & 15), a.n - 1);
    const uint8_t *const pb = a.b + (int64_t)rb * a.ldb + (lane >> 4) * 16, *const qb = a.bs + (int64_t)(rb >> a.shb) * a.lsb;
    struct Piece {
        v4i32 a[kSteps][kM][2], b[kSteps][2];
        unsigned wa[kM], wb;
    };
    auto load = [&](Piece& p, int step) {
        p.wb = *reinterpret_cast<const unsigned*>(qb + (step & ~3));
#pragma unroll
        for (int f = 0; f < kM; ++f) p.wa[f] = *reinterpret_cast<const unsigned*>(qa[f] + (step & ~3));
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t at = (int64_t)min(step + i, a.steps - 1) * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p.b[i][h] = *reinterpret_cast<const v4i32*>(pb + at + h * 64);
#pragma unroll
                for (int f = 0; f < kM; ++f) p.a[i][f][h] = *reinterpret_cast<const v4i32*>(pa[f] + at + h * 64);
            }
        }
    };
    floatx4 acc[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) acc[m] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Piece& p, int step) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (step + i >= a.steps) break;
            const int sh = 8 * (kSteps == 4 ? i : ((step & 3) + i));
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                if constexpr (!kWide) {
                    acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        __builtin_shufflevector(p.b[i][0], p.b[i][1], 0, 1, 2, 3, 4, 5, 6, 7),
                        __builtin_shufflevector(p.a[i][m][0], p.a[i][m][1], 0, 1, 2, 3, 4, 5, 6, 7), acc[m], 0, 0, 0, (int)(p.wb >> sh), 0,
                        (int)(p.wa[m] >> sh));
                } else {
                    const float sb = power_operand((p.wb >> sh) & 255u), sa = power_operand((p.wa[m] >> sh) & 255u);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            widen(p.b[i][q >> 1][2 * (q & 1)], p.b[i][q >> 1][2 * (q & 1) + 1], sb),
                            widen(p.a[i][m][q >> 1][2 * (q & 1)], p.a[i][m][q >> 1][2 * (q & 1) + 1], sa), acc[m], 0, 0, 0);
                }
            }
        }
    };
    const int jump = share * kSteps;
    int step = turn * kSteps;
    if (step < s1) {
        // Always a next piece (the last one again at the end): a branch around its loads would
        // make the compiler wait for all loads where the two ways meet.
        const int last = s1 - 1 - (s1 - 1 - step) % jump;
        Piece now, next;
        load(now, step);
        while (true) {
            load(next, min(step + jump, last));
            __builtin_amdgcn_sched_barrier(0);
            multiply(now, step);
            if ((step += jump) >= s1) break;
            load(now, min(step + jump, last));
            __builtin_amdgcn_sched_barrier(0);
            multiply(next, step);
            if ((step += jump) >= s1) break;
        }
    }
    // a lane holds columns 4 (l / 16) .. + 3 of row l % 16 of every pair of fragments
#pragma unroll
    for (int m = 0; m < kM; ++m) *reinterpret_cast<floatx4*>(red + ((wave * kM + m) * 64 + lane) * 4) = acc[m];
    __syncthreads();
    // the waves of a group write its result, columns next to each other by threads next to each other
    for (int i = turn * 64 + lane; i < kM * 256; i += share * 64) {
        const int c = i & 15, row = i >> 4;
        const int at = ((row >> 4) * 64 + (c >> 2) * 16 + (row & 15)) * 4 + (c & 3);
        float f = 0.f;
        for (int w = 0; w < share; ++w) f += red[(own * share + w) * kM * 256 + at];
        if (row < a.m && col0 + c < a.n) put1(a, row, col0 + c, f);
    }
}

template <int kM, bool kWide>
__global__ __launch_bounds__(64 * kFewWaves) void k_matmul8_few(Mat8Args a) {
    extern __shared__ float red[];
    matmul8_few<kM, kWide>(a, red);
}

// Few rows of A and many of B: B's bytes bound the product, and a load has to bring whole cache
// lines (8 rows of 128 bytes; 16 rows of 64 bytes straight to registers reach three quarters of
// the rate). A block of eight waves takes 128 rows of B, a wave 16 of them, and streams along k
// through a ring of kStages steps in LDS; A's rows come with them, an eighth by each wave, and are
// what the one barrier a step is for. The powers of the block's part of k are brought to LDS first.
constexpr int kStreamSteps = 128;  // steps of a part, at most

template <int kM>
struct StreamCfg {
    static constexpr int kStages = kM == 1 ? 7 : kM == 2 ? 6 : 5;
    static constexpr int kStage = 128 * 128 + kM * 16 * 128;
    static constexpr int kPowerRow = kStreamSteps + 4;
    static constexpr int kBytes = kStages * kStage + (128 + kM * 16) * kPowerRow;
    static_assert(kBytes <= 160 * 1024, "LDS");
};

template <int N>
__device__ __forceinline__ void wait_loads_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int kM, bool kWide>
__device__ __forceinline__ void matmul8_stream(const Mat8Args& a, uint8_t* smem) {
    typedef StreamCfg<kM> Cfg;
    constexpr int kStages = Cfg::kStages;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = (a.n + 127) / 128, part = blockIdx.x / blocks, col0 = (blockIdx.x - part * blocks) * 128;
    const int fours = (a.steps + 3) >> 2;
    const int s0 = 4 * (int)((int64_t)part * fours / a.splits);
    const int s1 = min(a.steps, 4 * (int)((int64_t)(part + 1) * fours / a.splits));
    const int nk = s1 - s0;
    const __amdgpu_buffer_rsrc_t ra = resource(a.a + (int64_t)s0 * 128);
    const __amdgpu_buffer_rsrc_t rb = resource(a.b + (int64_t)col0 * a.ldb + (int64_t)s0 * 128);
    uint32_t offb[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = wave * 16 + q * 8 + (lane >> 3);
        offb[q] = (uint32_t)min(r, a.n - 1 - col0) * (uint32_t)a.ldb + ((lane & 7) ^ ((r >> 1) & 7)) * 16;
    }
    const int rowa = wave * 2 * kM + (lane >> 3);
    const uint32_t offa = (uint32_t)min(rowa, a.m - 1) * (uint32_t)a.lda + ((lane & 7) ^ ((rowa >> 1) & 7)) * 16;
    auto load = [&](int step) {
        uint8_t* to = smem + step % kStages * Cfg::kStage;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(to + (wave * 2 + q) * 1024), 16, offb[q], step * 128, 0, 0);
        if (lane < 16 * kM)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(to + 128 * 128 + wave * 256 * kM), 16, offa, step * 128, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        if (i < nk) load(i);
    // powers, four steps a dword: B's 128 rows, then A's
    uint8_t* const powers = smem + kStages * Cfg::kStage;
    const int words = (nk + 3) >> 2;
    for (int i = threadIdx.x; i < (128 + kM * 16) * words; i += 512) {
        const int r = i / words, w = i - r * words;
        const uint8_t* from = r < 128 ? a.bs + (int64_t)(min(col0 + r, a.n - 1) >> a.shb) * a.lsb
                                      : a.as + (int64_t)(min(r - 128, a.m - 1) >> a.sha) * a.lsa;
        *reinterpret_cast<unsigned*>(powers + r * Cfg::kPowerRow + w * 4) = *reinterpret_cast<const unsigned*>(from + s0 + w * 4);
    }
    floatx4 acc[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) acc[m] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int lr = lane & 15, lg = lane >> 4, sw = (lr >> 1) & 7;
    const uint8_t *const powb = powers + (wave * 16 + lr) * Cfg::kPowerRow, *const powa = powers + (128 + lr) * Cfg::kPowerRow;
    for (int k = 0; k < nk; ++k) {
        // this wave's loads of the step, then everyone's; the step before has been read by all
        if (k + kStages - 2 < nk) wait_loads_but<3 * (kStages - 2)>();
        else wait_loads();
        wait_lds();
        barrier_no_fence();
        if (k + kStages - 1 < nk) load(k + kStages - 1);
        const uint8_t* st = smem + k % kStages * Cfg::kStage;
        auto frag = [&](int row, int c) { return *reinterpret_cast<const v4i32*>(st + row * 128 + ((c ^ sw) << 4)); };
        v4i32 fb[2], fa[kM][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fb[h] = frag(wave * 16 + lr, lg + 4 * h);
#pragma unroll
            for (int m = 0; m < kM; ++m) fa[m][h] = frag(128 + m * 16 + lr, lg + 4 * h);
        }
        const unsigned eb = powb[k];
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const unsigned ea = powa[m * 16 * Cfg::kPowerRow + k];
            if constexpr (!kWide) {
                acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    __builtin_shufflevector(fb[0], fb[1], 0, 1, 2, 3, 4, 5, 6, 7),
                    __builtin_shufflevector(fa[m][0], fa[m][1], 0, 1, 2, 3, 4, 5, 6, 7), acc[m], 0, 0, 0, (int)eb, 0, (int)ea);
            } else {
                const float sb = power_operand(eb), sa = power_operand(ea);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(fb[q >> 1][2 * (q & 1)], fb[q >> 1][2 * (q & 1) + 1], sb),
                                                                     widen(fa[m][q >> 1][2 * (q & 1)], fa[m][q >> 1][2 * (q & 1) + 1], sa),
                                                                     acc[m], 0, 0, 0);
            }
        }
    }
    Mat8Args o = a;
    if (a.splits > 1) {
        o.c = a.partial + (int64_t)part * a.m * a.n;
        o.ldc = a.n;
        o.dtype = kF32;
        o.accumulate = 0;
    }
#pragma unroll
    for (int m = 0; m < kM; ++m) {
        const int row = m * 16 + lr, col = col0 + wave * 16 + lg * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (row < a.m && col + e < a.n) put1(o, row, col + e, acc[m][e]);
    }
}

template <int kM, bool kWide>
__global__ __launch_bounds__(512) void k_matmul8_stream(Mat8Args a) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[StreamCfg<kM>::kBytes];
    matmul8_stream<kM, kWide>(a, smem);
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

// Few rows of A: where one piece of k is all that a wave of the small form has to do and B is
// 16 MiB at most, its one launch wins ([1, 4096] x [4096, 4096] 9.2 us; 12.5 through LDS with the
// parts' sum), elsewhere B goes through LDS ([8, 5120] x [30720, 5120] 31 us; 44 to 63 us in the
// small form, [16, 5120] x [5120, 5120] 12.9; 19.1).
// Tiles: the cut with the least estimated time. A block's step of 128 takes as many microseconds
// as below with a block a compute unit (two blocks of 128 on one take twice as long each), its
// start and end a few (two blocks of 128 share theirs), and parts of k are written, read and added
// at 8 TB/s (they are still in the caches) in a launch of their own.
// Measured on MI355X, us: [2048, 2048, 2048] 15 as 128-tiles, 27 as 256-tiles; [4096, 4096, 4096] 55
// as 256-tiles, 63 as 128-tiles; [2048, 5120, 20480] 226 and 292; [256, 5120, 5120] 23 in three parts
// of 128-tiles, 31 in one, 30 in six of 256-tiles; [128, 5120, 20480] 40 in six parts of 128-tiles, 141
// in one; fp32 [2048, 2048, 65536] 410 in four parts of 256-tiles, 441 in two of 128-tiles. Of 18 sizes
// timed with every cut the estimate takes the fastest or one within 4%, but for [512, 5120, 5120]: 31 in
// one part of 128-tiles, 29 in two or three.
Mat8Plan plan_matmul8(int64_t m, int64_t n, int64_t k, bool wide) {
    Mat8Plan p{};
    p.splits = 1;
    const int64_t steps = std::max<int64_t>(1, (k + 127) / 128), fours = (steps + 3) / 4;
    if (m <= 64) {
        p.few = m <= 16 ? 1 : m <= 32 ? 2 : 4;
        const int64_t groups = (n + 15) / 16, pieces = (steps + (p.few == 1 ? 3 : 1)) / (p.few == 1 ? 4 : 2);
        p.share = (int)std::max<int64_t>(1, std::min({4096 / groups, int64_t(kFewWaves), pieces}));
        if (n * k > (int64_t(16) << 20) || pieces > p.share) {
            p.stream = 1;
            const int64_t blocks = (n + 127) / 128;
            // a part's powers fit LDS (parts are cut at multiples of four steps)
            p.splits = (int)std::max((steps + kStreamSteps - 4) / (kStreamSteps - 3),
                                     std::min(std::max<int64_t>(1, kUnits / blocks), fours / 2));
        } else {
            p.waves = p.share * (int)std::max<int64_t>(1, std::min<int64_t>(kFewWaves / p.share, groups / kUnits));
        }
    } else {
        double best = 0;
        for (int tile = 128; tile <= 256; tile *= 2) {
            const int64_t tiles = ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
            const double step = tile == 128 ? (wide ? 1.0 : 0.56) : (wide ? 3.1 : 1.45), ends = tile == 128 ? 4 : 8;
            for (int64_t s = 1; s <= std::min<int64_t>(fours, 16) && (s == 1 || tiles * (s - 1) < kUnits); ++s) {
                const double rounds = double((tiles * s + kUnits - 1) / kUnits);
                const double turns = tile == 128 ? double((tiles * s + 2 * kUnits - 1) / (2 * kUnits)) : rounds;
                double t = rounds * double(std::min(steps, 4 * ((fours + s - 1) / s))) * step + turns * ends;
                if (s > 1) t += 5 + double(s) * double(m) * double(n) * 8 / 8e6;
                if (p.tile == 0 || t < best) {
                    best = t;
                    p.tile = tile;
                    p.splits = (int)s;
                }
            }
        }
    }
    if (p.splits > 1) p.partial_bytes = size_t(p.splits) * size_t(m) * size_t(n) * 4;
    return p;
}

template <bool kWide>
hipError_t launch_width(const Mat8Plan& p, const Mat8Args& args, hipStream_t s) {
    Mat8Args a = args;
    if (p.few) {
        if (p.stream) {
            const dim3 grid((unsigned)((a.n + 127) / 128 * a.splits)), block(512);
            if (p.few == 1) hipLaunchKernelGGL((k_matmul8_stream<1, kWide>), grid, block, 0, s, a);
            else if (p.few == 2) hipLaunchKernelGGL((k_matmul8_stream<2, kWide>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((k_matmul8_stream<4, kWide>), grid, block, 0, s, a);
            return hipGetLastError();
        }
        a.share = p.share;
        const int per_block = p.waves / p.share;
        const dim3 grid((unsigned)(((a.n + 15) / 16 + per_block - 1) / per_block)), block(64 * p.waves);
        const size_t lds = size_t(p.waves) * p.few * 1024;
        if (p.few == 1) hipLaunchKernelGGL((k_matmul8_few<1, kWide>), grid, block, lds, s, a);
        else if (p.few == 2) hipLaunchKernelGGL((k_matmul8_few<2, kWide>), grid, block, lds, s, a);
        else hipLaunchKernelGGL((k_matmul8_few<4, kWide>), grid, block, lds, s, a);
        return hipGetLastError();
    }
    const int64_t total = int64_t(a.tiles_m) * a.tiles_n * a.splits;
    const dim3 grid((unsigned)(8 * ((total + 7) / 8)));
    if (p.tile == 256) hipLaunchKernelGGL((k_matmul8<256, kWide>), grid, dim3(64 * Mat8Cfg<256, kWide>::kWaves), 0, s, a);
    else hipLaunchKernelGGL((k_matmul8<128, kWide>), grid, dim3(64 * Mat8Cfg<128, kWide>::kWaves), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_matmul8(const Mat8Plan& p, bool wide, const Mat8Args& a, hipStream_t s) {
    return wide ? launch_width<true>(p, a, s) : launch_width<false>(p, a, s);
}

hipError_t launch_matmul8_join(const Mat8Args& a, hipStream_t s) {
    const int chunks = (a.n + 7) / 8;
    const dim3 grid((unsigned)((int64_t(a.m) * chunks + 255) / 256)), block(256);
    hipLaunchKernelGGL(k_matmul8_join, grid, block, 0, s, a, chunks);
    return hipGetLastError();
}

}  // namespace muon

// ffn_gemm.hpp -- the matrix products of the gated feed-forward block
// (include/gdn_ffn.h), compiled once for each type.
//
// out[m][n] = sum_k Q[m][k] P[n][k], P the first operand of the matrix
// instruction, so that a lane holds four consecutive n of one m (element j of a
// 16 x 16 block: n = 4g + j, m = r of lane 16g + r) and stores them at once.
//
// A workgroup owns a BM x BN tile.  Each step brings 128 bytes of k for its rows
// (64 16-bit or 32 fp32 values) from memory straight into LDS, NST stages in a
// ring, one barrier a step, fragments read half a step ahead.  An operand lies in
// LDS as it lies in memory, k contiguous ("direct") or k strided ("trans"), in
// pieces of 16 bytes whose place in their row is permuted by the row so that
// fragment reads meet no bank twice:
//   direct: [row][8 pieces], piece c at c ^ (row & 7); a fragment is one 16-byte read
//   trans:  [k][row of the tile], piece c at c ^ swz(k); a 16-bit fragment is two
//           transposing 8-byte reads, an fp32 one four 4-byte reads
// The load's LDS side is fixed (lane i at 16 i), so it is the memory side that a
// lane permutes.
//
// Measured (bf16, 16384 tokens, D = 2048, F = 8192; kernel times): gate and up
// 0.86 ms without and 1.00 with what the backward needs, down 0.42 (1300 TFLOP/s), dh
// 0.69, the gradients' three products 2.15 (1280).  With zeros for operands the same code runs
// 12 % faster: it is the chip's power, not the schedule, that bounds the large
// products (the library's, k contiguous, 1240 to 1570 on the same operands, hot and
// cool; 970 to 1030 with k strided).  gate and up and dh add what they
// write and read, 1.3 and 1.6 GB, to their products' time.  Few tokens: the weights'
// reads (1 x 2048 x 8192: gate and up 12.8 us with weights that the call before left in cache, 16.6 to
// 18.2 with weights from memory, 3.7 TB/s).
#pragma once
#include "ffn_launch.hpp"
#include "gdr_device.hpp"
#include "layer_rows.hpp"
#include "../../include/gdn_ffn.h"

namespace ffn {
using gdr::bf16;
using gdr::f16;
using gdr::f32x4;
using gdr::i16x4;
using gdr::i16x8;

template <class E> struct Type {
    static constexpr int CE = 16 / sizeof(E);    // elements in a piece of 16 bytes
    static constexpr int KE = 128 / sizeof(E);   // k in a step
    using frag = typename gdr::Mma<E>::frag;
};
template <> struct Type<float> {
    static constexpr int CE = 4, KE = 32;
    using frag = f32x4;
};

// Two fragments of a step cover its k: 32 16-bit values each (k = 32 s + 8 g + i), or 16 fp32
// values each (k = 16 s + 4 g + j, element j in the j-th of four products).
template <class E> __device__ __forceinline__ f32x4 mma(typename Type<E>::frag a, typename Type<E>::frag b, f32x4 c) {
    if constexpr (sizeof(E) == 2) {
        return gdr::Mma<E>::run(a, b, c);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) c = gdr::Mma<float>::run(a[j], b[j], c);
        return c;
    }
}

// The permutation of pieces of a "trans" row (see above); NC pieces a row.
template <class E, int NC> __device__ __forceinline__ int swz(int k) {
    const int x = sizeof(E) == 2 ? (2 * (k & 3)) ^ (8 * ((k >> 3) & 1)) : 4 * ((k >> 2) & 3);
    return x & (NC - 1);
}

// 16 bytes of each lane from base + off to LDS at lds + 16 lane, the place in m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is named as overwritten so that no value of the compiler's is kept in it
__device__ __forceinline__ void load_to_lds(uint32_t lds, const char* base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N> __device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory"); }

// One operand of a tile.  ROWS: BM or BN.  PAIR: rows of two matrices in turn, 16 of each.
template <class E, int ROWS, int NW, bool TRANS, bool PAIR> struct Operand {
    static constexpr int CE = Type<E>::CE, KE = Type<E>::KE;
    static constexpr int UNITS = ROWS / 8, PER = (UNITS + NW - 1) / NW;   // KiB of a stage, of a wave's share
    static constexpr int NC = TRANS ? ROWS * (int)sizeof(E) / 16 : 8;     // pieces in a row of LDS
    static constexpr int BYTES = ROWS * 128;
    static_assert(UNITS % NW == 0, "waves load alike");

    uint32_t off[PER];      // of a lane's pieces from the base, for whole steps

    __device__ __forceinline__ static int row_in(int u, int lane) { return (u * 64 + lane) / NC; }
    __device__ __forceinline__ static int piece(int u, int lane) {
        const int row = row_in(u, lane), slot = (u * 64 + lane) % NC;
        return slot ^ (TRANS ? swz<E, NC>(row) : row & 7);
    }
    // first: the tile's first row (of each matrix of a pair); count: rows that exist
    __device__ __forceinline__ void init(int first, int count, int64_t ld, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int u = wave + NW * i;
            if constexpr (TRANS) {
                int c = first + piece(u, lane) * CE;   // rows past the end: any that exist, their sums are not stored
                c = c < count - CE ? c : count - CE;
                off[i] = (uint32_t)((row_in(u, lane) * ld + c) * sizeof(E));
            } else {
                int r = PAIR ? (u / 4) * 16 + (u % 2) * 8 + lane / 8 : row_in(u, lane);
                r = first + r < count ? r : count - 1 - first;
                off[i] = (uint32_t)((r * ld + piece(u, lane) * CE) * sizeof(E));
            }
        }
    }
    // Loads step kt (k from kt KE on) into LDS at `lds`; p0, p1: the matrices, from row `first` on if direct.
    // WHOLE: the step is not short.
    template <bool WHOLE>
    __device__ __forceinline__ void load(uint32_t lds, const char* p0, const char* p1, int psplit, int64_t ld, int kt,
                                         int K, int wave, int lane) const {
        const int left = K - kt * KE;   // a last step may be short: k past the end are read at the last k
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int u = wave + NW * i;
            const char* base;
            uint32_t o = off[i];
            if constexpr (TRANS) {
                const int k0 = kt * KE + u * 64 / NC;
                const bool second = p1 && k0 >= psplit;   // uniform: a unit's rows are on one side
                base = (second ? p1 : p0) + (int64_t)(second ? kt * KE - psplit : kt * KE) * ld * (int64_t)sizeof(E);
                if (!WHOLE && left < KE) {
                    const int over = row_in(u, lane) - (left - 1);
                    if (over > 0) o -= (uint32_t)(over * ld * sizeof(E));
                }
            } else {
                base = (PAIR && (u / 2) % 2 ? p1 : p0) + (int64_t)kt * 128;
                if (!WHOLE && left < KE) {
                    const int over = (piece(u, lane) + 1) * CE - left;
                    if (over > 0) o -= (uint32_t)(over * sizeof(E));
                }
            }
            load_to_lds(lds + u * 1024, base, o);
        }
    }
    // Zero for the k past the end in the pieces that this lane loaded.
    __device__ __forceinline__ void clear_tail(char* lds, int left, int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int u = wave + NW * i;
            const bool past = TRANS ? row_in(u, lane) >= left : piece(u, lane) * CE >= left;
            if (past) *(f32x4*)(lds + u * 1024 + lane * 16) = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    // Fragment s of the 16 rows from w0 + 16 i on.
    __device__ __forceinline__ static typename Type<E>::frag frag(const char* lds, int w0, int i, int s, int lane) {
        const int r = lane & 15, g = lane >> 4;
        using F = typename Type<E>::frag;
        if constexpr (!TRANS) {
            return *(const F*)(lds + (w0 + 16 * i + r) * 128 + ((4 * s + g) ^ (r & 7)) * 16);
        } else if constexpr (sizeof(E) == 2) {
            const int x = swz<E, NC>(8 * g + (r >> 2));
            const char* p = lds + (32 * s + 8 * g + (r >> 2)) * (ROWS * 2) +
                            (((w0 + 16 * i) / 8 + ((r >> 1) & 1)) ^ x) * 16 + (r & 1) * 8;
            const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, p));
            const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, p + 4 * ROWS * 2));
            const i16x8 c = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            return __builtin_bit_cast(F, c);
        } else {
            const char* p = lds + (16 * s + 4 * g) * (ROWS * 4) +
                            (((w0 + 16 * i) / 4 + (r >> 2)) ^ swz<E, NC>(4 * g)) * 16 + (r & 3) * 4;
            F f;
#pragma unroll
            for (int j = 0; j < 4; j++) f[j] = *(const float*)(p + j * ROWS * 4);
            return f;
        }
    }
};

// ----------------------------------------------------------------- epilogues
// sigmoid_f: layer_rows.hpp.
// gelu: x Phi(x), Phi(x) = erfc(-x / sqrt 2) / 2.  For z = |x| / sqrt 2, erfc(z) = exp(-z^2) t Q(t) with
// t = 1 / (1 + z / 2) and a polynomial Q, fitted by least squares on Chebyshev points, weighted towards the
// largest error: 8e-8 of the value at most for z < 9.5, past which exp(-z^2) is zero.  The exponential is the one
// that the slope takes.  In units of 2^-24, with one in the last place (2) each for rcp and exp2: t is off by 3 of itself near
// zero, where t Q(t) takes that 2.3 fold, the polynomial's nine roundings by 2.9, so that Phi is off by 8 at most; below zero
// by 16 + 1.2 x^2 of itself, the second term from the exponent's roundings.
__device__ __forceinline__ float gauss(float x, float& e) {   // Phi(x), exp(-x^2 / 2)
    constexpr float Q[9] = {-0.0588914342f, 0.283705056f, -0.485389888f, 0.275984913f, -0.0251820963f, 0.202071592f, 0.243260592f, 0.28235355f, 0.282087684f};
    const float t = __builtin_amdgcn_rcpf(1.f + fabsf(x) * 0.35355338f);
    float q = Q[0];
#pragma unroll
    for (int i = 1; i < 9; i++) q = __builtin_fmaf(q, t, Q[i]);
    e = __builtin_amdgcn_exp2f(x * x * -0.72134752f);
    const float tail = 0.5f * t * q * e;
    return x > 0.f ? 1.f - tail : tail;
}
template <int ACT> __device__ __forceinline__ float act_f(float x) {
    if constexpr (ACT == GDN_FFN_GELU) {
        float e;
        return x * gauss(x, e);
    }
    const float s = layer::sigmoid_f(x);
    return ACT == GDN_FFN_SILU ? x * s : s;
}
// act(x) and its slope.  With e = exp(-x), s = sigmoid(x) = 1 / (1 + e) and 1 - s = e s,
// which keeps its digits where s is close to 1.  Where e is beyond 2^126, and may be infinite, s is zero as in the
// forward (held above zero, x s would grow again for gates far below zero) and 1 - s is 1; comparisons, so that a NaN
// stays one.
template <int ACT> __device__ __forceinline__ void act_slope(float x, float& a, float& d) {
    if constexpr (ACT == GDN_FFN_GELU) {
        float e;
        const float phi = gauss(x, e);
        a = x * phi;
        d = phi + x * 0.39894228f * e;
    } else {
        const float e = layer::exp_neg(x), s = e > 0x1p126f ? 0.f : __builtin_amdgcn_rcpf(1.f + e), t = e > 0x1p126f ? 1.f : e * s;
        a = ACT == GDN_FFN_SILU ? x * s : s;
        d = ACT == GDN_FFN_SILU ? s * (1.f + x * t) : s * t;
    }
}

// Four consecutive elements of a row, those of them before `end`.
template <class E> __device__ __forceinline__ void store4(E* row, int64_t n, int64_t end, f32x4 v) {
    typedef typename layer::VecU<E, 4>::t V;
    if (n + 4 <= end) {
        V t;
#pragma unroll
        for (int e = 0; e < 4; e++) t[e] = (E)v[e];
        *(V*)(row + n) = t;
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (n + e < end) row[n + e] = (E)v[e];
    }
}
// Gate and up of four columns as kept by the forward.  Without branches, so that several stay on their way.
struct Kept {
    f32x4 g, u;
    __device__ __forceinline__ void load(const GemmArgs& a, int m, int n) {
        const float* row = a.gu + (int64_t)m * 2 * a.N + (n < a.N ? n : 0);
        g = *(const f32x4*)row, u = *(const f32x4*)(row + a.N);
    }
};

// Orders a wave's own accesses to LDS (they are carried out in their order).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// What becomes of four sums (n .. n+3 of row m): v of the product, w of the pair's second matrix.
template <class E, int KIND, int ACT>
__device__ __forceinline__ void finish(const GemmArgs& a, int m, int n, f32x4 v, f32x4 w, const Kept& kept) {
    if constexpr (KIND == GATE_UP) {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (n + e >= a.rowsP) v[e] = w[e] = 0.f;
        if (a.gu) {   // kept in fp32: rounded to the type they would add as much error to the gradients as the operands do
            float* row = a.gu + (int64_t)m * 2 * a.N + n;
            *(f32x4*)row = v, *(f32x4*)(row + a.N) = w;
        }
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; e++) h[e] = act_f<ACT>(v[e]) * w[e];
        store4<E>((E*)a.h + (int64_t)m * a.N, n, a.N, h);
    } else if constexpr (KIND == DH) {
        f32x4 dg, du;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if (n + e >= a.rowsP) v[e] = 0.f;   // a padded column's sum has an infinite dy times zero
            float act, slope;
            act_slope<ACT>(kept.g[e], act, slope);
            dg[e] = v[e] * kept.u[e] * slope;
            du[e] = v[e] * act;
        }
        E* d = (E*)a.dgu + (int64_t)m * 2 * a.N;
        store4<E>(d, n, a.N, dg);
        store4<E>(d + a.N, n, a.N, du);
    } else {
        const bool second = m >= a.osplit;
        if (second) m -= a.osplit;
        if (m < a.rows_out) store4<E>((E*)(second ? a.out1 : a.out0) + m * a.ldo, n, a.cols_out, v);
    }
}

// f(act): what the epilogue's code goes by, uniform
template <int KIND, class F> __device__ __forceinline__ void by_act(const GemmArgs& a, F&& f) {
    using std::integral_constant;
    if constexpr (KIND != GATE_UP && KIND != DH) f(integral_constant<int, 0>{});
    else if (a.act == GDN_FFN_SILU) f(integral_constant<int, GDN_FFN_SILU>{});
    else if (a.act == GDN_FFN_GELU) f(integral_constant<int, GDN_FFN_GELU>{});
    else f(integral_constant<int, GDN_FFN_SIGMOID>{});
}

// Workgroup `block` of a product.
template <class E, int KIND, int BM, int BN, int WM, int WN, int NST>
__device__ __forceinline__ void gemm_tile(const GemmArgs& a, int block, char* smem) {
    constexpr bool PAIR = KIND == GATE_UP, QT = KIND == DW, PT = KIND == DH || KIND == DX || KIND == DW;
    constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16, KE = Type<E>::KE;
    constexpr int BT = PAIR ? BN / 2 : BN;      // columns of a tile
    using Q = Operand<E, BM, NW, QT, false>;
    using P = Operand<E, BN, NW, PT, PAIR>;
    constexpr int STAGE = Q::BYTES + P::BYTES, LOADS = Q::PER + P::PER;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // Workgroups go to the chip's 8 parts in turn; each part takes a run of tiles, and within
    // it `rows` rows of tiles at a time, so that its L2 serves an operand's tile to several.  Rows of 256: three where
    // k is short and four beyond, a rule by measurement (an odd number spreads rows whose pitch is a power of two over
    // the memory's channels; three rows of Q are 3 MB of the part's 4 at 4 KB of k).  bf16, a forward that
    // keeps its gate and up rows, us, with 2, 3, 4, 6 and 8 rows: 16384 x 512 x 8192 634, 570, 664, 606, 745; 1024 879,
    // 835, 917, 875, 981; 2048 1448, 1427, 1505, 1455, 1532; 2560 1870, 1813, 1873, 1881, 1906; 8192 x 4096 x 12288 1964, 1981,
    // 1910, 1968, 1922; 8192 x 8192 x 4096 1322, 1271, 1244, 1260, 1239.  Backward with three and with four
    // everywhere (dh goes by D; the gradients have 2 F and the tokens for k, which is four in large sizes): 16384 x 512 x 8192
    // 1016, 1058; 1024 1602, 1618; 2048 2842, 2793; 2560 3861, 3864; 8192 x 4096 x 12288 4064, 3935.
    const int tiles = a.tilesM * a.tilesN, total = tiles * a.splits;
    const int xcd = block & 7, per = total >> 3, rem = total & 7;
    int id = xcd * per + (xcd < rem ? xcd : rem) + (block >> 3);
    const int split = id / tiles;
    id -= split * tiles;
    const int rows = BM < 256 ? 8 : a.K * (int)sizeof(E) <= 4096 ? 3 : 4;
    const int group = id / (rows * a.tilesN), in = id - group * rows * a.tilesN;
    const int high = a.tilesM - group * rows < rows ? a.tilesM - group * rows : rows;
    const int m0 = (group * rows + in % high) * BM, n0 = in / high * BT;

    const int all = (a.K + KE - 1) / KE, k0 = split * a.steps, k1 = k0 + a.steps < all ? k0 + a.steps : all;
    Q q;
    P p;
    q.init(m0, a.M, a.ldq, wave, lane);
    p.init(n0, PT ? a.N : a.rowsP, a.ldp, wave, lane);
    const char* qb = (const char*)a.q + (QT ? 0 : (int64_t)m0 * a.ldq * (int64_t)sizeof(E));
    const char* pb0 = (const char*)a.p0 + (PT ? 0 : (int64_t)n0 * a.ldp * (int64_t)sizeof(E));
    const char* pb1 = a.p1 ? (const char*)a.p1 + (PT ? 0 : (int64_t)n0 * a.ldp * (int64_t)sizeof(E)) : nullptr;
    const uint32_t lds0 = (uint32_t)(uintptr_t)LDS_PTR(char, smem);
    auto load = [&](auto whole, int kt, int stage) {
        constexpr bool W = decltype(whole)::value;
        q.template load<W>(lds0 + stage * STAGE, qb, nullptr, 0, a.ldq, kt, a.K, wave, lane);
        p.template load<W>(lds0 + stage * STAGE + Q::BYTES, pb0, pb1, a.psplit, a.ldp, kt, a.K, wave, lane);
    };

    f32x4 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; j++)
#pragma unroll
        for (int i = 0; i < TM; i++) acc[j][i] = gdr::zero4();

    using Frag = typename Type<E>::frag;
    Frag fp[2][TN], fq[2][TM];   // of a step's halves
    auto read = [&](int s, int stage) {
        const char* cur = smem + stage * STAGE;
#pragma unroll
        for (int i = 0; i < TM; i++) fq[s][i] = Q::frag(cur, wm * TM * 16, i, s, lane);
#pragma unroll
        for (int j = 0; j < TN; j++) fp[s][j] = P::frag(cur + Q::BYTES, wn * TN * 16, j, s, lane);
    };
    auto multiply = [&](int s) {
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int i = 0; i < TM; i++) acc[j][i] = mma<E>(fp[s][j], fq[s][i], acc[j][i]);
    };
    // Step kt is in LDS once every wave is here; `last`: the latest step on its way.
    auto land = [&](int kt, int stage, int last) {
        if (kt + NST - 2 < last) wait_loads<(NST - 1) * LOADS>();
        else if (NST > 2 && kt + NST - 2 == last) wait_loads<(NST - 2) * LOADS>();
        else wait_loads<0>();
        if (a.K - kt * KE < KE) {
            q.clear_tail(smem + stage * STAGE, a.K - kt * KE, wave, lane);
            p.clear_tail(smem + stage * STAGE + Q::BYTES, a.K - kt * KE, wave, lane);
        }
        gdr::lds_barrier();
    };

    // One product after each read while there are reads, for the scheduler: neither unit waits for the
    // other (16384 x 2048 x 8192 bf16, all products: 4690 -> 4540 us).
    auto mingle = [] {
        constexpr int TR = sizeof(E) == 2 ? 2 : 4, DS = TM * (QT ? TR : 1) + TN * (PT ? TR : 1);
#pragma unroll
        for (int i = 0; i < DS; i++) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix instruction
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 256, 0);
    };
    // The second half's fragments are read while the first half's products run, and the next
    // step's first half's while the second's do; a stage is free once the second half is read.
#pragma unroll
    for (int t = 0; t < NST; t++)
        if (k0 + t < k1) load(std::false_type{}, k0 + t, t);
    int stage = 0, kt = k0;
    if (k0 < k1) {
        land(k0, 0, k0 + NST - 1 < k1 ? k0 + NST - 1 : k1 - 1);
        read(0, 0);
        for (; kt < k1 - 1 - NST; kt++) {   // the step that is loaded is not the last
            const int next = stage + 1 == NST ? 0 : stage + 1;
            read(1, stage);
            multiply(0);
            mingle();
            wait_loads<(NST - 2) * LOADS>();
            gdr::lds_barrier();
            load(std::true_type{}, kt + NST, stage);
            read(0, next);
            multiply(1);
            mingle();
            stage = next;
        }
        for (; kt < k1 - 1; kt++) {
            const int next = stage + 1 == NST ? 0 : stage + 1;
            read(1, stage);
            multiply(0);
            land(kt + 1, next, kt + NST - 1 < k1 ? kt + NST - 1 : k1 - 1);
            if (kt + NST < k1) load(std::false_type{}, kt + NST, stage);
            read(0, next);
            multiply(1);
            stage = next;
        }
        read(1, stage);
        multiply(0);
        multiply(1);
    }

    // The sums go out through LDS, up to 64 rows of a wave at a time, so that lanes side by side hold
    // columns side by side: whole lines are written, and what the epilogue reads comes in whole lines,
    // DEPTH passes ahead.  Quad q of a row lies at q ^ row.
    constexpr int STEP = PAIR ? 2 : 1, COLS = 16 * TN / STEP, QUADS = 4 * TN;
    constexpr int LPR = COLS / 4, RPP = 64 / LPR;                      // lanes of a row, rows of a pass
    constexpr int CH = TM < 4 ? TM : 4, PC = 16 * CH / RPP, DEPTH = PC < 4 ? PC : BM * BN == 128 * 128 && NST == 2 ? 2 : 4;   // 2: registers for two workgroups
    static_assert(NW * 16 * CH * QUADS * 16 <= NST * STAGE && TM % CH == 0 && PC % DEPTH == 0, "fits the stages");
    const int r = lane & 15, g = lane >> 4;
    char* mine = smem + wave * 16 * CH * QUADS * 16;
    const int row0 = lane / LPR, col = lane % LPR * 4, n = n0 + wn * COLS + col, m1 = m0 + wm * TM * 16 + row0;
    auto quad = [&](int row, int q) { return (f32x4*)(mine + row * QUADS * 16 + (q ^ (row & (QUADS - 1))) * 16); };
    auto spread = [&](auto I) {
        constexpr int c = decltype(I)::value * CH;
#pragma unroll
        for (int i = 0; i < CH; i++)
#pragma unroll
            for (int j = 0; j < TN; j++)
                *quad(16 * i + r, PAIR ? j % 2 * (QUADS / 2) + j / 2 * 4 + g : j * 4 + g) = acc[j][c + i];
        wave_sync();
    };
    auto chunks = [&](auto&& f) {
        f(std::integral_constant<int, 0>{});
        if constexpr (TM > CH) f(std::integral_constant<int, 1>{});
        static_assert(TM <= 2 * CH, "two chunks at most");
    };
    if (a.splits > 1) {
        gdr::lds_barrier();   // the stages are no longer read
        chunks([&](auto I) {
            spread(I);
            for (int p = 0; p < PC; p++) {
                const int row = p * RPP + row0, m = m1 + decltype(I)::value * CH * 16 + p * RPP;
                const f32x4 v = *quad(row, col / 4), w = *quad(row, col / 4 + (PAIR ? QUADS / 2 : 0));
                if (m >= a.M || n >= a.N) continue;
                float* part = a.part + ((int64_t)split * a.M + m) * STEP * a.N + n;
                *(f32x4*)part = v;
                if constexpr (PAIR) *(f32x4*)(part + a.N) = w;
            }
            wave_sync();
        });
        return;
    }
    by_act<KIND>(a, [&](auto A) {
        constexpr int ACT = decltype(A)::value;
        Kept kept[DEPTH];
        auto fetch = [&](Kept& k, int p) {
            if constexpr (KIND == DH) {
                const int m = m1 + p * RPP;
                k.load(a, m < a.M ? m : a.M - 1, n);
            }
        };
#pragma unroll
        for (int d = 0; d < DEPTH; d++) fetch(kept[d], d);
        gdr::lds_barrier();   // the stages are no longer read
        chunks([&](auto I) {
            spread(I);
#pragma unroll 1
            for (int p = 0; p < PC; p += DEPTH)
#pragma unroll
                for (int d = 0; d < DEPTH; d++) {
                    const int at = decltype(I)::value * PC + p + d, row = (p + d) * RPP + row0, m = m1 + at * RPP;
                    const f32x4 v = *quad(row, col / 4), w = *quad(row, col / 4 + (PAIR ? QUADS / 2 : 0));
                    if (m < a.M && n < a.N) finish<E, KIND, ACT>(a, m, n, v, w, kept[d]);
                    fetch(kept[d], at + DEPTH);
                }
            wave_sync();
        });
    });
}

// Registers for as many workgroups as a CU's 160 KB of LDS hold.
#define FFN_BOUNDS __launch_bounds__(64 * WM * WN, 163840 / ((BM + BN) * 128 * NST) * WM * WN / 4)
template <class E, int KIND, int BM, int BN, int WM, int WN, int NST> __global__ FFN_BOUNDS void ffn_gemm_kernel(GemmArgs a) {
    __shared__ __attribute__((aligned(1024))) char smem[NST * (BM + BN) * 128];
    gemm_tile<E, KIND, BM, BN, WM, WN, NST>(a, blockIdx.x, smem);
}
// The gradients' products in one launch, one after another in the grid: alone each of them fills the chip badly where
// there are few tokens.  Each begins at a multiple of 8, so that its tiles keep to their parts of the chip.
template <class E, int BM, int BN, int WM, int WN, int NST> __global__ FFN_BOUNDS void ffn_grads_kernel(GradArgs p) {
    __shared__ __attribute__((aligned(1024))) char smem[NST * (BM + BN) * 128];
    int block = blockIdx.x;
    GemmArgs a = p.g[0];
    bool dx = p.dx[0];
    if (block >= p.start[1]) a = p.g[1], dx = p.dx[1];
    if (block >= p.start[2]) a = p.g[2], dx = p.dx[2];
    block -= block >= p.start[2] ? p.start[2] : block >= p.start[1] ? p.start[1] : 0;
    if (block >= a.tilesM * a.tilesN * a.splits) return;
    if (dx) gemm_tile<E, DX, BM, BN, WM, WN, NST>(a, block, smem);
    else gemm_tile<E, DW, BM, BN, WM, WN, NST>(a, block, smem);
}

// The splits' sums in their order, and what becomes of them: four columns a lane, eight splits on their way at a time,
// workgroups of one wave, since a token's sums are few (8 splits of 1 x 2048 with all of its forward, us: 23.4 with four
// at a time in workgroups of 256, 22.4 so; 20 x 1024 x 8192 18.1 and 16.3).
constexpr int JOIN_THREADS = 64;
template <class E, int KIND> __device__ __forceinline__ void join_splits(const GemmArgs& a) {
    constexpr int STEP = KIND == GATE_UP ? 2 : 1;
    const int quads = a.N / 4;
    const int64_t total = (int64_t)a.M * quads, plane = (int64_t)a.M * STEP * a.N;
    for (int64_t id = (int64_t)blockIdx.x * JOIN_THREADS + threadIdx.x; id < total; id += (int64_t)gridDim.x * JOIN_THREADS) {
        const int m = total >> 32 ? (int)(id / quads) : (int)((uint32_t)id / (uint32_t)quads), n = 4 * (int)(id - (int64_t)m * quads);
        const float* p = a.part + (int64_t)m * STEP * a.N + n;
        f32x4 v = *(const f32x4*)p, w = *(const f32x4*)(p + (STEP - 1) * a.N);
        constexpr int AT = 8;
        for (int s = 1; s < a.splits; s += AT) {
            f32x4 x[AT], y[AT];
#pragma unroll
            for (int i = 0; i < AT; i++) {
                if (s + i >= a.splits) break;
                const float* at = p + (s + i) * plane;
                x[i] = *(const f32x4*)at;
                if constexpr (STEP == 2) y[i] = *(const f32x4*)(at + a.N);
            }
#pragma unroll
            for (int i = 0; i < AT; i++) {
                if (s + i >= a.splits) break;
                v += x[i];
                if constexpr (STEP == 2) w += y[i];
            }
        }
        by_act<KIND>(a, [&](auto A) {
            Kept kept;
            if constexpr (KIND == DH) kept.load(a, m, n);
            finish<E, KIND, decltype(A)::value>(a, m, n, v, w, kept);
        });
    }
}

template <class E, int KIND> __global__ __launch_bounds__(JOIN_THREADS) void ffn_join_kernel(GemmArgs a) { join_splits<E, KIND>(a); }
template <class E> __global__ __launch_bounds__(JOIN_THREADS) void ffn_join_grads_kernel(GradArgs p) {   // dx and dw end alike
    GemmArgs a = p.g[0];
    if (blockIdx.y == 1) a = p.g[1];
    if (blockIdx.y == 2) a = p.g[2];
    if (a.splits > 1) join_splits<E, DX>(a);
}

inline unsigned join_blocks(const GemmArgs& a) {
    const int64_t n = ((int64_t)a.M * (a.N / 4) + JOIN_THREADS - 1) / JOIN_THREADS;
    return (unsigned)(n < 16384 ? n : 16384);
}
template <class E, int BM, int BN, int WM, int WN, int NST> hipError_t run_grads_shape(const GradArgs& p, hipStream_t s) {
    hipLaunchKernelGGL((ffn_grads_kernel<E, BM, BN, WM, WN, NST>), dim3((unsigned)p.start[3]), dim3(64 * WM * WN), 0, s, p);
    unsigned most = 0;
    for (const GemmArgs& a : p.g)
        if (a.splits > 1 && join_blocks(a) > most) most = join_blocks(a);
    if (most) hipLaunchKernelGGL(ffn_join_grads_kernel<E>, dim3(most, 3), dim3(JOIN_THREADS), 0, s, p);
    return hipGetLastError();
}
template <class E, int KIND, int BM, int BN, int WM, int WN, int NST>
hipError_t run_shape(const GemmArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((ffn_gemm_kernel<E, KIND, BM, BN, WM, WN, NST>), dim3((unsigned)(a.tilesM * a.tilesN * a.splits)),
                       dim3(64 * WM * WN), 0, s, a);
    if (a.splits > 1) hipLaunchKernelGGL((ffn_join_kernel<E, KIND>), dim3(join_blocks(a)), dim3(JOIN_THREADS), 0, s, a);
    return hipGetLastError();
}

template <class E, int KIND> hipError_t run_kind(const GemmArgs& a, int cfg, hipStream_t s) {
    if constexpr (sizeof(E) == 2) {
        if (cfg == BIG) return run_shape<E, KIND, 256, 256, 2, 4, 2>(a, s);
        if (cfg == WIDE) return run_shape<E, KIND, 256, 128, 4, 2, 3>(a, s);
        if (cfg == DEEP) return run_shape<E, KIND, 128, 128, 2, 4, 4>(a, s);
    }
    if constexpr (KIND == GATE_UP || KIND == DOWN) {
        if (cfg == THIN) return run_shape<E, KIND, 32, 64, 2, 2, 6>(a, s);
    }
    switch (cfg) {
        case MIDDLE: return run_shape<E, KIND, 128, 128, 2, 4, 2>(a, s);
        case LOW: return run_shape<E, KIND, 64, 128, 2, 4, 3>(a, s);
        default: return run_shape<E, KIND, 64, 64, 2, 2, 4>(a, s);
    }
}
template <class E> hipError_t run_gemm(Kind kind, const GemmArgs& a, int cfg, hipStream_t s) {
    switch (kind) {
        case GATE_UP: return run_kind<E, GATE_UP>(a, cfg, s);
        case DOWN: return run_kind<E, DOWN>(a, cfg, s);
        default: return run_kind<E, DH>(a, cfg, s);
    }
}
template <class E> hipError_t run_grads(const GradArgs& p, int cfg, hipStream_t s) {
    if constexpr (sizeof(E) == 2) {
        if (cfg == BIG) return run_grads_shape<E, 256, 256, 2, 4, 2>(p, s);
        if (cfg == WIDE) return run_grads_shape<E, 256, 128, 4, 2, 3>(p, s);
        return run_grads_shape<E, 128, 128, 2, 4, 2>(p, s);
    } else {
        return cfg == MIDDLE ? run_grads_shape<E, 128, 128, 2, 4, 2>(p, s) : run_grads_shape<E, 64, 64, 2, 2, 4>(p, s);
    }
}

}  // namespace ffn

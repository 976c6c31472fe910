// layer_rows.hpp -- device and host pieces shared by the two norms
// (layer_gated_norm.hip, layer_add_norm.hip).
//
// A row of D elements is held by TPR lanes (a part of a wave, a wave, or
// several waves of one workgroup), NV vectors of VEC elements each: 16 bytes of
// the widest type per load.  All arithmetic is fp32; outputs are rounded once.
#pragma once
#include <type_traits>

#include "../../include/gdn_layer.h"
#include "gdr_device.hpp"
#include "layer_launch.hpp"

namespace layer {
using gdr::bf16;
using gdr::f16;

// N elements at any element-aligned address: the vector type's alignment is the
// element's, so rows of odd length keep wide loads (unaligned global accesses
// are native on gfx950).
template <class E, int N> struct VecU { typedef E t __attribute__((ext_vector_type(N), aligned(sizeof(E)))); };

template <class E, int VEC> struct Raw {
    typename VecU<E, VEC>::t v;   // as loaded; widened to fp32 where it is used
};

// 16 bytes moved down by `bytes` (uniform, below 16), zeros above.
template <class V> __device__ __forceinline__ V move_down(V v, int bytes) {
    static_assert(sizeof(V) == 16 || sizeof(V) == 8, "a vector load");
    typedef unsigned long long u64;
    u64 lo, hi = 0;
    if constexpr (sizeof(V) == 16) {
        u64 u[2];
        __builtin_memcpy(u, &v, 16);
        lo = u[0], hi = u[1];
        if (bytes >= 8) lo = hi, hi = 0, bytes -= 8;
        if (bytes > 0) lo = lo >> 8 * bytes | hi << (64 - 8 * bytes), hi >>= 8 * bytes;
        u[0] = lo, u[1] = hi;
        __builtin_memcpy(&v, u, 16);
    } else {
        __builtin_memcpy(&lo, &v, 8);
        lo >>= 8 * bytes;
        __builtin_memcpy(&v, &lo, 8);
    }
    return v;
}

// A lane's i-th VEC elements of a row of a stream; columns past D read as zero.
// The vector that a row ends in is read from the row's last VEC elements and
// moved down (one load for all lanes; element by element only where D < VEC).  The
// elements before the vector's own are another lane's, of another wave perhaps, which
// may be writing them already where an output replaces this input: whatever is read
// there, the move drops it.  Its own elements only this lane writes, after their use.
// Non-temporal: every element is read once in the launch.
template <int TPR, class E, int VEC>
__device__ __forceinline__ void load_raw(Raw<E, VEC>& r, const E* row, int i, int lane, int D) {
    using V = typename VecU<E, VEC>::t;
    const int rem = D % VEC, c = (i * TPR + lane) * VEC;
    if (rem == 0 || D > VEC) {
        const bool tail = c + VEC > D && c < D;
        V v;
#pragma unroll
        for (int e = 0; e < VEC; e++) v[e] = (E)0.f;
        if (c < D) v = __builtin_nontemporal_load((const V*)(row + (tail ? D - VEC : c)));
        if (rem != 0 && (i + 1) * TPR * VEC > D) {   // the row ends here, in one of the lanes
            const V m = move_down<V>(v, (VEC - rem) * (int)sizeof(E));
            v = tail ? m : v;
        }
        r.v = v;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e++) r.v[e] = c + e < D ? row[c + e] : (E)0.f;
    }
}
// The same of a weight, which every row reads (non-temporal reads of those doubled
// the add norm's backward).
template <int VEC>
__device__ __forceinline__ void load_weight(float (&w)[VEC], const float* p, int c, int D) {
#pragma unroll
    for (int e = 0; e < VEC; e++) w[e] = 0.f;
    if (c + VEC <= D) {
        const auto t = *(const typename VecU<float, VEC>::t*)(p + c);
#pragma unroll
        for (int e = 0; e < VEC; e++) w[e] = t[e];
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e++)
            if (c + e < D) w[e] = p[c + e];
    }
}
template <int VEC, int TPR, int NV>
__device__ __forceinline__ void load_weights(float (&w)[NV][VEC], const float* p, int lane, int D) {
#pragma unroll
    for (int i = 0; i < NV; i++) load_weight<VEC>(w[i], p, (i * TPR + lane) * VEC, D);
}
// N elements of x, from element O on, to p + O.
template <int O, int N, class E, int VEC> __device__ __forceinline__ void store_part(E* p, const float (&x)[VEC]) {
    if constexpr (O + N <= VEC) {
        typename VecU<E, N>::t t;
#pragma unroll
        for (int e = 0; e < N; e++) t[e] = (E)x[O + e];
        __builtin_nontemporal_store(t, (typename VecU<E, N>::t*)(p + O));
    }
}
// VEC elements of a row from column c, those before D; the vector that an odd row
// ends in in pieces of 4, 2 and 1.
template <class E, int VEC>
__device__ __forceinline__ void store_vec(E* row, int c, int D, const float (&x)[VEC]) {
    E* p = row + c;
    if (c + VEC <= D) {
        store_part<0, VEC>(p, x);
    } else if (c < D) {
        switch (D % VEC) {   // uniform
            case 1: store_part<0, 1>(p, x); break;
            case 2: store_part<0, 2>(p, x); break;
            case 3: store_part<0, 2>(p, x); store_part<2, 1>(p, x); break;
            case 4: store_part<0, 4>(p, x); break;
            case 5: store_part<0, 4>(p, x); store_part<4, 1>(p, x); break;
            case 6: store_part<0, 4>(p, x); store_part<4, 2>(p, x); break;
            case 7: store_part<0, 4>(p, x); store_part<4, 2>(p, x); store_part<6, 1>(p, x); break;
        }
    }
}

// exp(-z) with its one rounding of the exponent (see sigmoid_f).
__device__ __forceinline__ float exp_neg(float z) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(-z, 0x1.715476p+0f, -z * 0x1.4ae0cp-26f));
}
// sigmoid in fp32, off by at most (|z| + 5) 2^-24 of itself: the exponent's one
// rounding, |z| 2^-24 (log2(e) in two parts: its one-part rounding adds 0.22 |z|),
// one unit in the last place, 2 2^-24, each for exp2 and rcp, and the sum's
// rounding; zero below 2^-126.
__device__ __forceinline__ float sigmoid_f(float z) {
    return __builtin_amdgcn_rcpf(1.f + exp_neg(z));
}

// Sum over the TPR lanes of a row; for TPR above 64 over the group's waves
// through `lds` (one float per wave of the workgroup and value, used
// alternately by `phase` so that one barrier per row is enough).
template <int TPR, int NVAL, int THREADS>
__device__ __forceinline__ void row_sum(float (&s)[NVAL], float* lds, int phase) {
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int m = 1; m < W; m *= 2)
#pragma unroll
        for (int j = 0; j < NVAL; j++) s[j] += __shfl_xor(s[j], m, 64);
    if constexpr (TPR > 64) {
        constexpr int NW = THREADS / 64;
        float* buf = lds + phase * NW * NVAL;
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int j = 0; j < NVAL; j++) buf[w * NVAL + j] = s[j];
        gdr::lds_barrier();
        const int w0 = w & ~(TPR / 64 - 1);
#pragma unroll
        for (int j = 0; j < NVAL; j++) {
            s[j] = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 64; i++) s[j] += buf[(w0 + i) * NVAL + j];
        }
    }
}



// Joins the groups' column sums pairwise and writes them to `out`.
template <int VEC, int TPR, int NV, int BT>
__device__ __forceinline__ void write_part(const float (&acc)[NV][VEC], float* out, int D, float* lds) {
    constexpr int GR = BT / TPR;
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    float* mine = lds + (grp * TPR + lane) * VEC;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; e++) mine[e] = acc[i][e];
        __syncthreads();
        for (int m = GR / 2; m >= 1; m /= 2) {
            if (grp < m)
#pragma unroll
                for (int e = 0; e < VEC; e++) mine[e] += mine[m * TPR * VEC + e];
            __syncthreads();
        }
        if (grp == 0) {
            const int c = (i * TPR + lane) * VEC;
            if (c + VEC <= D) {
                typename VecU<float, VEC>::t t;
#pragma unroll
                for (int e = 0; e < VEC; e++) t[e] = mine[e];
                *(typename VecU<float, VEC>::t*)(out + c) = t;
            } else {
                for (int e = 0; c + e < D; e++) out[c + e] = mine[e];
            }
        }
    }
}

// Calls f(TPR, NV) for a row of nvt vectors: the smallest power of two of lanes
// with one vector each, 1024 with two beyond.  Rows of more than 512 vectors take 512
// lanes with two each (1024 with one: forward 8000 x 5000 bf16 89 and 73 us, 8000 x
// 4096 fp32 83 and 70, gated backward 30000 x 8192 bf16 584 and 446), but in the
// backward with vectors of 4 (5000 x 4096 fp32: 98 and 107); there 1024 lanes have
// room to read ahead.  In the forward with vectors of 4 more than 256 take 256 lanes
// (8000 x 2048: 40 and 36; vectors of 8, 30000 x 4096: 160 and 163).  FINE: every
// power of two, and 16 lanes with three vectors each instead of a wave where those
// suffice (a wave against 16 lanes at 2^18 rows of 257 bf16 elements: 124 and 101 us
// forward, 289 and 208 backward; 4 and 8 lanes with three each were slower than 16
// and 32 with one); else every second power below a wave.
template <bool FINE, bool BWD, int VEC, class F> hipError_t split_rows(int nvt, F&& f) {
#define LAYER_CASE(T, N) return f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{})
    if constexpr (FINE) {
        if (nvt <= 1) LAYER_CASE(1, 1);
        if (nvt <= 2) LAYER_CASE(2, 1);
        if (nvt <= 4) LAYER_CASE(4, 1);
        if (nvt <= 8) LAYER_CASE(8, 1);
        if (nvt <= 16) LAYER_CASE(16, 1);
        if (nvt <= 32) LAYER_CASE(32, 1);
        if (nvt <= 48) LAYER_CASE(16, 3);
    } else {
        if (nvt <= 2) LAYER_CASE(2, 1);
        if (nvt <= 8) LAYER_CASE(8, 1);
        if (nvt <= 32) LAYER_CASE(32, 1);
    }
    if (nvt <= 64) LAYER_CASE(64, 1);
    if (nvt <= 128) LAYER_CASE(128, 1);
    if (nvt <= 256) LAYER_CASE(256, 1);
    if (nvt <= 512) LAYER_CASE((VEC == 4 && !BWD ? 256 : 512), (VEC == 4 && !BWD ? 2 : 1));
    if constexpr (VEC == 4) {
        if (nvt > 1024) LAYER_CASE(1024, 2);
    }
    LAYER_CASE((VEC == 4 && BWD ? 1024 : 512), (VEC == 4 && BWD ? 1 : 2));
#undef LAYER_CASE
}

// Workgroups of a launch: enough to fill the chip several times over where each
// is short-lived (8192 against one for every row: 68 and 71 us for the gated norm
// at T=32768 H=16 D=128), and what the chip holds where each keeps weight
// gradients and reads ahead (512 against 1024: 145 and 152 us for the add norm's
// backward at 16384 x 4096).
constexpr int MAX_FWD_BLOCKS = 8192, MAX_BWD_BLOCKS = 512;
constexpr int BWD_THREADS = 512;   // of a backward workgroup, at least

inline int grid_rows(long rows, int per, long most) {
    const long n = (rows + per - 1) / per;
    return (int)(n < most ? n : most);
}

// Workgroups of a backward whose workgroups take `per` rows at a time, and where
// they leave their column sums: one workgroup writes dw and dscale itself and takes
// up to SOLO times `per` rows, which spares the launch that joins them and the
// workspace (us on the GPU alone and with the second launch, add norm D = 4096 fp32:
// 1 row 5.6 and 8.2, 4 rows 12.1 and 9.1; gated norm D = 128: 64 rows, two turns,
// 6.1 and 7.0, 128 rows 8.8 and 7.1); else every workgroup has about as many rows as
// the others.  Half of MAX_BWD_BLOCKS where that many fill the chip (`wide`: rows of
// more than 512 vectors) and up to 1024 turns in all, since each workgroup's sums are
// 8 D bytes to write and to read again (512 and 256, add norm bf16: 300 x 4096 19.4
// and 14.7 us, 900 x 2048 17.0 and 14.1, 8000 x 8192 167 and 154, with an fp32 residual
// 2400 x 4096 52.6 and 46.1; fp32 1313 x 1024 15.1 and 16.4, 8192 x 8192 320 and 326).
constexpr int SOLO = 2, FEW = 1024;
inline int bwd_blocks(NormArgs& a, int per, bool wide) {
    const long n = (a.rows + per - 1) / per;
    const long most = wide || n <= FEW ? MAX_BWD_BLOCKS / 2 : MAX_BWD_BLOCKS;
    const long turns = n <= SOLO ? n : (n + most - 1) / most;
    const int blocks = (int)((n + turns - 1) / turns);
    a.pitch = a.scale ? 2 * a.D : a.D;
    if (blocks == 1) a.part = a.dw, a.part_s = a.dscale;
    else a.part_s = a.part + a.D;
    return blocks;
}
// Joins them in a second launch (layer_add_norm.hip).
hipError_t norm_wsum(const NormArgs& a, int blocks, hipStream_t s);
hipError_t norm_zero_grads(const NormArgs& a, hipStream_t s);

}  // namespace layer

// layer_step.hip -- single-token steps on states kept in a pool (include/gdn_layer.h).
//
// gdr_step, per row and value head, with S the K x V state, a = exp(g):
//   d = beta (v - a S^T k),  S <- a S + k d^T,
//   o = scale (a S^T q + (q.k) d)          (= scale S^T q of the new state)
// so one pass over the state gives both sums S^T k and S^T q, and the state is
// read once and written once: 8 K V bytes per row and head against some 8 K V
// operations, bound by HBM.  The columns of S are independent, so a workgroup
// of 256 lanes takes VS columns of one (row, head): a lane holds 4 columns of
// K * VS / 1024 state rows, the row sums are joined over the lanes of a wave by
// shuffles and over the four waves through LDS.  The state's loads and stores are
// non-temporal (8192 heads: 212 -> 201 us).
// The state stays in registers over all rows of one slot, which are that
// state's successive tokens: the workgroup of the first such row takes them all.
#include "../../include/gdn_layer.h"
#include "gdr_device.hpp"
#include "layer_launch.hpp"

namespace layer {
namespace {

using gdr::bf16;
using gdr::f16;
using gdr::f32x4;
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Rows that share a slot: the first one after `from` (N: none), and whether one
// comes before row n.  The lanes of a wave look at 64 rows at a time.
__device__ __forceinline__ int next_row(const int32_t* slots, int slot, int from, int N) {
    const int l = threadIdx.x & 63;
    for (int m0 = from + 1; m0 < N; m0 += 64) {
        const unsigned long long hit = __ballot(m0 + l < N && slots[min(m0 + l, N - 1)] == slot);
        if (hit) return m0 + __builtin_ctzll(hit);
    }
    return N;
}
__device__ __forceinline__ bool row_before(const int32_t* slots, int slot, int n) {
    const int l = threadIdx.x & 63;
    for (int m0 = 0; m0 < n; m0 += 64)
        if (__ballot(m0 + l < n && slots[min(m0 + l, n - 1)] == slot)) return true;
    return false;
}

template <class E, int KD, int VS>
__global__ __launch_bounds__(256) void gdr_step_kernel(StepArgs a) {
    constexpr int CL = VS / 4;          // lanes across the columns
    constexpr int RW = 64 / CL;         // state rows a wave covers per load
    constexpr int NR = KD / (4 * RW);   // state rows per lane
    constexpr int NSL = KD / VS;        // column slices of a head (V = K)
    constexpr int NA = 8 / RW;          // residues modulo 8 among a lane's rows
    static_assert(8 % RW == 0 && NR % NA == 0, "sums by residue");
    __shared__ float kq[2][KD];
    __shared__ float red[4][2][VS];
    const int sl = blockIdx.x % NSL, hv = blockIdx.x / NSL % a.HV, n0 = blockIdx.x / NSL / a.HV;
    const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
    const int cl = l % CL, col = sl * VS + 4 * cl, row0 = w * RW * NR + l / CL;
    const int slot = a.slots ? a.slots[n0] : n0;
    if (slot < 0 || slot >= a.nslots) {   // padding
        if (tid < VS) ((E*)a.o)[((long)n0 * a.HV + hv) * KD + sl * VS + tid] = (E)0.f;
        return;
    }
    if (a.slots && row_before(a.slots, slot, n0)) return;   // an earlier row's workgroup takes this one
    float* S = a.state + ((long)slot * a.HV + hv) * KD * KD + (long)row0 * KD + col;
    f32x4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; i++) s[i] = __builtin_nontemporal_load((const f32x4u*)(S + i * RW * KD));
    const int hk = hv / (a.HV / a.HK);
    for (int n = n0; n < a.N;) {
        __syncthreads();   // the previous token's kq and red are read
        if (tid < 2 * KD && tid < 256) {
            const E* src = (const E*)(tid < KD ? a.k : a.q) + ((long)n * a.HK + hk) * KD;
            kq[tid / KD][tid % KD] = (float)src[tid % KD];
        }
        const float al = expf(a.g[(long)n * a.HV + hv]), be = (float)((const E*)a.beta)[(long)n * a.HV + hv];
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = (float)((const E*)a.v)[((long)n * a.HV + hv) * KD + col + e];
        __syncthreads();
        // The order of the sums over k does not depend on VS, so a row's results do
        // not depend on how many others the call has: a wave's rows by their residue
        // modulo 8, each in order, the residues joined pairwise by their lowest bit.
        float kk[NR], qk = 0.f;
        f32x4 su[NA], sq[NA];
#pragma unroll
        for (int i = 0; i < NA; i++) su[i] = sq[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NR; i++) {
            kk[i] = kq[0][row0 + i * RW];
            const float qq = kq[1][row0 + i * RW];
            su[i % NA] += kk[i] * s[i];
            sq[i % NA] += qq * s[i];
        }
        for (int i = l; i < KD; i += 64) qk += kq[0][i] * kq[1][i];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            qk += __shfl_xor(qk, m, 64);
            if (m >= CL)
#pragma unroll
                for (int i = 0; i < NA; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        su[i][e] += __shfl_xor(su[i][e], m, 64);
                        sq[i][e] += __shfl_xor(sq[i][e], m, 64);
                    }
        }
#pragma unroll
        for (int m = 1; m < NA; m *= 2)
#pragma unroll
            for (int i = 0; i < NA; i += 2 * m) su[i] += su[i + m], sq[i] += sq[i + m];
        if (l < CL) {
            *(f32x4*)&red[w][0][4 * cl] = su[0];
            *(f32x4*)&red[w][1][4 * cl] = sq[0];
        }
        __syncthreads();
        const f32x4 u = *(f32x4*)&red[0][0][4 * cl] + *(f32x4*)&red[1][0][4 * cl] + *(f32x4*)&red[2][0][4 * cl] +
                        *(f32x4*)&red[3][0][4 * cl];
        const f32x4 o = *(f32x4*)&red[0][1][4 * cl] + *(f32x4*)&red[1][1][4 * cl] + *(f32x4*)&red[2][1][4 * cl] +
                        *(f32x4*)&red[3][1][4 * cl];
        f32x4 d;
#pragma unroll
        for (int e = 0; e < 4; e++) d[e] = be * (v[e] - al * u[e]);
#pragma unroll
        for (int i = 0; i < NR; i++) s[i] = al * s[i] + kk[i] * d;
        if (w == 0 && l < CL) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                ((E*)a.o)[((long)n * a.HV + hv) * KD + col + e] = (E)(a.scale * (al * o[e] + qk * d[e]));
        }
        n = a.slots ? next_row(a.slots, slot, n, a.N) : a.N;
    }
#pragma unroll
    for (int i = 0; i < NR; i++) __builtin_nontemporal_store((f32x4u)s[i], (f32x4u*)(S + i * RW * KD));
}

// glr_step: h = exp(g) S + x per channel, 12 to 16 bytes of traffic each; four
// channels a lane, the last ones of an odd row one by one.
constexpr int STEP_LANES = 128;
struct Chan4 {
    int n;   // channels of this lane
    template <class T> __device__ __forceinline__ f32x4 load(const T* p) const {
        typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        f32x4 r = {0.f, 0.f, 0.f, 0.f};
        if (n == 4) return __builtin_convertvector(*(const t4*)p, f32x4);
        for (int i = 0; i < n; i++) r[i] = (float)p[i];
        return r;
    }
    template <class T> __device__ __forceinline__ void store(T* p, f32x4 v) const {
        typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
        if (n == 4) *(t4*)p = __builtin_convertvector(v, t4);
        else
            for (int i = 0; i < n; i++) p[i] = (T)v[i];
    }
};
template <class E>
__global__ __launch_bounds__(STEP_LANES) void glr_step_kernel(StepArgs a) {
    const int nb = (a.D + 4 * STEP_LANES - 1) / (4 * STEP_LANES);
    const int n0 = blockIdx.x / nb, c = (blockIdx.x % nb * STEP_LANES + threadIdx.x) * 4;
    const Chan4 ch{c < a.D ? min(a.D - c, 4) : 0};
    const int slot = a.slots ? a.slots[n0] : n0;
    if (slot < 0 || slot >= a.nslots) {
        ch.store((E*)a.o + (long)n0 * a.D + c, f32x4{0.f, 0.f, 0.f, 0.f});
        return;
    }
    if (a.slots && row_before(a.slots, slot, n0)) return;
    float* S = a.state + (long)slot * a.D + c;
    f32x4 s = ch.load(S);
    for (int n = n0; n < a.N;) {
        const long at = (long)n * a.D + c;
        const f32x4 g = ch.load(a.g + at), x = ch.load((const E*)a.v + at);
#pragma unroll
        for (int e = 0; e < 4; e++) s[e] = expf(g[e]) * s[e] + x[e];
        ch.store((E*)a.o + at, s);
        n = a.slots ? next_row(a.slots, slot, n, a.N) : a.N;
    }
    ch.store(S, s);
}

// Columns of a workgroup at K = 128, by the heads there are (rows times value
// heads): narrow slices spread few heads over the chip, whole heads move most
// per workgroup.  us at slices of 32 / 64 / 128 columns: 16 heads 3.3 / 3.6 / 4.3,
// 64: 4.2 / 4.6 / 5.5, 128: 5.5 / 5.4 / 6.1, 512: 14.3 / 11.9 / 12.8, 1024: 27.2 /
// 25.3 / 26.2, 8192: 202 / 194 / 190 (5.66 TB/s).  At K = 64 whole heads are as
// fast as halves for few heads and faster from 256 on (8192: 50.8 / 56.8).
template <class E, int KD, int VS> hipError_t launch(const StepArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((gdr_step_kernel<E, KD, VS>), dim3(a.N * a.HV * (KD / VS)), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <class E> hipError_t gdr(const StepArgs& a, hipStream_t s) {
    const int heads = a.N * a.HV;
    if (a.K == 64) return launch<E, 64, 64>(a, s);
    if (heads < 128) return launch<E, 128, 32>(a, s);
    return heads < 4096 ? launch<E, 128, 64>(a, s) : launch<E, 128, 128>(a, s);
}
template <class E> hipError_t glr(const StepArgs& a, hipStream_t s) {
    const int per = 4 * STEP_LANES;
    hipLaunchKernelGGL((glr_step_kernel<E>), dim3(a.N * ((a.D + per - 1) / per)), dim3(STEP_LANES), 0, s, a);
    return hipGetLastError();
}

}  // namespace

#define BY_TYPE(F, a, s)                     \
    switch (a.dtype) {                       \
        case GDR_F32: return F<float>(a, s); \
        case GDR_F16: return F<f16>(a, s);   \
        default: return F<bf16>(a, s);       \
    }

hipError_t launch_gdr_step(const StepArgs& a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    BY_TYPE(gdr, a, s)
}
hipError_t launch_glr_step(const StepArgs& a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    BY_TYPE(glr, a, s)
}

}  // namespace layer

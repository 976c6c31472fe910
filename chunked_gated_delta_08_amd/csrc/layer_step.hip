// layer_step.hip -- single-token steps on states kept in a pool (include/gdn_layer.h).
//
// gdr_step, per row and value head, with S the K x V state, a = exp(g):
//   u = a S^T k,  d = beta (v - u),  S <- a S + k d^T,
//   o = scale (a S^T q + (q.k) d)          (= scale S^T q of the new state)
// so one pass over the state gives both sums S^T k and S^T q, and the state is
// read once and written once: 8 K V bytes per row and head against some 8 K V
// operations, bound by HBM.  The columns of S are independent, so a workgroup
// of 256 lanes takes VS columns of one (row, head): a lane holds 4 columns of
// K * VS / 1024 state rows, the row sums are joined over the lanes of a wave by
// shuffles and over the four waves through LDS.
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
    for (int i = 0; i < NR; i++) s[i] = *(const f32x4u*)(S + i * RW * KD);
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
        float kk[NR], qk = 0.f;
        f32x4 su = {0.f, 0.f, 0.f, 0.f}, sq = su;
#pragma unroll
        for (int i = 0; i < NR; i++) {
            kk[i] = kq[0][row0 + i * RW];
            const float qq = kq[1][row0 + i * RW];
            su += kk[i] * s[i];
            sq += qq * s[i];
        }
        for (int i = l; i < KD; i += 64) qk += kq[0][i] * kq[1][i];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            qk += __shfl_xor(qk, m, 64);
            if (m >= CL)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    su[e] += __shfl_xor(su[e], m, 64);
                    sq[e] += __shfl_xor(sq[e], m, 64);
                }
        }
        if (l < CL) {
            *(f32x4*)&red[w][0][4 * cl] = su;
            *(f32x4*)&red[w][1][4 * cl] = sq;
        }
        __syncthreads();
        su = *(f32x4*)&red[0][0][4 * cl] + *(f32x4*)&red[1][0][4 * cl] + *(f32x4*)&red[2][0][4 * cl] +
             *(f32x4*)&red[3][0][4 * cl];
        sq = *(f32x4*)&red[0][1][4 * cl] + *(f32x4*)&red[1][1][4 * cl] + *(f32x4*)&red[2][1][4 * cl] +
             *(f32x4*)&red[3][1][4 * cl];
        f32x4 d;
#pragma unroll
        for (int e = 0; e < 4; e++) d[e] = be * (v[e] - al * su[e]);
#pragma unroll
        for (int i = 0; i < NR; i++) s[i] = al * s[i] + kk[i] * d;
        if (w == 0 && l < CL) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                ((E*)a.o)[((long)n * a.HV + hv) * KD + col + e] = (E)(a.scale * (al * sq[e] + qk * d[e]));
        }
        n = a.slots ? next_row(a.slots, slot, n, a.N) : a.N;
    }
#pragma unroll
    for (int i = 0; i < NR; i++) *(f32x4u*)(S + i * RW * KD) = s[i];
}

// glr_step: h = exp(g) S + x per channel; one lane per channel, 12 to 16 bytes
// of traffic each.
template <class E>
__global__ __launch_bounds__(256) void glr_step_kernel(StepArgs a) {
    const int nb = (a.D + 255) / 256;
    const int n0 = blockIdx.x / nb, c = blockIdx.x % nb * 256 + threadIdx.x;
    const int slot = a.slots ? a.slots[n0] : n0;
    const bool in = c < a.D;
    if (slot < 0 || slot >= a.nslots) {
        if (in) ((E*)a.o)[(long)n0 * a.D + c] = (E)0.f;
        return;
    }
    if (a.slots && row_before(a.slots, slot, n0)) return;
    float* S = a.state + (long)slot * a.D + c;
    float s = in ? *S : 0.f;
    for (int n = n0; n < a.N;) {
        if (in) {
            s = expf(a.g[(long)n * a.D + c]) * s + (float)((const E*)a.v)[(long)n * a.D + c];
            ((E*)a.o)[(long)n * a.D + c] = (E)s;
        }
        n = a.slots ? next_row(a.slots, slot, n, a.N) : a.N;
    }
    if (in) *S = s;
}

template <class E> hipError_t gdr(const StepArgs& a, hipStream_t s) {
    const int grid = a.N * a.HV;
    if (a.K == 128) hipLaunchKernelGGL((gdr_step_kernel<E, 128, 32>), dim3(grid * 4), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((gdr_step_kernel<E, 64, 32>), dim3(grid * 2), dim3(256), 0, s, a);
    return hipGetLastError();
}
template <class E> hipError_t glr(const StepArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((glr_step_kernel<E>), dim3(a.N * ((a.D + 255) / 256)), dim3(256), 0, s, a);
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

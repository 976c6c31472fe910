// layer_gated_norm.hip -- the gated RMSNorm, forward and backward (include/gdn_layer.h).
//
// Per row of D elements, with r = (sum x^2 / D + eps)^(-1/2) and n = x r:
//   y = n w act(z)
//   dn = dy w act(z),  dx = r (dn - n mean(dn n)),  dz = dy n w act'(z),  dw = sum_rows dy n act(z)
// A few operations per element, so both directions are bound by HBM: each reads
// its rows once into registers and writes each output once.  Both sums of the
// backward (x^2 and dn x) need no r, so it has one reduction per row too.  dw
// stays in registers over all rows of a persistent workgroup; the workgroups'
// partial sums are joined in a fixed order by a second launch.
// Measured (bf16, D = 128): 2^19 rows forward 67 us (6.0 TB/s of 403 MB), 2^21 rows
// backward 521 us and 5 for the join (5.1 TB/s of 2.68 GB, near a large copy's rate;
// 512 to 533 on other cards); 128 rows 3 to 4 us, which
// is the launch.
#include "layer_rows.hpp"

namespace layer {
namespace {

// act(z) from s = sigmoid(z).
__device__ __forceinline__ float act_of(float z, float s, bool silu) { return silu ? z * s : s; }
// act(z) and its derivative for the backward, from one value that is held in between.
// silu, s (1 + z (1 - s)): s itself.  Where s is near one, 1 - s has few digits, but it
// is small next to 1.  sigmoid, s (1 - s): there every digit of the smaller factor
// counts (s is 1 in fp32 from z = 17 on), so that is held, sigmoid(-|z|) with z's sign.
template <int ACT> struct Gate {
    float v;
    __device__ __forceinline__ void of(float z) {
        v = ACT == GDN_ACT_SILU ? sigmoid_f(z) : copysignf(sigmoid_f(-fabsf(z)), z);
    }
    __device__ __forceinline__ float act(float z) const {
        return ACT == GDN_ACT_SILU ? z * v : (__float_as_int(v) < 0 ? 0.f : 1.f) - v;
    }
    __device__ __forceinline__ float slope(float z) const {
        const float p = fabsf(v);
        return ACT == GDN_ACT_SILU ? v * (1.f + z * (1.f - v)) : p * (1.f - p);
    }
};
constexpr int NO_GATE = -1;

template <class E, int VEC, int NV> struct Rows {   // a row of x, z and dy as loaded
    Raw<E, VEC> x[NV], z[NV], g[NV];
};
template <class E, int VEC, int TPR, int NV, bool GATE, bool BWD>
__device__ __forceinline__ void load_rows(Rows<E, VEC, NV>& r, const NormArgs& a, long row, int lane) {
    const long off = (row < a.rows ? row : a.rows - 1) * a.D;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        load_raw<TPR>(r.x[i], (const E*)a.x + off, i, lane, a.D);
        if constexpr (GATE) load_raw<TPR>(r.z[i], (const E*)a.z + off, i, lane, a.D);
        if constexpr (BWD) load_raw<TPR>(r.g[i], (const E*)a.dy + off, i, lane, a.D);
    }
}
// One pass: many short-lived workgroups, whose next rows' loads overlap by themselves.
template <class E, int VEC, int TPR, int NV, bool GATE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void gated_norm_fwd_kernel(NormArgs a) {
    constexpr int NT = TPR > 256 ? TPR : 256, GR = NT / TPR;   // rows a workgroup takes at a time
    __shared__ float lds[TPR > 64 ? 2 * NT / 64 : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = a.D;
    const float inv = 1.f / (float)D;
    const bool silu = a.act == GDN_ACT_SILU;
    float w[NV][VEC];
    load_weights<VEC, TPR, NV>(w, a.w, lane, D);
    int phase = 0;
    for (long r0 = (long)blockIdx.x * GR; r0 < a.rows; r0 += (long)gridDim.x * GR, phase ^= 1) {
        Rows<E, VEC, NV> in;
        load_rows<E, VEC, TPR, NV, GATE, false>(in, a, r0 + grp, lane);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float v = (float)in.x[i].v[e];
                s[0] += v * v;
            }
        row_sum<TPR, 1, NT>(s, lds, phase);
        const float r = rsqrtf(s[0] * inv + a.eps);
        if (r0 + grp >= a.rows) continue;
        E* y = (E*)a.y + (r0 + grp) * D;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                o[e] = (float)in.x[i].v[e] * r * w[i][e];
                if constexpr (GATE) {
                    const float z = (float)in.z[i].v[e];
                    o[e] *= act_of(z, sigmoid_f(z), silu);
                }
            }
            store_vec<E, VEC>(y, (i * TPR + lane) * VEC, D, o);
        }
    }
}

// A workgroup takes rows in turn, the next one's on their way meanwhile.
template <class E, int VEC, int TPR, int NV, int ACT, int BT>
__global__ __launch_bounds__(BT) void gated_norm_bwd_kernel(NormArgs a) {
    constexpr int GR = BT / TPR;
    constexpr bool GATE = ACT != NO_GATE;
    __shared__ float lds[BT * VEC];
    __shared__ float red[TPR > 64 ? 2 * 2 * (BT / 64) : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = a.D;
    const float inv = 1.f / (float)D;
    float w[NV][VEC], dw[NV][VEC];
    load_weights<VEC, TPR, NV>(w, a.w, lane, D);
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++) dw[i][e] = 0.f;
    int phase = 0;
    Rows<E, VEC, NV> in, next;
    load_rows<E, VEC, TPR, NV, GATE, true>(in, a, (long)blockIdx.x * GR + grp, lane);
    for (long r0 = (long)blockIdx.x * GR; r0 < a.rows; r0 += (long)gridDim.x * GR, phase ^= 1) {
        if constexpr (NV == 1) load_rows<E, VEC, TPR, NV, GATE, true>(next, a, r0 + (long)gridDim.x * GR + grp, lane);
        float s[2] = {0.f, 0.f};
        Gate<ACT> gate[GATE ? NV : 1][VEC];   // formed once
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float x = (float)in.x[i].v[e];
                float dn = (float)in.g[i].v[e] * w[i][e];
                if constexpr (GATE) {
                    const float z = (float)in.z[i].v[e];
                    gate[i][e].of(z);
                    dn *= gate[i][e].act(z);
                }
                s[0] += x * x;
                s[1] += dn * x;
            }
        row_sum<TPR, 2, BT>(s, red, phase);
        const float r = rsqrtf(s[0] * inv + a.eps), m = r * s[1] * inv;   // m = mean(dn n)
        if (r0 + grp < a.rows) {
            const long off = (r0 + grp) * D;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = (i * TPR + lane) * VEC;
                float dx[VEC], dz[VEC];
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const float n = (float)in.x[i].v[e] * r, g = (float)in.g[i].v[e];
                    float dn = g * w[i][e], t = g * n;   // t = dy n
                    if constexpr (GATE) {
                        const float z = (float)in.z[i].v[e], f = gate[i][e].act(z);
                        dn *= f;
                        dz[e] = t * w[i][e] * gate[i][e].slope(z);
                        t *= f;
                    }
                    dw[i][e] += t;
                    dx[e] = r * (dn - n * m);
                }
                store_vec<E, VEC>((E*)a.dx + off, c, D, dx);
                if constexpr (GATE) store_vec<E, VEC>((E*)a.dz + off, c, D, dz);
            }
        }
        if constexpr (NV == 1) in = next;
        else   // no registers to read ahead
            load_rows<E, VEC, TPR, NV, GATE, true>(in, a, r0 + (long)gridDim.x * GR + grp, lane);
    }
    write_part<VEC, TPR, NV, BT>(dw, a.part + (long)blockIdx.x * a.pitch, D, lds);
}

template <class E> hipError_t gated_fwd(const NormArgs& a, hipStream_t s) {
    constexpr int VEC = sizeof(E) == 4 ? 4 : 8;
    return split_rows<true, false, VEC>((a.D + VEC - 1) / VEC, [&](auto T, auto N) {
        constexpr int TPR = decltype(T)::value, NV = decltype(N)::value, NT = TPR > 256 ? TPR : 256;
        const dim3 grid(grid_rows(a.rows, NT / TPR, MAX_FWD_BLOCKS));
        if (a.z) hipLaunchKernelGGL((gated_norm_fwd_kernel<E, VEC, TPR, NV, true>), grid, dim3(NT), 0, s, a);
        else hipLaunchKernelGGL((gated_norm_fwd_kernel<E, VEC, TPR, NV, false>), grid, dim3(NT), 0, s, a);
        return hipGetLastError();
    });
}

template <class E> hipError_t gated_bwd(const NormArgs& a0, hipStream_t s) {
    constexpr int VEC = sizeof(E) == 4 ? 4 : 8;
    NormArgs a = a0;
    int blocks = 1;
    const hipError_t e = split_rows<true, true, VEC>((a.D + VEC - 1) / VEC, [&](auto T, auto N) {
        constexpr int TPR = decltype(T)::value, NV = decltype(N)::value, BT = TPR > BWD_THREADS ? TPR : BWD_THREADS;
        blocks = bwd_blocks(a, BT / TPR, TPR * NV > 512);
        const auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(BT), 0, s, a); };
        if (!a.z) run(gated_norm_bwd_kernel<E, VEC, TPR, NV, NO_GATE, BT>);
        else if (a.act == GDN_ACT_SILU) run(gated_norm_bwd_kernel<E, VEC, TPR, NV, GDN_ACT_SILU, BT>);
        else run(gated_norm_bwd_kernel<E, VEC, TPR, NV, GDN_ACT_SIGMOID, BT>);
        return hipGetLastError();
    });
    return e != hipSuccess ? e : norm_wsum(a, blocks, s);
}

}  // namespace

#define BY_TYPE(F, a, s)                     \
    switch (a.dtype) {                       \
        case GDR_F32: return F<float>(a, s); \
        case GDR_F16: return F<f16>(a, s);   \
        default: return F<bf16>(a, s);       \
    }

hipError_t launch_gated_norm_fwd(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    BY_TYPE(gated_fwd, a, s)
}
hipError_t launch_gated_norm_bwd(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return norm_zero_grads(a, s);
    BY_TYPE(gated_bwd, a, s)
}

}  // namespace layer

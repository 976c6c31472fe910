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
#include "layer_rows.hpp"

namespace layer {
namespace {

__device__ __forceinline__ void gate(float z, int act, float& f, float& df) {
    const float s = sigmoid_f(z);
    if (act == GDN_ACT_SILU) {
        f = z * s;
        df = s * (1.f + z * (1.f - s));
    } else {
        f = s;
        df = s * (1.f - s);
    }
}

// ---------------------------------------------------------------- forward
template <class E, int VEC, int TPR, int NV, bool GATE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void gated_norm_fwd_kernel(NormArgs a) {
    constexpr int NT = TPR > 256 ? TPR : 256, GR = NT / TPR;   // rows a workgroup takes at a time
    __shared__ float lds[TPR > 64 ? 2 * NT / 64 : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = a.D;
    const float inv = 1.f / (float)D;
    float w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        Raw<float, VEC> t;
        load_raw<float, VEC>(t, a.w, (i * TPR + lane) * VEC, D);
#pragma unroll
        for (int e = 0; e < VEC; e++) w[i][e] = t.v[e];
    }
    int phase = 0;
    for (long r0 = (long)blockIdx.x * GR; r0 < a.rows; r0 += (long)gridDim.x * GR, phase ^= 1) {
        const bool live = r0 + grp < a.rows;
        const long off = (live ? r0 + grp : a.rows - 1) * D;
        const E* x = (const E*)a.x + off;
        const E* z = (const E*)a.z + off;
        E* y = (E*)a.y + off;
        Raw<E, VEC> xr[NV], zr[GATE ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; i++) load_raw<E, VEC>(xr[i], x, (i * TPR + lane) * VEC, D);
        if constexpr (GATE)
#pragma unroll
            for (int i = 0; i < NV; i++) load_raw<E, VEC>(zr[i], z, (i * TPR + lane) * VEC, D);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float v = (float)xr[i].v[e];
                s[0] += v * v;
            }
        row_sum<TPR, 1, NT>(s, lds, phase);
        const float r = rsqrtf(s[0] * inv + a.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                o[e] = (float)xr[i].v[e] * r * w[i][e];
                if constexpr (GATE) {
                    const float zz = (float)zr[i].v[e], sg = sigmoid_f(zz);
                    o[e] *= a.act == GDN_ACT_SILU ? zz * sg : sg;
                }
            }
            store_vec<E, VEC>(y, (i * TPR + lane) * VEC, D, o);
        }
    }
}

template <class E, int VEC, int TPR, int NV, bool GATE>
__global__ __launch_bounds__(BT) void gated_norm_bwd_kernel(NormArgs a) {
    constexpr int GR = BT / TPR;
    __shared__ float lds[BT * VEC];
    __shared__ float red[TPR > 64 ? 2 * 2 * (BT / 64) : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = a.D;
    const float inv = 1.f / (float)D;
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        Raw<float, VEC> t;
        load_raw<float, VEC>(t, a.w, (i * TPR + lane) * VEC, D);
#pragma unroll
        for (int e = 0; e < VEC; e++) w[i][e] = t.v[e], dw[i][e] = 0.f;
    }
    int phase = 0;
    for (long r0 = (long)blockIdx.x * GR; r0 < a.rows; r0 += (long)gridDim.x * GR, phase ^= 1) {
        const bool live = r0 + grp < a.rows;
        const long off = (live ? r0 + grp : a.rows - 1) * D;
        Raw<E, VEC> xr[NV], gr[NV], zr[GATE ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * VEC;
            load_raw<E, VEC>(xr[i], (const E*)a.x + off, c, D);
            load_raw<E, VEC>(gr[i], (const E*)a.dy + off, c, D);
            if constexpr (GATE) load_raw<E, VEC>(zr[i], (const E*)a.z + off, c, D);
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float x = (float)xr[i].v[e];
                float dn = (float)gr[i].v[e] * w[i][e];
                if constexpr (GATE) {
                    float f, df;
                    gate((float)zr[i].v[e], a.act, f, df);
                    dn *= f;
                }
                s[0] += x * x;
                s[1] += dn * x;
            }
        row_sum<TPR, 2, BT>(s, red, phase);
        const float r = rsqrtf(s[0] * inv + a.eps), m = r * s[1] * inv;   // m = mean(dn n)
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * VEC;
            float dx[VEC], dz[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float n = (float)xr[i].v[e] * r, g = (float)gr[i].v[e];
                float dn = g * w[i][e], t = g * n;   // t = dy n
                if constexpr (GATE) {
                    float f, df;
                    gate((float)zr[i].v[e], a.act, f, df);
                    dn *= f;
                    dz[e] = t * w[i][e] * df;
                    t *= f;
                }
                dw[i][e] += t;
                dx[e] = r * (dn - n * m);
            }
            store_vec<E, VEC>((E*)a.dx + off, c, D, dx);
            if constexpr (GATE) store_vec<E, VEC>((E*)a.dz + off, c, D, dz);
        }
    }
    write_part<VEC, TPR, NV>(dw, a.part + (long)blockIdx.x * D, D, lds);
}


template <class E> hipError_t gated_fwd(const NormArgs& a, hipStream_t s) {
    constexpr int VEC = sizeof(E) == 4 ? 4 : 8;
    return split_rows<8, VEC>((a.D + VEC - 1) / VEC, [&](auto T, auto N) {
        constexpr int TPR = decltype(T)::value, NV = decltype(N)::value, NT = TPR > 256 ? TPR : 256;
        const dim3 grid(grid_rows(a.rows, NT / TPR, 1 << 20));
        if (a.z) hipLaunchKernelGGL((gated_norm_fwd_kernel<E, VEC, TPR, NV, true>), grid, dim3(NT), 0, s, a);
        else hipLaunchKernelGGL((gated_norm_fwd_kernel<E, VEC, TPR, NV, false>), grid, dim3(NT), 0, s, a);
        return hipGetLastError();
    });
}

template <class E> hipError_t gated_bwd(const NormArgs& a0, hipStream_t s) {
    constexpr int VEC = sizeof(E) == 4 ? 4 : 8;
    NormArgs a = a0;
    int blocks = 1;
    const hipError_t e = split_rows<8, VEC>((a.D + VEC - 1) / VEC, [&](auto T, auto N) {
        constexpr int TPR = decltype(T)::value, NV = decltype(N)::value;
        blocks = grid_rows(a.rows, BT / TPR, MAX_BWD_BLOCKS);
        if (blocks == 1) a.part = a.dw;
        if (a.z) hipLaunchKernelGGL((gated_norm_bwd_kernel<E, VEC, TPR, NV, true>), dim3(blocks), dim3(BT), 0, s, a);
        else hipLaunchKernelGGL((gated_norm_bwd_kernel<E, VEC, TPR, NV, false>), dim3(blocks), dim3(BT), 0, s, a);
        return hipGetLastError();
    });
    return e != hipSuccess ? e : norm_wsum(a, blocks, a.D, s);
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

// layer_add_norm.hip -- the residual add with RMSNorm, forward and backward
// (include/gdn_layer.h), and the join of both norms' weight gradients.
//
// Per row of D elements:
//   h = res + s x,  r = (sum h^2 / D + eps)^(-1/2),  n = h r,  y = n w,  res' = h
//   dn = dy w,  dh = dres + r (dn - n mean(dn n)),
//   dx = s dh,  ds = sum_rows dh x,  dw = sum_rows dy n
// With dropout (DROP) x stands for m x, m = 1 / (1 - p) or 0 from the generator of
// layer_dropout.hpp, in the backward again: dx = m s dh, ds = sum_rows dh m x.
// y is formed from the unrounded h; the backward takes the stored res' for h.
// Bound by HBM, built like the gated norm (layer_gated_norm.hip).  Measured:
// forward 32768 x 2048 bf16 92 us (5.8 TB/s of 537 MB), backward 16384 x 4096 fp16
// 142 us and 7 for the join (5.4 TB/s of 805 MB), 5 x 2048 3 to 4 us, which is the
// launch; with dropout forward 32768 x 2048 bf16 91 us, backward 16384 x 4096 fp16 155.  Larger
// forwards fall off (131072 x 2048 bf16 439 us, with dropout 471, 4.9 and 4.6 TB/s; 262144 4.5 and 4.4), the
// backward's fewer workgroups do not (380 us, 5.65; 5.35).
// No value is spilled but in the backward with an fp32 residual and a scale beyond D = 4096
// (three in fp32, seven with dropout, one with dropout and bf16 rows).
#include "layer_dropout.hpp"
#include "layer_rows.hpp"

namespace layer {
namespace {

template <class E, class R, int VEC, int NV> struct Rows {   // a row as loaded: x (or dy), res, dres and x
    Raw<E, VEC> e[NV], x[NV];
    Raw<R, VEC> res[NV], dres[NV];
};
template <class T, int VEC, int TPR, int NV>
__device__ __forceinline__ void load_row(Raw<T, VEC> (&r)[NV], const void* p, long off, int lane, int D) {
#pragma unroll
    for (int i = 0; i < NV; i++) load_raw<TPR>(r[i], (const T*)p + off, i, lane, D);
}
template <class E, class R, int VEC, int TPR, int NV, bool SCALE, bool DROP>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void add_norm_fwd_kernel(NormArgs a) {
    constexpr int NT = TPR > 256 ? TPR : 256, GR = NT / TPR;
    __shared__ float lds[TPR > 64 ? 2 * NT / 64 : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = a.D;
    const float inv = 1.f / (float)D;
    float w[NV][VEC], sc[SCALE ? NV : 1][VEC];
    load_weights<VEC, TPR, NV>(w, a.w, lane, D);
    if constexpr (SCALE) load_weights<VEC, TPR, NV>(sc, a.scale, lane, D);
    const Keep keep(a.drop);
    int phase = 0;
    for (long r0 = (long)blockIdx.x * GR; r0 < a.rows; r0 += (long)gridDim.x * GR, phase ^= 1) {
        const bool live = r0 + grp < a.rows;
        const long row = live ? r0 + grp : a.rows - 1, off = row * D;
        Rows<E, R, VEC, NV> in;
        load_row<E, VEC, TPR, NV>(in.e, a.x, off, lane, D);
        load_row<R, VEC, TPR, NV>(in.res, a.res, off, lane, D);
        float h[NV][VEC], s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            uint32_t m = 0;
            if constexpr (DROP) m = keep.mask<VEC>(row, (D + 7) / 8, (i * TPR + lane) * VEC);
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                float v = (float)in.e[i].v[e];
                if constexpr (DROP) v = m >> e & 1 ? v * keep.mul : 0.f;
                h[i][e] = (float)in.res[i].v[e] + (SCALE ? sc[i][e] * v : v);
                s[0] += h[i][e] * h[i][e];
            }
        }
        row_sum<TPR, 1, NT>(s, lds, phase);
        const float r = rsqrtf(s[0] * inv + a.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * VEC;
            store_vec<R, VEC>((R*)a.res_out + off, c, D, h[i]);
#pragma unroll
            for (int e = 0; e < VEC; e++) h[i][e] *= r * w[i][e];
            store_vec<E, VEC>((E*)a.y + off, c, D, h[i]);
        }
    }
}

template <class E, class R, int VEC, int TPR, int NV, bool SCALE>
__device__ __forceinline__ void load_rows(Rows<E, R, VEC, NV>& r, const NormArgs& a, long row, int lane) {
    const long off = (row < a.rows ? row : a.rows - 1) * a.D;
    load_row<E, VEC, TPR, NV>(r.e, a.dy, off, lane, a.D);
    load_row<R, VEC, TPR, NV>(r.res, a.res, off, lane, a.D);
    if (a.dres) load_row<R, VEC, TPR, NV>(r.dres, a.dres, off, lane, a.D);
    if constexpr (SCALE) load_row<E, VEC, TPR, NV>(r.x, a.x, off, lane, a.D);
}

template <class E, class R, int VEC, int TPR, int NV, bool SCALE, bool DROP, int BT>
__global__ __launch_bounds__(BT) void add_norm_bwd_kernel(NormArgs a) {
    constexpr int GR = BT / TPR;
    __shared__ float lds[BT * VEC];
    __shared__ float red[TPR > 64 ? 2 * 2 * (BT / 64) : 1];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR, D = a.D;
    const float inv = 1.f / (float)D;
    float w[NV][VEC], dw[NV][VEC], sc[SCALE ? NV : 1][VEC], ds[SCALE ? NV : 1][VEC];
    load_weights<VEC, TPR, NV>(w, a.w, lane, D);
    if constexpr (SCALE) load_weights<VEC, TPR, NV>(sc, a.scale, lane, D);
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < VEC; e++) {
            dw[i][e] = 0.f;
            if (SCALE) ds[i][e] = 0.f;
        }
    const Keep keep(a.drop);
    int phase = 0;
    Rows<E, R, VEC, NV> in, next;
    load_rows<E, R, VEC, TPR, NV, SCALE>(in, a, (long)blockIdx.x * GR + grp, lane);
    for (long r0 = (long)blockIdx.x * GR; r0 < a.rows; r0 += (long)gridDim.x * GR, phase ^= 1) {
        if constexpr (NV == 1) load_rows<E, R, VEC, TPR, NV, SCALE>(next, a, r0 + (long)gridDim.x * GR + grp, lane);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const float h = (float)in.res[i].v[e];
                s[0] += h * h;
                s[1] += (float)in.e[i].v[e] * w[i][e] * h;
            }
        row_sum<TPR, 2, BT>(s, red, phase);
        const float r = rsqrtf(s[0] * inv + a.eps), m = r * s[1] * inv;
        if (r0 + grp < a.rows) {
            const long off = (r0 + grp) * D;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = (i * TPR + lane) * VEC;
                float dh[VEC], dx[VEC];
                uint32_t m01 = 0;
                if constexpr (DROP) m01 = keep.mask<VEC>(r0 + grp, (D + 7) / 8, c);
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const float n = (float)in.res[i].v[e] * r, g = (float)in.e[i].v[e];
                    dh[e] = r * (g * w[i][e] - n * m) + (a.dres ? (float)in.dres[i].v[e] : 0.f);
                    dw[i][e] += g * n;
                    dx[e] = dh[e];
                    if constexpr (DROP) dx[e] = m01 >> e & 1 ? dh[e] * keep.mul : 0.f;
                    if constexpr (SCALE) {
                        ds[i][e] += DROP && !(m01 >> e & 1) ? 0.f : dx[e] * (float)in.x[i].v[e];
                        dx[e] *= sc[i][e];
                    }
                }
                store_vec<R, VEC>((R*)a.dres_out + off, c, D, dh);
                if (a.dx) store_vec<E, VEC>((E*)a.dx + off, c, D, dx);
            }
        }
        if constexpr (NV == 1) in = next;
        else   // no registers to read ahead
            load_rows<E, R, VEC, TPR, NV, SCALE>(in, a, r0 + (long)gridDim.x * GR + grp, lane);
    }
    const long at = (long)blockIdx.x * a.pitch;
    write_part<VEC, TPR, NV, BT>(dw, a.part + at, D, lds);
    if constexpr (SCALE) write_part<VEC, TPR, NV, BT>(ds, a.part_s + at, D, lds);
}

// out[c] = sum over the partial rows in a fixed order: 16 columns per
// workgroup, 64 row slices, joined pairwise within a wave, then over the waves.
// Column c < D goes to dw, the others to dscale.
__global__ __launch_bounds__(1024) void norm_wsum_kernel(const float* part, int blocks, int n, int D, float* dw,
                                                         float* dscale) {
    __shared__ float lds[16][17];
    const int k = threadIdx.x & 15, c = blockIdx.x * 16 + k, sl = threadIdx.x >> 4;
    float v[MAX_BWD_BLOCKS / 64], t = 0.f;   // all loads on their way at once
#pragma unroll
    for (int i = 0; i < MAX_BWD_BLOCKS / 64; i++) {
        const int b = sl + 64 * i;
        v[i] = b < blocks && c < n ? part[(long)b * n + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < MAX_BWD_BLOCKS / 64; i++) t += v[i];
    t += __shfl_xor(t, 16);
    t += __shfl_xor(t, 32);
    if ((threadIdx.x & 63) < 16) lds[threadIdx.x >> 6][k] = t;
    __syncthreads();
    if (threadIdx.x < 16 && c < n) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) t += lds[i][k];
        (c < D ? dw[c] : dscale[c - D]) = t;
    }
}

__global__ void zero_kernel(float* a, float* b, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    a[i] = 0.f;
    if (b) b[i] = 0.f;
}

// f(has a scale, is dropped out)
template <class F> void by_branch(const NormArgs& a, F&& f) {
    if (a.dropped) a.scale ? f(std::true_type{}, std::true_type{}) : f(std::false_type{}, std::true_type{});
    else a.scale ? f(std::true_type{}, std::false_type{}) : f(std::false_type{}, std::false_type{});
}

template <class E, class R> hipError_t add_fwd(const NormArgs& a, hipStream_t s) {
    constexpr int VEC = sizeof(R) == 4 ? 4 : 8;
    return split_rows<false, false, VEC>((a.D + VEC - 1) / VEC, [&](auto T, auto N) {
        constexpr int TPR = decltype(T)::value, NV = decltype(N)::value, NT = TPR > 256 ? TPR : 256;
        const dim3 grid(grid_rows(a.rows, NT / TPR, MAX_FWD_BLOCKS));
        by_branch(a, [&](auto S, auto K) {
            hipLaunchKernelGGL((add_norm_fwd_kernel<E, R, VEC, TPR, NV, decltype(S)::value, decltype(K)::value>), grid,
                               dim3(NT), 0, s, a);
        });
        return hipGetLastError();
    });
}

template <class E, class R> hipError_t add_bwd(const NormArgs& a0, hipStream_t s) {
    constexpr int VEC = sizeof(R) == 4 ? 4 : 8;
    NormArgs a = a0;
    int blocks = 1;
    const hipError_t e = split_rows<false, true, VEC>((a.D + VEC - 1) / VEC, [&](auto T, auto N) {
        constexpr int TPR = decltype(T)::value, NV = decltype(N)::value, BT = TPR > BWD_THREADS ? TPR : BWD_THREADS;
        blocks = bwd_blocks(a, BT / TPR, TPR * NV > 512);
        by_branch(a, [&](auto S, auto K) {
            hipLaunchKernelGGL((add_norm_bwd_kernel<E, R, VEC, TPR, NV, decltype(S)::value, decltype(K)::value, BT>),
                               dim3(blocks), dim3(BT), 0, s, a);
        });
        return hipGetLastError();
    });
    return e != hipSuccess ? e : norm_wsum(a, blocks, s);
}

}  // namespace

// Enough for every type and both norms: with vectors of 4 a row has the most lanes,
// and a workgroup the fewest rows at a time.
size_t norm_part_floats(long rows, int D) {
    int per = 1;
    (void)split_rows<false, true, 4>((D + 3) / 4, [&](auto T, auto) {
        constexpr int TPR = decltype(T)::value;
        per = (TPR > BWD_THREADS ? TPR : BWD_THREADS) / TPR;
        return hipSuccess;
    });
    const long n = (rows + per - 1) / per;
    if (n <= SOLO) return 0;
    return (size_t)grid_rows(rows, 1, MAX_BWD_BLOCKS) * D * 2;
}

hipError_t norm_wsum(const NormArgs& a, int blocks, hipStream_t s) {
    if (blocks == 1) return hipSuccess;
    hipLaunchKernelGGL(norm_wsum_kernel, dim3((a.pitch + 15) / 16), dim3(1024), 0, s, a.part, blocks, a.pitch, a.D,
                       a.dw, a.dscale);
    return hipGetLastError();
}
hipError_t norm_zero_grads(const NormArgs& a, hipStream_t s) {   // no rows: the column sums are zero
    hipLaunchKernelGGL(zero_kernel, dim3((a.D + 255) / 256), dim3(256), 0, s, a.dw, a.dscale, a.D);
    return hipGetLastError();
}

#define BY_TYPES(F, a, s)                                                                      \
    switch (a.dtype) {                                                                         \
        case GDR_F32: return F<float, float>(a, s);                                            \
        case GDR_F16: return a.res_dtype == GDR_F32 ? F<f16, float>(a, s) : F<f16, f16>(a, s); \
        default: return a.res_dtype == GDR_F32 ? F<bf16, float>(a, s) : F<bf16, bf16>(a, s);   \
    }

hipError_t launch_add_norm_fwd(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    BY_TYPES(add_fwd, a, s)
}
hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return norm_zero_grads(a, s);
    BY_TYPES(add_bwd, a, s)
}

}  // namespace layer

// glr.hip -- the per-channel gated linear recurrence, forward and backward
// (include/gdn_layer.h).
//
// Forward, per sequence and channel, a_t = exp(g_t):
//   h_t = a_t h_{t-1} + x_t,   h_{-1} = h0
// Backward, lambda_t the gradient of h_t:
//   lambda_t = dh_t + a_{t+1} lambda_{t+1}   (dht added at the last token)
//   dx_t = lambda_t,  dg_t = lambda_t a_t h_{t-1},  dh0 = a_0 lambda_0
// The states are carried in fp32; h, dx are rounded once.
// The backward recomputes h_{t-1} from the states that the forward saved at
// every GLR_TILE tokens, not from the rounded h: dg is an fp32 output.
#include "../../include/gdn_layer.h"
#include "gdr_device.hpp"
#include "layer_launch.hpp"

namespace layer {
namespace {

using gdr::bf16;
using gdr::f16;
constexpr int L = GLR_TILE;

// A lane walks one channel of one sequence in time order.
template <class E>
__global__ __launch_bounds__(64) void glr_walk_fwd_kernel(GlrArgs a) {
    const int nb = (a.D + 63) / 64;
    const int n = blockIdx.x / nb, c = blockIdx.x % nb * 64 + threadIdx.x;
    if (c >= a.D) return;
    const long t0 = a.cu ? a.cu[n] : (long)n * a.T, t1 = a.cu ? a.cu[n + 1] : t0 + a.T;
    float h = a.h0 ? a.h0[(long)n * a.D + c] : 0.f;
    for (long t = t0; t < t1; t++) {
        if (a.states && t % L == 0) a.states[t / L * a.D + c] = h;
        h = expf(a.g[t * a.D + c]) * h + (float)((const E*)a.x)[t * a.D + c];
        ((E*)a.h)[t * a.D + c] = (E)h;
    }
    if (a.ht) a.ht[(long)n * a.D + c] = h;
}

template <class E>
__global__ __launch_bounds__(64) void glr_walk_bwd_kernel(GlrArgs a) {
    const int nb = (a.D + 63) / 64;
    const int n = blockIdx.x / nb, c = blockIdx.x % nb * 64 + threadIdx.x;
    if (c >= a.D) return;
    const long t0 = a.cu ? a.cu[n] : (long)n * a.T, t1 = a.cu ? a.cu[n + 1] : t0 + a.T;
    float mu = a.dht ? a.dht[(long)n * a.D + c] : 0.f;   // a_{t+1} lambda_{t+1}
    for (long t = t1; t > t0;) {
        const long b = (t - 1) / L * L, s = b > t0 ? b : t0;   // tokens [s, t) lie in one tile
        float h = s > t0 ? a.states[s / L * a.D + c] : a.h0 ? a.h0[(long)n * a.D + c] : 0.f;
        float al[L], hp[L];
#pragma unroll
        for (int i = 0; i < L; i++)
            if (s + i < t) {
                al[i] = expf(a.g[(s + i) * a.D + c]);
                hp[i] = h;
                h = al[i] * h + (float)((const E*)a.x)[(s + i) * a.D + c];
            }
#pragma unroll
        for (int i = L - 1; i >= 0; i--)
            if (s + i < t) {
                const float lam = (float)((const E*)a.dh)[(s + i) * a.D + c] + mu;
                mu = al[i] * lam;
                ((E*)a.dx)[(s + i) * a.D + c] = (E)lam;
                a.dg[(s + i) * a.D + c] = mu * hp[i];
            }
        t = s;
    }
    if (a.dh0) a.dh0[(long)n * a.D + c] = mu;
}

template <class E> hipError_t fwd(const GlrArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((glr_walk_fwd_kernel<E>), dim3((unsigned)a.nseq * ((a.D + 63) / 64)), dim3(64), 0, s, a);
    return hipGetLastError();
}
template <class E> hipError_t bwd(const GlrArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((glr_walk_bwd_kernel<E>), dim3((unsigned)a.nseq * ((a.D + 63) / 64)), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t glr_ws_bytes(const GlrArgs&) { return 0; }

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) {
    switch (a.dtype) {
        case GDR_F32: return fwd<float>(a, s);
        case GDR_F16: return fwd<f16>(a, s);
        default: return fwd<bf16>(a, s);
    }
}
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s) {
    switch (a.dtype) {
        case GDR_F32: return bwd<float>(a, s);
        case GDR_F16: return bwd<f16>(a, s);
        default: return bwd<bf16>(a, s);
    }
}

}  // namespace layer

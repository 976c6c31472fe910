// layer_dropout.hip -- dropout with a mask that is computed where it is needed
// (include/gdn_layer.h): y = x / (1 - p) where the generator keeps the element,
// else 0 (also for an infinite or NaN x).  Its gradient is the same call on dy.
//
// One read, one write: bound by HBM (32768 x 2048 bf16: 42.5 us, 6.3 TB/s, 65536 x 2048 80,
// 6.7).  Past what the chip's 256 MB cache helps with the rate falls, to 4.5 TB/s at 262144 x 2048
// (473 us) and 4.6 to 5.0 in fp32, where an elementwise copy keeps 6.2.  A lane takes the 8 elements
// of one generator call, 16 or 32 bytes.
#include "layer_dropout.hpp"

namespace layer {
namespace {

// WHOLE: D is a multiple of 8, groups lie one after another.
template <class E, bool WHOLE>
__global__ __launch_bounds__(256) void dropout_kernel(const E* x, E* y, int64_t rows, int64_t D, int64_t groups, Drop d) {
    constexpr int V = 16 / sizeof(E);   // elements in 16 bytes
    typedef typename VecU<E, V>::t Vec;
    const Keep keep(d);
    const int64_t total = rows * groups;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        int64_t at = 8 * i;
        int n = 8;
        if constexpr (!WHOLE) {
            const int64_t row = total >> 32 ? i / groups : (int64_t)((uint32_t)i / (uint32_t)groups), c = 8 * (i - row * groups);
            at = row * D + c;
            n = D - c < 8 ? (int)(D - c) : 8;
        }
        uint32_t w[4];
        E v[8];
        if (WHOLE || n == 8) {
#pragma unroll
            for (int j = 0; j < 8 / V; j++) {
                const Vec t = __builtin_nontemporal_load((const Vec*)(x + at) + j);
#pragma unroll
                for (int e = 0; e < V; e++) v[j * V + e] = t[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = e < n ? x[at + e] : (E)0.f;
        }
        keep.bits((uint64_t)i, w);
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = keep.kept(w, e) ? (E)((float)v[e] * keep.mul) : (E)0.f;
        if (WHOLE || n == 8) {
#pragma unroll
            for (int j = 0; j < 8 / V; j++) {
                Vec t;
#pragma unroll
                for (int e = 0; e < V; e++) t[e] = v[j * V + e];
                __builtin_nontemporal_store(t, (Vec*)(y + at) + j);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (e < n) y[at + e] = v[e];
        }
    }
}

template <class E> hipError_t run(const void* x, void* y, int64_t rows, int64_t D, const Drop& d, hipStream_t s) {
    const int64_t groups = (D + 7) / 8, blocks = (rows * groups + 255) / 256;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (D % 8 == 0)
        hipLaunchKernelGGL((dropout_kernel<E, true>), grid, dim3(256), 0, s, (const E*)x, (E*)y, rows, D, groups, d);
    else
        hipLaunchKernelGGL((dropout_kernel<E, false>), grid, dim3(256), 0, s, (const E*)x, (E*)y, rows, D, groups, d);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(int dtype, const void* x, void* y, int64_t rows, int64_t D, const Drop& d, hipStream_t s) {
    switch (dtype) {
        case GDR_F32: return run<float>(x, y, rows, D, d, s);
        case GDR_F16: return run<f16>(x, y, rows, D, d, s);
        default: return run<bf16>(x, y, rows, D, d, s);
    }
}

}  // namespace layer

// ffn.hip -- the launches of the feed-forward block's products as planned (ffn_plan.hpp), and the
// copy into padded rows.
#include "ffn_launch.hpp"
#include "../../include/gdr.h"

namespace ffn {

hipError_t launch_gemm(int dtype, Kind kind, GemmArgs a, hipStream_t s) {
    if (a.M == 0 || a.N == 0) return hipSuccess;
    const Shape sh = shape_of(kind, a.M, a.N, a.K, dtype == GDR_F32 ? 4 : 2);
    a.tilesM = sh.tilesM, a.tilesN = sh.tilesN, a.splits = sh.splits, a.steps = sh.steps;
    switch (dtype) {
        case GDR_F32: return gemm_f32(kind, a, sh.cfg, s);
        case GDR_F16: return gemm_f16(kind, a, sh.cfg, s);
        default: return gemm_bf16(kind, a, sh.cfg, s);
    }
}

hipError_t launch_grads(int dtype, const GradPlan& plan, const GemmArgs (&g)[3], const bool (&want)[3], float* part,
                        hipStream_t s) {
    GradArgs p{};
    int at = 0;
    for (int i = 0; i < 3; i++) {
        const int j = plan.order[i];
        const Shape& x = plan.s[i];
        GemmArgs& a = p.g[i];
        a = g[j];
        p.dx[i] = j == 0;
        p.start[i] = at;
        if (!want[j] || a.M == 0) continue;
        a.tilesM = x.tilesM, a.tilesN = x.tilesN, a.splits = x.splits, a.steps = x.steps;
        if (a.splits > 1) a.part = part, part += (size_t)a.splits * a.M * a.N;
        at += (a.tilesM * a.tilesN * a.splits + 7) / 8 * 8;
    }
    p.start[3] = at;
    if (at == 0) return hipSuccess;
    switch (dtype) {
        case GDR_F32: return grads_f32(p, plan.cfg, s);
        case GDR_F16: return grads_f16(p, plan.cfg, s);
        default: return grads_bf16(p, plan.cfg, s);
    }
}

namespace {
// A lane writes 16 bytes of a padded row.
template <class U> __global__ __launch_bounds__(256) void ffn_pad_kernel(PadArgs a) {
    constexpr int V = 16 / sizeof(U);
    typedef U Vec __attribute__((ext_vector_type(V)));
    typedef U Loose __attribute__((ext_vector_type(V), aligned(sizeof(U))));
    const PadItem& it = a.item[blockIdx.y];
    const int per = it.cols_dst / V;
    const int64_t total = it.rows_dst * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = total >> 32 ? i / per : (int64_t)((uint32_t)i / (uint32_t)per);
        const int c = (int)(i - r * per) * V;
        const U* src = (const U*)it.src + r * it.cols + c;
        Vec v;
        if (r < it.rows && c + V <= it.cols) {
            const Loose t = *(const Loose*)src;
#pragma unroll
            for (int e = 0; e < V; e++) v[e] = t[e];
        } else {
#pragma unroll
            for (int e = 0; e < V; e++) v[e] = r < it.rows && c + e < it.cols ? src[e] : (U)0;
        }
        ((Vec*)it.dst)[i] = v;
    }
}
}  // namespace

hipError_t launch_pad(int esize, const PadArgs& a, hipStream_t s) {
    int64_t most = 1;
    for (int i = 0; i < a.n; i++) {
        const int64_t n = (a.item[i].rows_dst * a.item[i].cols_dst * esize / 16 + 255) / 256;
        if (n > most) most = n;
    }
    const dim3 grid((unsigned)(most < 4096 ? most : 4096), a.n);
    if (esize == 4) hipLaunchKernelGGL(ffn_pad_kernel<uint32_t>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(ffn_pad_kernel<uint16_t>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace ffn

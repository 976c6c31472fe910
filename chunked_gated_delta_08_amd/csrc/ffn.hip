// ffn.hip -- which tile and how many splits a product of the feed-forward block takes, and the
// copy into padded rows.
#include "ffn_launch.hpp"
#include "../../include/gdr.h"

namespace ffn {

Shape shape_of(Kind kind, int M, int N, int K, int esize) {
    static const int bm[] = {256, 128, 64, 32}, bn[] = {256, 128, 64, 64};
    const int ke = 128 / esize, all = (K + ke - 1) / ke;
    auto tiles = [&](int c) {
        const int bt = kind == GATE_UP ? bn[c] / 2 : bn[c];
        return (int64_t)((M + bm[c] - 1) / bm[c]) * ((N + bt - 1) / bt);
    };
    int c = M <= 32 ? 3 : M <= 64 ? 2 : tiles(0) >= 192 ? 0 : 1;
    if (c == 1 && tiles(1) < 128) c = 2;
    Shape s{};
    s.cfg = c, s.bm = bm[c], s.bn = bn[c];
    const int bt = kind == GATE_UP ? s.bn / 2 : s.bn;
    s.tilesM = (M + s.bm - 1) / s.bm, s.tilesN = (N + bt - 1) / bt;
    int64_t want = c == 0 ? 1 : 512 / tiles(c);
    if (want > all / 4) want = all / 4;
    if (want > 16) want = 16;
    if (want < 1) want = 1;
    s.steps = (int)((all + want - 1) / want);
    s.splits = s.steps ? (all + s.steps - 1) / s.steps : 1;
    return s;
}

size_t part_floats(Kind kind, int M, int N, int K, int esize) {
    const Shape s = shape_of(kind, M, N, K, esize);
    return s.splits > 1 ? (size_t)s.splits * M * N * (kind == GATE_UP ? 2 : 1) : 0;
}

hipError_t launch_gemm(int dtype, Kind kind, GemmArgs a, hipStream_t s) {
    if (a.M == 0 || a.N == 0) return hipSuccess;
    const Shape sh = shape_of(kind, a.M, a.N, a.K, dtype == GDR_F32 ? 4 : 2);
    a.tilesM = sh.tilesM, a.tilesN = sh.tilesN, a.splits = sh.splits, a.steps = sh.steps;
    switch (dtype) {
        case GDR_F32: return gemm_f32(kind, a, sh, s);
        case GDR_F16: return gemm_f16(kind, a, sh, s);
        default: return gemm_bf16(kind, a, sh, s);
    }
}

namespace {
template <class U> __global__ __launch_bounds__(256) void ffn_pad_kernel(PadArgs a) {
    const PadItem& it = a.item[blockIdx.y];
    const int64_t total = it.rows_dst * it.cols_dst;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / it.cols_dst;
        const int c = (int)(i - r * it.cols_dst);
        ((U*)it.dst)[i] = r < it.rows && c < it.cols ? ((const U*)it.src)[r * it.cols + c] : (U)0;
    }
}
}  // namespace

hipError_t launch_pad(int esize, const PadArgs& a, hipStream_t s) {
    int64_t most = 1;
    for (int i = 0; i < a.n; i++) {
        const int64_t n = (a.item[i].rows_dst * a.item[i].cols_dst + 1023) / 1024;
        if (n > most) most = n;
    }
    const dim3 grid((unsigned)(most < 4096 ? most : 4096), a.n);
    if (esize == 4) hipLaunchKernelGGL(ffn_pad_kernel<uint32_t>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(ffn_pad_kernel<uint16_t>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace ffn

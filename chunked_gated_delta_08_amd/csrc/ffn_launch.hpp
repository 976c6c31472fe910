// ffn_launch.hpp -- host-side launchers of the gated feed-forward block
// (include/gdn_ffn.h; internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ffn_plan.hpp"

namespace ffn {

// One product out[m][n] = sum_k Q[m][k] P[n][k].  Leading dimensions are in
// elements; every row that is read begins on 16 bytes.
struct GemmArgs {
    const void* q; int64_t ldq;                     // Q stored [m][k], or [k][m]
    const void* p0; const void* p1; int64_t ldp;    // P stored [n][k], or [k][n]; the second matrix of a pair
    int psplit;                                     // P stored [k][n]: rows from psplit on are p1's
    int M, N, K;                                    // N of one matrix of a pair
    int rowsP;                                      // gate and up, down, dh: columns n that exist, up to 7 fewer than N
    int tilesM, tilesN, splits, steps;              // steps: k-steps of a split
    float* part;                                    // splits > 1: sums of each split, [split][M][width of a row]
    // epilogue
    void* out0; void* out1; int64_t ldo;            // plain: rows from osplit on are out1's
    int osplit, rows_out, cols_out;                 // rows of each that exist, columns that exist
    float* gu;                                      // gate and up before the activation, [M][2 N]
    void* h; void* dgu;                             // act(gate) up [M][N], and the gradients of gate and up [M][2 N]
    int act;
};

// The products dx, dw of gate and up, dw of down, in any order: where each begins in the grid, and its end.
struct GradArgs {
    GemmArgs g[3];
    bool dx[3];
    int start[4];
};

// A tensor to copy into rows of another length: dst[r][c] = src[r][c] where that exists, else zero.
struct PadItem {
    const void* src; void* dst;
    int64_t rows, rows_dst;
    int cols, cols_dst;
};
struct PadArgs {
    PadItem item[5];
    int n;
};

hipError_t launch_gemm(int dtype, Kind kind, GemmArgs a, hipStream_t s);

hipError_t launch_grads(int dtype, const GradPlan& p, const GemmArgs (&g)[3], const bool (&want)[3], float* part,
                        hipStream_t s);
hipError_t launch_pad(int esize, const PadArgs& a, hipStream_t s);

#define FFN_TYPE(T)                                                                      \
    hipError_t gemm_##T(Kind kind, const GemmArgs& a, int cfg, hipStream_t s);           \
    hipError_t grads_##T(const GradArgs& p, int cfg, hipStream_t s);
FFN_TYPE(bf16)
FFN_TYPE(f16)
FFN_TYPE(f32)
#undef FFN_TYPE

}  // namespace ffn

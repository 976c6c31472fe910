// ffn_plan.hpp -- host-side plan of the gated feed-forward block's products
// (include/gdn_ffn.h; internal): plain C++, nothing of HIP.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace ffn {

enum Kind { GATE_UP, DOWN, DH, DX, DW };            // which product: orientations and epilogue

// Tile shape and number of splits along k of a product.
enum Config { BIG, WIDE, MIDDLE, DEEP, LOW, SMALL, THIN, TILES };
struct Shape {
    int cfg, splits, steps, tilesM, tilesN;
};
Shape shape_of(Kind kind, int M, int N, int K, int esize);
size_t part_floats(Kind kind, int M, int N, int K, int esize);

// The gradients' products: 0 dx, 1 dw of gate and up, 2 dw of down, in one launch and in this order.
struct GradPlan {
    int cfg;
    Shape s[3];
    int order[3];
};
GradPlan grad_plan(int T, int D, int F, int esize);
size_t grad_floats(const GradPlan& p, int T, int D, int F);

}  // namespace ffn

// The feed-forward block's planner (csrc/ffn_plan.cpp) for the host compiler, with C entries.
#include "../chunked_gated_delta_08_amd/csrc/ffn_plan.cpp"

static int* put(int* out, const ffn::Shape& s) {
    *out++ = s.cfg, *out++ = s.splits, *out++ = s.steps, *out++ = s.tilesM, *out++ = s.tilesN;
    return out;
}
extern "C" void ffn_plan_one(int kind, int M, int N, int K, int esize, int* out) {
    put(out, ffn::shape_of((ffn::Kind)kind, M, N, K, esize));
}
// dx, dw of gate and up, dw of down
extern "C" void ffn_plan_grads(int T, int D, int F, int esize, int* out) {
    const ffn::GradPlan p = ffn::grad_plan(T, D, F, esize);
    for (int i = 0; i < 3; i++) put(out + 5 * p.order[i], p.s[i]), out[5 * p.order[i]] = p.cfg;
}

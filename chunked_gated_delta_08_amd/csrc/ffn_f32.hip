// ffn_f32.hip -- the feed-forward block's matrix products (ffn_gemm.hpp) in this type.
#include "ffn_gemm.hpp"

namespace ffn {
hipError_t gemm_f32(Kind kind, const GemmArgs& a, int cfg, hipStream_t s) { return run_gemm<float>(kind, a, cfg, s); }
hipError_t grads_f32(const GradArgs& p, int cfg, hipStream_t s) { return run_grads<float>(p, cfg, s); }
}  // namespace ffn

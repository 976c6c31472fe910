// ffn_f16.hip -- the feed-forward block's matrix products (ffn_gemm.hpp) in this type.
#include "ffn_gemm.hpp"

namespace ffn {
hipError_t gemm_f16(Kind kind, const GemmArgs& a, int cfg, hipStream_t s) { return run_gemm<f16>(kind, a, cfg, s); }
hipError_t grads_f16(const GradArgs& p, int cfg, hipStream_t s) { return run_grads<f16>(p, cfg, s); }
}  // namespace ffn

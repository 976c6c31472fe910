// ffn_bf16.hip -- the feed-forward block's matrix products (ffn_gemm.hpp) in this type.
#include "ffn_gemm.hpp"

namespace ffn {
hipError_t gemm_bf16(Kind kind, const GemmArgs& a, int cfg, hipStream_t s) { return run_gemm<bf16>(kind, a, cfg, s); }
hipError_t grads_bf16(const GradArgs& p, int cfg, hipStream_t s) { return run_grads<bf16>(p, cfg, s); }
}  // namespace ffn

// ffn_f32.hip -- the feed-forward block's matrix products (ffn_gemm.hpp) in this type.
#include "ffn_gemm.hpp"

namespace ffn {
hipError_t gemm_f32(Kind kind, const GemmArgs& a, const Shape& sh, hipStream_t s) {
    return run_gemm<float>(kind, a, sh.cfg, s);
}
}  // namespace ffn

// Cross attention for head_dim 64.
#include "cross_tc.cuh"

namespace pkv {
int launch_cross_d64(const AttnParams& p, const CrossArgs& c, int q_dtype, int kv_dtype, int ctas,
                     cudaStream_t stream) {
  return cross_tc::launch_cross_dim<64>(p, c, q_dtype, kv_dtype, ctas, stream);
}
}  // namespace pkv

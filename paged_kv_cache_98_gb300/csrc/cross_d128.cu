// Cross attention for head_dim 128.
#include "cross_tc.cuh"

namespace pkv {
int launch_cross_d128(const AttnParams& p, const CrossArgs& c, int q_dtype, int kv_dtype, int ctas,
                      cudaStream_t stream) {
  return cross_tc::launch_cross_dim<128>(p, c, q_dtype, kv_dtype, ctas, stream);
}
}  // namespace pkv

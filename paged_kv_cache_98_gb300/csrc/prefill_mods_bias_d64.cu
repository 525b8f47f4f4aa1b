// Biased chunked prefill with a distance bias, head_dim 64.
#include "prefill_mods.cuh"

namespace pkv {
int launch_prefill_bias_d64(const AttnParams& p, int q_dtype, int kv_dtype, int total_q,
                            cudaStream_t stream) {
  return pre_mods::launch_mods_dim<pre_mods::kModBias, 64>(p, q_dtype, kv_dtype, total_q,
                                      stream);
}
}  // namespace pkv

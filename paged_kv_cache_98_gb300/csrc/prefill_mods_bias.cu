// Biased chunked prefill with a distance bias.
#include "prefill_mods.cuh"

namespace pkv {
int launch_prefill_bias(const AttnParams& p, int q_dtype, int kv_dtype, int total_q,
                       cudaStream_t stream) {
  return pre_mods::launch_mods_typed<pre_mods::kModBias>(p, q_dtype, kv_dtype, total_q, stream);
}
}  // namespace pkv

// Biased chunked prefill with key intervals alone, head_dim 128.
#include "prefill_mods.cuh"

namespace pkv {
int launch_prefill_keys_d128(const AttnParams& p, int q_dtype, int kv_dtype, int total_q,
                             cudaStream_t stream) {
  return pre_mods::launch_mods_dim<0, 128>(p, q_dtype, kv_dtype, total_q,
                                      stream);
}
}  // namespace pkv

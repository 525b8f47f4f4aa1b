// Biased chunked prefill: which calls it takes, and the choice of the kernel (one
// translation unit per set of modifiers and head dimension).

#include "common.cuh"
#include "launch.h"

namespace pkv {

bool prefill_mods_supported(const AttnParams& p) {
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  // items are counted in 32 bits, and so are the rows of the tensor maps
  return p.group <= 16 && kv_rows + 16 < (1ull << 31) &&
         (uint64_t)p.num_rows * p.num_heads < (1ull << 31) && tmap_available();
}

int launch_prefill_mods(const AttnParams& p, int q_dtype, int kv_dtype, int head_dim, int total_q,
                        cudaStream_t stream) {
  const int mods = (p.softcap > 0.0f ? 1 : 0) | (p.alibi ? 2 : 0);
  using Launch = int (*)(const AttnParams&, int, int, int, cudaStream_t);
  static const Launch d64[4] = {launch_prefill_keys_d64, launch_prefill_cap_d64,
                                launch_prefill_bias_d64, launch_prefill_cap_bias_d64};
  static const Launch d128[4] = {launch_prefill_keys_d128, launch_prefill_cap_d128,
                                 launch_prefill_bias_d128, launch_prefill_cap_bias_d128};
  return (head_dim == 64 ? d64 : d128)[mods](p, q_dtype, kv_dtype, total_q, stream);
}

}  // namespace pkv

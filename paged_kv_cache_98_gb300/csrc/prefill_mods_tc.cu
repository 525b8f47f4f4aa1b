// Biased chunked prefill: choice of the kernel, and the key-interval-only one.

#include "prefill_mods.cuh"

namespace pkv {

bool prefill_mods_supported(const AttnParams& p, int head_dim) {
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  // items are counted in 32 bits, and so are the rows of the tensor maps
  return head_dim == pre_tc::kD && p.group <= 16 && kv_rows + 16 < (1ull << 31) &&
         2 * (uint64_t)p.num_rows * p.num_heads < (1ull << 31) && tmap_available();
}

int launch_prefill_mods(const AttnParams& p, int q_dtype, int kv_dtype, int total_q,
                        cudaStream_t stream) {
  if (p.softcap > 0.0f)
    return p.alibi ? launch_prefill_cap_bias(p, q_dtype, kv_dtype, total_q, stream)
                   : launch_prefill_cap(p, q_dtype, kv_dtype, total_q, stream);
  return p.alibi ? launch_prefill_bias(p, q_dtype, kv_dtype, total_q, stream)
                 : pre_mods::launch_mods_typed<0>(p, q_dtype, kv_dtype, total_q, stream);
}

}  // namespace pkv

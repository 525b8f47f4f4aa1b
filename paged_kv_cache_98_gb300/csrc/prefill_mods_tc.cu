// Biased chunked prefill: choice of the kernel, and the key-interval-only one.

#include "prefill_mods.cuh"

namespace pkv {

bool prefill_mods_supported(const AttnParams& p, int head_dim) {
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  // items are counted in 32 bits, and so are the rows of the tensor maps
  return head_dim == pre_tc::kD && p.group <= 16 && kv_rows + 16 < (1ull << 31) &&
         2 * (uint64_t)p.num_rows * p.num_heads < (1ull << 31) && tmap_available();
}

int launch_prefill_mods(const AttnParams& p, int q_dtype, int kv_dtype, int total_q, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  AttnParams c = p;
  const uint8_t* q8 = nullptr;
  if (kv_dtype == PKV_FP8_E4M3) {
    const int rc = launch_split_query(p, q_dtype, total_q, workspace, workspace_bytes, true, &q8,
                                      &c.q8_scale, stream);
    if (rc != PKV_OK) return rc;
  }
  if (p.softcap > 0.0f)
    return p.alibi ? launch_prefill_cap_bias(c, q_dtype, total_q, q8, stream)
                   : launch_prefill_cap(c, q_dtype, total_q, q8, stream);
  return p.alibi ? launch_prefill_bias(c, q_dtype, total_q, q8, stream)
                 : pre_mods::launch_mods_typed<0>(c, q_dtype, total_q, q8, stream);
}

}  // namespace pkv

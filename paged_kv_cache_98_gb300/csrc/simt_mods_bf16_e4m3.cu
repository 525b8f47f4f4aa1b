// CUDA-core paged attention under score modifiers: q BF16, cache E4M3.
#include "decode_simt.cuh"

namespace pkv {
int launch_simt_mods_bf16_e4m3(const AttnParams& p, int head_dim, int g_pad, cudaStream_t s) {
  return launch_simt_typed<BF16, E4M3, true>(p, head_dim, g_pad, s);
}
}  // namespace pkv

// Grouped-query paged decode on tcgen05 under score modifiers: the biased
// instantiations of the kernel in decode_tc.cuh.

#include "decode_tc_launch.cuh"

namespace pkv {
namespace {

template <class QT, bool FP8>
int launch(const AttnParams& p, cudaStream_t stream) {
  if (p.group > 8) return launch_tc_typed<QT, true, FP8, 16, true>(p, stream, false);
  if (p.group > 4) return launch_tc_typed<QT, false, FP8, 8, true>(p, stream, false);
  return launch_tc_typed<QT, false, FP8, 4, true>(p, stream, false);
}

}  // namespace

int launch_paged_decode_mods(const AttnParams& p, int q_dtype, int kv_dtype, cudaStream_t stream) {
  const bool fp8 = kv_dtype == PKV_FP8_E4M3;
  if (q_dtype == PKV_BF16) return fp8 ? launch<BF16, true>(p, stream) : launch<BF16, false>(p, stream);
  return fp8 ? launch<F16, true>(p, stream) : launch<F16, false>(p, stream);
}

}  // namespace pkv

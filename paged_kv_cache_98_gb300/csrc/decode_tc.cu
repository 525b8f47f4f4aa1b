// Grouped-query paged decode on tcgen05: the kernel and its launcher.  The
// device code (design notes, layouts, roles) is in decode_tc.cuh, shared with
// the fused mixed-batch kernel.

#include "decode_tc_launch.cuh"

namespace pkv {
bool tc_decode_supported(const AttnParams& p, int q_dtype, int kv_dtype, int head_dim) {
  if (head_dim != dec_tc::kD || (kv_dtype != q_dtype && kv_dtype != PKV_FP8_E4M3)) return false;
  if (p.query_start_loc != nullptr || p.partition != dec_tc::kPart) return false;
  if (p.group < 2 || p.group > 16) return false;
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  if (kv_rows + 16 >= (1ull << 31)) return false;
  if ((uint64_t)p.num_rows * p.num_heads + 16 >= (1ull << 31)) return false;
  if ((long long)p.num_rows * p.num_kv_heads * p.max_parts >= (1ll << 31)) return false;
  // the packed per-sequence table holds up to 2^22 (sequence, partition) pairs
  if ((long long)dec_tc::max_seqs(false) * p.max_parts >= (1ll << (31 - dec_tc::kLenBits))) return false;
  return tmap_available();
}

int launch_paged_decode_tc(const AttnParams& p, int q_dtype, int kv_dtype, cudaStream_t stream,
                           bool dependent) {
  if (p.mods) return launch_paged_decode_mods(p, q_dtype, kv_dtype, stream);
  const bool g16 = p.group > 8, g4 = p.group <= 4;
  if (kv_dtype == PKV_FP8_E4M3) {
    if (q_dtype == PKV_BF16)
      return g16  ? launch_tc_typed<BF16, true, true>(p, stream, dependent)
             : g4 ? launch_tc_typed<BF16, false, true, 4>(p, stream, dependent)
                  : launch_tc_typed<BF16, false, true>(p, stream, dependent);
    return g16  ? launch_tc_typed<F16, true, true>(p, stream, dependent)
           : g4 ? launch_tc_typed<F16, false, true, 4>(p, stream, dependent)
                : launch_tc_typed<F16, false, true>(p, stream, dependent);
  }
  if (q_dtype == PKV_BF16)
    return g16  ? launch_tc_typed<BF16, true, false>(p, stream, dependent)
           : g4 ? launch_tc_typed<BF16, false, false, 4>(p, stream, dependent)
                : launch_tc_typed<BF16, false, false>(p, stream, dependent);
  return g16  ? launch_tc_typed<F16, true, false>(p, stream, dependent)
         : g4 ? launch_tc_typed<F16, false, false, 4>(p, stream, dependent)
              : launch_tc_typed<F16, false, false>(p, stream, dependent);
}

}  // namespace pkv

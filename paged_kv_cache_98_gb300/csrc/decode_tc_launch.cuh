// Launcher of the grouped-query paged decode kernel, shared by the plain and the
// biased translation units.
#ifndef PKV_DECODE_TC_LAUNCH_CUH
#define PKV_DECODE_TC_LAUNCH_CUH

#include "decode_tc.cuh"

namespace pkv {
namespace {
using namespace dec_tc;

// kH: heads the softmax computes (4 for groups of at most 4, else all rows)
// kMods: modified scores and first keys (the biased decode)
template <class QT, bool G16, bool FP8, int kH, bool kMods = false>
__global__ void __launch_bounds__(tc_threads(G16, FP8), 1)
    paged_decode_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_q, int kv_rows) {
  extern __shared__ uint8_t smem_raw[];
  // launched as a dependent (cascade decode), this grid does not read its
  // predecessor but ends only after it.  (Letting the merge start early here
  // was measured slower: its resident CTAs slowed the decode.)
  decode_body<QT, G16, FP8, tc_threads(G16, FP8), kH, kMods>(p, tm_k, tm_v, tm_q, kv_rows,
                                                            blockIdx.x, gridDim.x, smem_raw);
  tc::grid_dependency_wait();
}

// ---- host side ---------------------------------------------------------------------------
template <class QT, bool G16, bool FP8, int kH = (G16 ? 16 : 8), bool kMods = false>
int launch_tc_typed(const AttnParams& p, cudaStream_t stream, bool dependent) {
  const bool bf16 = std::is_same<QT, BF16>::value;
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  CUtensorMap tk, tv;
  const bool maps = FP8 ? make_map_e4m3(&tk, p.k_cache, kv_rows, 16) &&
                              make_map_e4m3(&tv, p.v_cache, kv_rows, 16)
                        : make_map_2d(&tk, p.k_cache, kv_rows, bf16, 16) &&
                              make_map_2d(&tv, p.v_cache, kv_rows, bf16, 16);
  if (!maps) return PKV_ERR_CUDA;
  using SM = Smem<G16, FP8, kMods>;
  using L = Layout<G16, FP8, kMods>;
  const size_t smem = sizeof(SM) + 1024;
  static_assert(sizeof(SM) + 1024 <= 232448, "shared memory budget of one CTA");
  static_assert(offsetof(SM, kring) % 1024 == 0 && offsetof(SM, vring) % 1024 == 0 &&
                    offsetof(SM, q) % 1024 == 0 && offsetof(SM, pmat) % 1024 == 0 &&
                    offsetof(SM, tail) % 1024 == 0 && L::kTileBytes % 1024 == 0 &&
                    L::kQHalf % 1024 == 0 && L::kQBytes % 1024 == 0,
                "swizzled buffers must start on 1024-byte boundaries");
  static_assert(L::kStepKeys * L::kRowBytes == kTailBytes, "tail buffer = one MMA step of V");
  auto kern = paged_decode_tc_kernel<QT, G16, FP8, kH, kMods>;
  constexpr int kMaxSeqs = max_seqs(kMods);
  static std::atomic<unsigned long long> configured{0};
  if (!smem_once(kern, smem, configured)) return PKV_ERR_CUDA;
  using OutT = typename QT::T;
  // launches of at most kMaxSeqs sequences each (their rows are independent)
  for (int r0 = 0; r0 < p.num_rows; r0 += kMaxSeqs) {
    AttnParams c = p;
    c.num_rows = p.num_rows - r0 < kMaxSeqs ? p.num_rows - r0 : kMaxSeqs;
    c.num_seqs = c.num_rows;
    const size_t head0 = (size_t)r0 * p.num_heads;
    c.out = static_cast<OutT*>(p.out) + head0 * kD;
    c.q = static_cast<const OutT*>(p.q) + head0 * kD;
    c.block_tables = p.block_tables + (size_t)r0 * p.max_blocks_per_seq;
    c.context_lens = p.context_lens + r0;
    if (p.prefix_lens) c.prefix_lens = p.prefix_lens + r0;
    if (p.key_start) c.key_start = p.key_start + r0;
    if (p.lse) {
      c.lse = p.lse + head0 * p.max_parts;
      c.o_part = p.o_part + head0 * p.max_parts * kD;
    }
    CUtensorMap tq;  // read by TMA on 16-bit caches, unused on E4M3 (split query)
    if (!make_map_2d(&tq, c.q, (uint64_t)c.num_rows * p.num_heads, bf16, L::kRows))
      return PKV_ERR_CUDA;
    const long long items = (long long)c.num_rows * p.num_kv_heads * p.max_parts;
    int grid = sm_count();
    if (items < grid) grid = (int)items;
    if (grid < 1) grid = 1;
    if (dependent && r0 == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(grid);
      cfg.blockDim = dim3(tc_threads(G16, FP8));
      cfg.dynamicSmemBytes = smem;
      cfg.stream = stream;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr.val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (cudaLaunchKernelEx(&cfg, kern, c, tk, tv, tq, (int)kv_rows) != cudaSuccess)
        return PKV_ERR_CUDA;
    } else {
      kern<<<grid, tc_threads(G16, FP8), smem, stream>>>(c, tk, tv, tq, (int)kv_rows);
    }
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  }
  return PKV_OK;
}


}  // namespace
}  // namespace pkv

#endif  // PKV_DECODE_TC_LAUNCH_CUH

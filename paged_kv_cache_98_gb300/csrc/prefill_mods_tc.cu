// Chunked-prefill attention on tcgen05 under score modifiers: the biased mode of
// the kernel in prefill_tc.cuh, and its launcher.

#include "prefill_tc.cuh"

namespace pkv {
namespace {
using namespace pre_tc;

template <class QT, bool kFP8>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_mods_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_q, int kv_rows) {
  extern __shared__ uint8_t smem_raw[];
  prefill_body<QT, false, false, kFP8, true>(p, tm_k, tm_v, tm_q, kv_rows, blockIdx.x, gridDim.x,
                                             smem_raw);
}

template <class QT, bool kFP8>
int launch(const AttnParams& p, int total_q, const uint8_t* q8, cudaStream_t stream) {
  const bool bf16 = std::is_same<QT, BF16>::value;
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  const uint32_t g = (uint32_t)p.group, tokens = kRowsM / g, heads = (uint32_t)p.num_heads;
  CUtensorMap tk, tv, tq;
  const bool maps =
      kFP8 ? make_map_e4m3(&tk, p.k_cache, kv_rows, 16) && make_map_e4m3(&tv, p.v_cache, kv_rows, 16) &&
                 make_map_q3d_e4m3(&tq, q8, 2 * (uint64_t)total_q, heads, g, tokens)
           : make_map_2d(&tk, p.k_cache, kv_rows, bf16, 16) &&
                 make_map_2d(&tv, p.v_cache, kv_rows, bf16, 16) &&
                 make_map_q3d(&tq, p.q, (uint64_t)total_q, heads, bf16, g, tokens);
  if (!maps) return PKV_ERR_CUDA;
  const size_t smem = sizeof(Smem) + 1024;
  auto kern = prefill_mods_kernel<QT, kFP8>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return PKV_ERR_CUDA;
  // launches of at most kMaxSeqs sequences each; their query rows stay absolute
  for (int s0 = 0; s0 < p.num_seqs; s0 += kMaxSeqs) {
    AttnParams c = p;
    c.num_seqs = p.num_seqs - s0 < kMaxSeqs ? p.num_seqs - s0 : kMaxSeqs;
    c.block_tables = p.block_tables + (size_t)s0 * p.max_blocks_per_seq;
    c.context_lens = p.context_lens + s0;
    c.query_start_loc = p.query_start_loc + s0;
    if (p.bidir_lens) c.bidir_lens = p.bidir_lens + s0;
    // an upper bound of the items: every sequence's pairs of query tiles, times the KV heads
    const long long tiles = (total_q + (long long)tokens - 1) / tokens + c.num_seqs;
    const long long items = (tiles + c.num_seqs) / 2 * p.num_kv_heads;
    const int sms = sm_count();
    const int grid = (int)(items < sms ? (items > 0 ? items : 1) : sms);
    kern<<<grid, kThreads, smem, stream>>>(c, tk, tv, tq, (int)kv_rows);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

}  // namespace

bool prefill_mods_supported(const AttnParams& p, int head_dim) {
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  // items are counted in 32 bits, and so are the rows of the tensor maps
  return head_dim == kD && p.group <= 16 && kv_rows + 16 < (1ull << 31) &&
         2 * (uint64_t)p.num_rows * p.num_heads < (1ull << 31) && tmap_available();
}

int launch_prefill_mods(const AttnParams& p, int q_dtype, int kv_dtype, int total_q, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  if (kv_dtype != PKV_FP8_E4M3)
    return q_dtype == PKV_BF16 ? launch<BF16, false>(p, total_q, nullptr, stream)
                               : launch<F16, false>(p, total_q, nullptr, stream);
  AttnParams c = p;
  const uint8_t* q8;
  const int rc = launch_split_query(p, q_dtype, total_q, workspace, workspace_bytes, true, &q8,
                                    &c.q8_scale, stream);
  if (rc != PKV_OK) return rc;
  return q_dtype == PKV_BF16 ? launch<BF16, true>(c, total_q, q8, stream)
                             : launch<F16, true>(c, total_q, q8, stream);
}

}  // namespace pkv

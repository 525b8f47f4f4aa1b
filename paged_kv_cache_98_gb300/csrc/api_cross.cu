// C ABI of cross attention.  Declarations and semantics are in include/pagedkv.h.

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "cross.h"

namespace {

constexpr int kMaxSeqs = 1024;  // of a launch
constexpr int kCtas = 152;      // parts the work of a launch is cut into, at most

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Rows of a partial: those of two query tiles, or where the sequences have one at most,
// of their tokens.
int part_rows(int group, int max_q_len) {
  const int tokens = 128 / group;
  return max_q_len > tokens ? 256 : std::max(max_q_len, 1) * group;
}

// Units of one key tile are never cut.
bool may_cut(int max_encoder_len) { return max_encoder_len > 128; }

constexpr size_t kCutBytes = 2 * kCtas * 16;
static_assert(kCutBytes % 256 == 0, "what follows is aligned");

}  // namespace

extern "C" {

size_t pkv_cross_workspace_size(int num_seqs, int total_q, int num_heads, int num_kv_heads,
                                int head_dim, int max_encoder_len, int max_q_len) {
  if (num_seqs <= 0 || total_q <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_q_len <= 0 || num_heads % num_kv_heads != 0 || num_heads / num_kv_heads > 16 ||
      !may_cut(max_encoder_len))
    return 0;
  const size_t rows = 2 * (size_t)kCtas * part_rows(num_heads / num_kv_heads, std::min(max_q_len, total_q));
  return kCutBytes + round_up(rows * sizeof(float), 256) + rows * head_dim * sizeof(float);
}

int pkv_paged_attention_cross(void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* encoder_lens,
                              const int32_t* query_start_loc, int num_seqs, int total_q,
                              int max_q_len, int num_heads, int num_kv_heads, int head_dim,
                              int block_size, int max_blocks_per_seq, int num_blocks,
                              int max_encoder_len, float scale, pkv_dtype q_dtype,
                              pkv_dtype kv_dtype, float k_scale, float v_scale, void* workspace,
                              size_t workspace_bytes, uint32_t* device_errors, void* stream) {
  if (num_seqs < 0 || total_q < 0 || max_q_len < 0 || max_encoder_len < 0 || num_heads <= 0 ||
      num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_heads % num_kv_heads != 0 || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (!k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(encoder_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(device_errors, 4))
    return PKV_ERR_INVALID_ARG;
  if (block_size != pkv::kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (num_heads / num_kv_heads > 16) return PKV_ERR_UNSUPPORTED;
  if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (kv_dtype != q_dtype && kv_dtype != PKV_FP8_E4M3) return PKV_ERR_UNSUPPORTED;
  const bool fp8 = kv_dtype == PKV_FP8_E4M3;
  if (fp8 && (!(k_scale > 0.0f) || !(v_scale > 0.0f) || !std::isfinite(k_scale) ||
              !std::isfinite(v_scale)))
    return PKV_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * pkv::kBlockSize > (1LL << 30)) return PKV_ERR_UNSUPPORTED;
  const long long cache_rows = (long long)num_blocks * num_kv_heads * pkv::kBlockSize;
  if ((long long)num_blocks * num_kv_heads > 0x7fffffffLL || cache_rows > 0x7fffffffLL ||
      (long long)total_q * num_heads > 0x7fffffffLL)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PKV_OK;
  if (!out || !q || !block_tables || !encoder_lens || !query_start_loc) return PKV_ERR_INVALID_ARG;
  const unsigned long long n = 2ull * total_q * num_heads * head_dim;
  const unsigned long long cb = (unsigned long long)cache_rows * head_dim * (fp8 ? 1 : 2);
  if (pkv::bytes_overlap(out, n, q, n) || pkv::bytes_overlap(out, n, k_cache, cb) ||
      pkv::bytes_overlap(out, n, v_cache, cb))
    return PKV_ERR_INVALID_ARG;
  if (max_q_len == 0) return PKV_OK;  // (no sequence has a query)
  const size_t need = pkv_cross_workspace_size(num_seqs, total_q, num_heads, num_kv_heads, head_dim,
                                               max_encoder_len, max_q_len);
  if (need > 0 && (!workspace || workspace_bytes < need)) return PKV_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return PKV_ERR_INVALID_ARG;
  if (!pkv::tmap_available()) return PKV_ERR_CUDA;
  pkv::AttnParams p = {};
  p.out = out;
  p.q = q;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.num_rows = total_q;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.max_context = max_encoder_len;
  p.q_scale = scale * pkv::kLog2e * (fp8 ? k_scale : 1.0f);
  p.v_scale = fp8 ? v_scale : 1.0f;
  p.errors = device_errors;
  pkv::CrossArgs c = {};
  c.max_q = std::min(max_q_len, total_q);
  c.part_rows = part_rows(p.group, c.max_q);
  c.box_tokens = std::min(128 / p.group, c.max_q);
  if (need > 0) {
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const size_t rows = 2 * (size_t)kCtas * c.part_rows;
    c.cuts = reinterpret_cast<int4*>(w);
    p.lse = reinterpret_cast<float*>(w + kCutBytes);
    p.o_part = reinterpret_cast<float*>(w + kCutBytes + round_up(rows * sizeof(float), 256));
  }
  pkv::take_debug_hook(p);
  const int ctas = std::min(pkv::sm_count(), kCtas);
  for (int s0 = 0; s0 < num_seqs; s0 += kMaxSeqs) {
    p.num_seqs = std::min(num_seqs - s0, kMaxSeqs);
    p.block_tables = block_tables + (size_t)s0 * max_blocks_per_seq;
    p.context_lens = encoder_lens + s0;
    p.query_start_loc = query_start_loc + s0;
    const auto launch = head_dim == 64 ? pkv::launch_cross_d64 : pkv::launch_cross_d128;
    const int rc = launch(p, c, (int)q_dtype, (int)kv_dtype, ctas, static_cast<cudaStream_t>(stream));
    if (rc != PKV_OK) return rc;
  }
  return PKV_OK;
}

}  // extern "C"

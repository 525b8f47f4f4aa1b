// C ABI of the step's preparation: step maps, rotary positions with the cache
// write.  Declarations and semantics are in include/pagedkv.h.

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
  const void* p;
  unsigned long long bytes;
};
bool overlap(const Range& a, const Range& b) {
  return a.bytes > 0 && b.bytes > 0 && pkv::bytes_overlap(a.p, a.bytes, b.p, b.bytes);
}

}  // namespace

extern "C" {

int pkv_build_step_maps(int32_t* block_tables, int32_t* context_lens, int32_t* query_start_loc,
                        int64_t* slot_mapping, int32_t* positions, int32_t* request_tables,
                        const int32_t* rows, const int32_t* cached_lens, const int32_t* q_lens,
                        const int32_t* new_blocks, int num_seqs, int num_request_rows,
                        int max_blocks_per_seq, int num_tokens, int num_new_blocks,
                        int block_size, int num_blocks, uint32_t* device_errors, void* stream) {
  if (num_seqs < 0 || num_request_rows <= 0 || max_blocks_per_seq <= 0 || num_tokens < 0 ||
      num_new_blocks < 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (!query_start_loc) return PKV_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!block_tables || !context_lens || !request_tables || !rows ||
                       !cached_lens || !q_lens))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!slot_mapping || !positions)) return PKV_ERR_INVALID_ARG;
  if (num_new_blocks > 0 && !new_blocks) return PKV_ERR_INVALID_ARG;
  if (!aligned(slot_mapping, 8) || !aligned(block_tables, 4) || !aligned(request_tables, 4) ||
      !aligned(device_errors, 4))
    return PKV_ERR_INVALID_ARG;
  if (block_size != pkv::kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > PKV_STEP_MAPS_MAX_SEQS) return PKV_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * pkv::kBlockSize > (1LL << 30)) return PKV_ERR_UNSUPPORTED;
  // CTAs read the inputs while others write: no output may share memory with an
  // input or with another output (lengths updated in place, tables that are one)
  const unsigned long long S = num_seqs, row = 4ull * max_blocks_per_seq;
  const Range out[] = {{block_tables, S * row}, {context_lens, 4 * S}, {query_start_loc, 4 * (S + 1)},
                       {slot_mapping, 8ull * num_tokens}, {positions, 4ull * num_tokens},
                       {request_tables, S > 0 ? num_request_rows * row : 0}};
  const Range in[] = {{rows, 4 * S}, {cached_lens, 4 * S}, {q_lens, 4 * S}, {new_blocks, 4ull * num_new_blocks}};
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PKV_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i], in[j])) return PKV_ERR_INVALID_ARG;
  }
  return pkv::launch_step_maps(block_tables, context_lens, query_start_loc, slot_mapping,
                               positions, request_tables, rows, cached_lens, q_lens, new_blocks,
                               num_seqs, num_request_rows, max_blocks_per_seq, num_tokens,
                               num_new_blocks, num_blocks, device_errors,
                               static_cast<cudaStream_t>(stream));
}

int pkv_rotary_frequencies(double* inv_freq, int rotary_dim, double base,
                           pkv_rotary_scaling scaling, double factor, double low, double high,
                           int original_len, float* attn_factor_out) {
  const double two_pi = 6.283185307179586476925286766559;
  if (!inv_freq || rotary_dim < 2 || rotary_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
    return PKV_ERR_INVALID_ARG;
  const int kind = (int)scaling;
  if (kind < PKV_ROTARY_PLAIN || kind > PKV_ROTARY_YARN) return PKV_ERR_INVALID_ARG;
  if (kind != PKV_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return PKV_ERR_INVALID_ARG;
  if (kind >= PKV_ROTARY_BANDS &&
      (original_len <= 0 || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return PKV_ERR_INVALID_ARG;
  if (kind == PKV_ROTARY_NTK && rotary_dim > 2)
    base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
  // yarn: the dimension index whose frequency turns r times over original_len
  auto turning = [&](double r) {
    return rotary_dim * std::log(original_len / (r * two_pi)) / (2.0 * std::log(base));
  };
  double ramp0 = 0.0, ramp1 = 0.0;
  if (kind == PKV_ROTARY_YARN) {
    ramp0 = std::fmax(std::floor(turning(high)), 0.0);
    ramp1 = std::fmin(std::ceil(turning(low)), rotary_dim - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double inv = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1.0;  // share of the unscaled frequency
    if (kind == PKV_ROTARY_LINEAR) {
      keep = 0.0;
    } else if (kind == PKV_ROTARY_BANDS) {
      keep = (original_len * inv / two_pi - low) / (high - low);
    } else if (kind == PKV_ROTARY_YARN) {
      keep = ramp1 > ramp0 ? 1.0 - (i - ramp0) / (ramp1 - ramp0) : (i <= ramp0 ? 1.0 : 0.0);
    }
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    inv_freq[i] = kind == PKV_ROTARY_PLAIN || kind == PKV_ROTARY_NTK
                      ? inv
                      : keep * inv + (1.0 - keep) * inv / factor;
  }
  if (attn_factor_out)
    *attn_factor_out = kind == PKV_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return PKV_OK;
}

int pkv_rotary_and_cache(void* q_out, const void* q, const void* k, const void* v, void* k_cache,
                         void* v_cache, const int64_t* slot_mapping, const int32_t* positions,
                         const double* inv_freq, int64_t q_stride, int64_t k_stride,
                         int64_t v_stride, int num_tokens, int num_heads, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, int rotary_dim,
                         pkv_rotary_layout layout, float attn_factor, pkv_dtype src_dtype,
                         pkv_dtype cache_dtype, float k_scale, float v_scale,
                         uint32_t* device_errors, void* stream) {
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (block_size != pkv::kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (src_dtype != PKV_F16 && src_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (cache_dtype != src_dtype && cache_dtype != PKV_FP8_E4M3) return PKV_ERR_UNSUPPORTED;
  if (((long long)num_heads + 2LL * num_kv_heads) * head_dim > (1LL << 24))
    return PKV_ERR_UNSUPPORTED;
  if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2 != 0) return PKV_ERR_INVALID_ARG;
  if (layout != PKV_ROTARY_HALF && layout != PKV_ROTARY_INTERLEAVED) return PKV_ERR_INVALID_ARG;
  if (!std::isfinite(attn_factor)) return PKV_ERR_INVALID_ARG;
  if (cache_dtype == PKV_FP8_E4M3 && (!(k_scale > 0.0f) || !(v_scale > 0.0f) ||
                                      !std::isfinite(k_scale) || !std::isfinite(v_scale)))
    return PKV_ERR_INVALID_ARG;
  if (!inv_freq || !aligned(device_errors, 4)) return PKV_ERR_INVALID_ARG;
  // (the range for which the phases are good to 2^-63 turns)
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!(std::fabs(inv_freq[i]) <= 1.0e3)) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !q || !k || !v || !k_cache || !v_cache || !slot_mapping || !positions)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PKV_ERR_INVALID_ARG;
  const long long qrow = (long long)num_heads * head_dim, krow = (long long)num_kv_heads * head_dim;
  const long long most = 1LL << 40;  // elements between tokens
  if (q_stride < qrow || k_stride < krow || v_stride < krow || q_stride > most ||
      k_stride > most || v_stride > most || q_stride % 8 != 0 || k_stride % 8 != 0 ||
      v_stride % 8 != 0)
    return PKV_ERR_INVALID_ARG;
  // q_out may be q with the same layout; any other overlap would be read after it is written
  const unsigned long long t1 = (unsigned long long)num_tokens - 1;
  const Range ro{q_out, 2 * (t1 + 1) * qrow}, rq{q, 2 * (t1 * q_stride + qrow)};
  const Range rk{k, 2 * (t1 * k_stride + krow)}, rv{v, 2 * (t1 * v_stride + krow)};
  const unsigned long long nc = (unsigned long long)num_blocks * pkv::kBlockSize * krow *
                                (cache_dtype == PKV_FP8_E4M3 ? 1 : 2);
  if (!(q_out == q && q_stride == qrow) && overlap(ro, rq)) return PKV_ERR_INVALID_ARG;
  if (overlap(ro, rk) || overlap(ro, rv)) return PKV_ERR_INVALID_ARG;
  for (const Range& c : {Range{k_cache, nc}, Range{v_cache, nc}})
    if (overlap(c, ro) || overlap(c, rq) || overlap(c, rk) || overlap(c, rv))
      return PKV_ERR_INVALID_ARG;
  if (overlap({k_cache, nc}, {v_cache, nc})) return PKV_ERR_INVALID_ARG;
  pkv::RotaryArgs a{q_out, q, k, v, k_cache, v_cache, slot_mapping, positions,
                    q_stride, k_stride, v_stride, num_tokens, num_heads, num_kv_heads, head_dim,
                    num_blocks, rotary_dim, (int)layout, (int)src_dtype, (int)cache_dtype,
                    attn_factor, k_scale, v_scale, device_errors};
  return pkv::launch_rotary_and_cache(a, inv_freq, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

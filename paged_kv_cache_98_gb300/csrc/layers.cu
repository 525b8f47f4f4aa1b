// Bytes moved in the caches of all layers: whole blocks (the device half of
// copy-on-write) and the kept tokens of a sequence.  Declarations and semantics are in
// include/pagedkv.h.

#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// The caches of a launch: K of every layer, then V.
struct Caches {
  void* p[2 * PKV_LAYERS_PER_LAUNCH];
};

// ---- block copies ------------------------------------------------------------------------
// A CTA copies one block of one cache, eight 16-byte loads a thread in flight before the
// first store (a block of 8 heads of 128 16-bit elements is 32 KB: one such turn).  Bound
// by HBM, 2 x block bytes a pair, layer and cache: 188 MB in 27.8 us, 6.7 TB/s (2.6 us for a few
// pairs of four layers).
__global__ void __launch_bounds__(kThreads)
    copy_layers_kernel(const __grid_constant__ Caches caches, const int32_t* __restrict__ pairs,
                       int num_blocks, long long vecs, uint32_t* errors) {
  const int src = __ldg(pairs + 2 * (size_t)blockIdx.x), dst = __ldg(pairs + 2 * (size_t)blockIdx.x + 1);
  if (src < 0) return;
  if (src >= num_blocks || dst < 0 || dst >= num_blocks) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(errors, PKV_DEVERR_BLOCK_ID);
    return;
  }
  uint4* const cache = static_cast<uint4*>(caches.p[blockIdx.y]);
  const uint4* s = cache + (long long)src * vecs;
  uint4* d = cache + (long long)dst * vecs;
  constexpr int kDeep = 8;
  for (long long j0 = threadIdx.x; j0 < vecs; j0 += kDeep * kThreads) {
    uint4 w[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (j0 + u * kThreads < vecs) w[u] = __ldg(s + j0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (j0 + u * kThreads < vecs) d[j0 + u * kThreads] = w[u];
  }
}

// ---- kept tokens moved together ------------------------------------------------------------
// Token keep[j] of a sequence goes to place base + j.  As the list ascends from base on,
// base + j <= keep[j]: tokens only move towards the front, and a place that the first j
// tokens go to is no source of a later one.  So a unit, the rows of one sequence, cache and
// KV head, can be moved in place by threads that walk its list in ascending turns: all rows
// of a turn are read, then (a barrier) written, and the next turn's reads need no barrier
// behind those writes.  A unit is a warp's where lists are short for how many units there are
// (a drafted path) and a CTA's where they are long.  Bound by HBM, two row bytes a moved
// token (6.4 TB/s with 16 sequences of 8192 tokens, 8 layers), with few units by their turns, one
// after the other (4 sequences of up to 16384 tokens, 2 layers: 105 us, 4.2 TB/s); by launch
// and four dependent reads (list, table, row) for short lists.  (The next turn's rows loaded
// before this one's are stored, in as many or twice the registers: 108 to 116 us.)
constexpr int kDeep = 4;        // rows a thread reads in a turn
// Kept tokens a sequence (on average) from which a CTA moves a unit: one for every kLongUnits
// units, but within the other two.  Measured with a warp and a CTA: 128 units 3.6 and 4.1 us with 8
// kept tokens, 5.0 and 4.0 with 16; 1024 units 5.2 and 6.5 with 16, 7.4 and 7.0 with 32; 2048
// units 13.4 and 14.3 with 64, 23.2 and 22.5 with 128; 4096 units 47 and 54 with 128, 99 and
// 93 with 256.
constexpr int kLongUnits = 20, kLeastLong = 12, kMostLong = 256;
// Below as many, CTAs' units are 64 bytes of each row: 4 x 16384 tokens kept by half in 128 units
// take 105 us instead of 198, 16 x in 512 units 315 instead of 331.
constexpr long long kManyUnits = 608;

struct CompactArgs {
  const int32_t *tables, *context, *base, *starts, *keep;
  int32_t* new_lens;
  const int32_t* counts;
  int num_seqs, num_keep, kv_heads, width, num_blocks;
  int caches;  // of the launch
  int first;   // 1: the launch that writes new_lens and flags lists
  uint32_t* errors;
};

template <int kWarps, int kRowBytes, int kPartBytes>
__global__ void __launch_bounds__(kThreads, 4)
    compact_kernel(const __grid_constant__ Caches caches, const CompactArgs a) {
  constexpr int kUnit = 32 * kWarps;             // threads of a unit
  constexpr int kParts = kRowBytes / kPartBytes; // units that share the rows
  constexpr int kChunks = kPartBytes / 16;       // 16-byte chunks, and threads, of a row
  constexpr int kRows = kUnit / kChunks;         // rows read at once
  __shared__ int s_moved;
  const int t = threadIdx.x % kUnit;
  const long long unit = (long long)blockIdx.x * (kThreads / kUnit) + threadIdx.x / kUnit;
  const int per_seq = a.caches * a.kv_heads * kParts;
  const int s = (int)(unit / per_seq);
  if (s >= a.num_seqs) return;                   // (a CTA's units end together: kWarps = 8 has one)
  const int of = (int)(unit % per_seq), part = of % kParts;
  const int cache = of / kParts / a.kv_heads, head = of / kParts % a.kv_heads;
  auto any = [&](bool x) -> bool {
    if constexpr (kWarps == 1) return __any_sync(kFull, x);
    else return __syncthreads_or(x);
  };
  const bool tell = a.first && of == 0;
  const int cap = a.width * kBlockSize;
  const int ctx = __ldg(a.context + s), base = __ldg(a.base + s);
  const int k0 = __ldg(a.starts + s), k1 = __ldg(a.starts + s + 1);
  const bool fits = ctx >= 0 && ctx <= cap && base >= 0 && base <= ctx && k0 >= 0 && k0 <= k1 &&
                    k1 <= a.num_keep && k1 - k0 <= ctx - base;
  const int n = fits ? k1 - k0 : 0;
  const int32_t* keep = a.keep + (fits ? k0 : 0);
  // the list ascends within [base, ctx); its tokens before `moved` are in place
  bool bad = !fits;
  int moved = n;
#pragma unroll 8
  for (int j = t; j < n; j += kUnit) {
    const int v = __ldg(keep + j), before = j ? __ldg(keep + j - 1) : base - 1;
    bad |= v <= before || v >= ctx;
    if (v != base + j) moved = min(moved, j);
  }
  if constexpr (kWarps == 1) {
    moved = __reduce_min_sync(kFull, moved);
  } else {
    if (t == 0) s_moved = n;
    __syncthreads();
    atomicMin(&s_moved, moved);
    __syncthreads();
    moved = s_moved;
  }
  bad = any(bad);
  const int32_t* table = a.tables + (size_t)s * a.width;
  bool shared = false;
  if (!bad && a.counts && moved < n) {
    const int b1 = (base + n - 1) / kBlockSize;
    for (int b = (base + moved) / kBlockSize + t; b <= b1; b += kUnit) {
      const int blk = __ldg(table + b);
      if (blk >= 0 && blk < a.num_blocks) shared |= __ldg(a.counts + blk) > 1;
    }
  }
  shared = any(shared);
  if (tell && t == 0) {
    if (bad) flag_error(a.errors, PKV_DEVERR_CONTEXT);
    if (shared) flag_error(a.errors, PKV_DEVERR_SHARED);
    a.new_lens[s] = bad || shared ? min(max(ctx, 0), cap) : base + n;
  }
  if (bad || shared) return;
  uint8_t* const rows = static_cast<uint8_t*>(caches.p[cache]) +
                        (size_t)head * (kBlockSize * kRowBytes) + part * kPartBytes +
                        (t % kChunks) * 16;
  const size_t block_bytes = (size_t)a.kv_heads * (kBlockSize * kRowBytes);
  // block and row of the j-th kept token (to: of its new place) as 16 block + row; -1 past the
  // list or in a block outside the pool
  auto slot = [&](int j, bool to) -> int {
    if (j >= n) return -1;
    const int place = to ? base + j : __ldg(keep + j);
    const int blk = __ldg(table + place / kBlockSize);
    if (blk < 0 || blk >= a.num_blocks) {
      if (tell) flag_error(a.errors, PKV_DEVERR_BLOCK_ID);
      return -1;
    }
    return blk * kBlockSize + place % kBlockSize;
  };
  auto at = [&](int s) {
    return reinterpret_cast<uint4*>(rows + (size_t)(s / kBlockSize) * block_bytes + (s % kBlockSize) * kRowBytes);
  };
  // the next turn's places are looked up while a turn's rows are on their way
  int from[kDeep], to[kDeep];
  auto look_up = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      from[u] = slot(j0 + u * kRows, false);
      to[u] = slot(j0 + u * kRows, true);
    }
  };
  int j0 = moved + t / kChunks;
  look_up(j0);
  for (; j0 - t / kChunks < n; j0 += kRows * kDeep) {
    uint4 w[kDeep];
    int dst[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      dst[u] = from[u] < 0 ? -1 : to[u];
      if (dst[u] >= 0) w[u] = *at(from[u]);
    }
    look_up(j0 + kRows * kDeep);
    if constexpr (kWarps == 1) __syncwarp();
    else __syncthreads();
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (dst[u] >= 0) *at(dst[u]) = w[u];
  }
}

template <int kWarps, int kRowBytes, int kPartBytes>
int launch_compact(const Caches& c, const CompactArgs& a, cudaStream_t stream) {
  const long long units = (long long)a.num_seqs * a.caches * a.kv_heads * (kRowBytes / kPartBytes);
  constexpr int kPer = kThreads / (32 * kWarps);
  const long long ctas = (units + kPer - 1) / kPer;
  if (ctas > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  compact_kernel<kWarps, kRowBytes, kPartBytes><<<(unsigned)ctas, kThreads, 0, stream>>>(c, a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int kRowBytes>
int launch_compact_rows(const Caches& c, const CompactArgs& a, cudaStream_t stream) {
  const long long units = (long long)a.num_seqs * a.caches * a.kv_heads;
  if (a.num_keep < std::clamp(units / kLongUnits, (long long)kLeastLong, (long long)kMostLong) * a.num_seqs)
    return launch_compact<1, kRowBytes, kRowBytes>(c, a, stream);
  if constexpr (kRowBytes > 64)
    if (units < kManyUnits)
      return launch_compact<8, kRowBytes, 64>(c, a, stream);
  return launch_compact<8, kRowBytes, kRowBytes>(c, a, stream);
}

// Every cache given, on a 16-byte boundary, and none overlapping another.
int check_caches(void* const* k, void* const* v, int num_layers, unsigned long long bytes) {
  if (!k || !v) return PKV_ERR_INVALID_ARG;
  uintptr_t at[2 * PKV_LAYERS_PER_LAUNCH];
  // (overlaps: of neighbours in the order of their addresses, or of every pair where the array
  // does not hold all caches)
  for (int i = 0; i < 2 * num_layers; ++i) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(i < num_layers ? k[i] : v[i - num_layers]);
    if (!p || (p & 15u)) return PKV_ERR_INVALID_ARG;
    if (i < 2 * PKV_LAYERS_PER_LAUNCH) at[i] = p;
  }
  if (num_layers <= PKV_LAYERS_PER_LAUNCH) {
    std::sort(at, at + 2 * num_layers);
    for (int i = 1; i < 2 * num_layers; ++i)
      if (at[i] - at[i - 1] < bytes) return PKV_ERR_INVALID_ARG;
    return PKV_OK;
  }
  for (int i = 0; i < 2 * num_layers; ++i)
    for (int j = 0; j < i; ++j) {
      const void* p = i < num_layers ? k[i] : v[i - num_layers];
      const void* q = j < num_layers ? k[j] : v[j - num_layers];
      if (bytes_overlap(p, bytes, q, bytes)) return PKV_ERR_INVALID_ARG;
    }
  return PKV_OK;
}

// Layers [l0, l0 + n) as a launch's caches.
Caches caches_of(void* const* k, void* const* v, int l0, int n) {
  Caches c = {};
  for (int i = 0; i < n; ++i) {
    c.p[i] = k[l0 + i];
    c.p[n + i] = v[l0 + i];
  }
  return c;
}

bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_copy_blocks_layers(void* const* k_caches, void* const* v_caches, int num_layers,
                           const int32_t* block_pairs, int num_pairs, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks, pkv_dtype cache_dtype,
                           uint32_t* device_errors, void* stream) {
  using namespace pkv;
  if (num_layers < 0 || num_pairs < 0 || num_kv_heads <= 0 || num_blocks <= 0 || head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_pairs > 0 && !block_pairs) return PKV_ERR_INVALID_ARG;
  if (!words(block_pairs) || !words(device_errors)) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (cache_dtype != PKV_F16 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
    return PKV_ERR_UNSUPPORTED;
  const long long elem = cache_dtype == PKV_FP8_E4M3 ? 1 : 2;
  if ((long long)num_kv_heads * head_dim > (1LL << 24)) return PKV_ERR_UNSUPPORTED;
  const long long block_bytes = (long long)num_kv_heads * block_size * head_dim * elem;
  if (num_layers > 0) {
    const int rc = check_caches(k_caches, v_caches, num_layers,
                                (unsigned long long)block_bytes * num_blocks);
    if (rc != PKV_OK) return rc;
  }
  if (num_pairs == 0) return PKV_OK;
  for (int l0 = 0; l0 < num_layers; l0 += PKV_LAYERS_PER_LAUNCH) {
    const int n = std::min(num_layers - l0, PKV_LAYERS_PER_LAUNCH);
    copy_layers_kernel<<<dim3(num_pairs, 2 * n), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        caches_of(k_caches, v_caches, l0, n), block_pairs, num_blocks, block_bytes / 16,
        device_errors);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

int pkv_compact_tokens(void* const* k_caches, void* const* v_caches, int num_layers,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* base_lens, const int32_t* keep_start_loc,
                       const int32_t* keep, int32_t* new_lens, const int32_t* ref_counts,
                       int num_seqs, int num_keep, int num_kv_heads, int head_dim, int block_size,
                       int max_blocks_per_seq, int num_blocks, pkv_dtype cache_dtype,
                       uint32_t* device_errors, void* stream) {
  using namespace pkv;
  if (num_layers <= 0 || num_seqs < 0 || num_keep < 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!block_tables || !context_lens || !base_lens || !keep_start_loc || !new_lens))
    return PKV_ERR_INVALID_ARG;
  if (num_keep > 0 && !keep) return PKV_ERR_INVALID_ARG;
  if (!words(block_tables) || !words(context_lens) || !words(base_lens) ||
      !words(keep_start_loc) || !words(keep) || !words(new_lens) || !words(ref_counts) ||
      !words(device_errors))
    return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (cache_dtype != PKV_F16 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
    return PKV_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * kBlockSize > (1LL << 30) ||
      (long long)num_blocks * kBlockSize > 0x7fffffffLL)
    return PKV_ERR_UNSUPPORTED;
  const int row_bytes = head_dim * (cache_dtype == PKV_FP8_E4M3 ? 1 : 2);
  const unsigned long long bytes = (unsigned long long)num_blocks * num_kv_heads * kBlockSize * row_bytes;
  const int rc = check_caches(k_caches, v_caches, num_layers, bytes);
  if (rc != PKV_OK) return rc;
  const unsigned long long S = num_seqs;
  const struct { const void* p; unsigned long long n; } in[] = {
      {block_tables, 4 * S * max_blocks_per_seq}, {context_lens, 4 * S}, {base_lens, 4 * S},
      {keep_start_loc, 4 * (S + 1)}, {keep, 4ull * num_keep},
      {ref_counts, ref_counts ? 4ull * num_blocks : 0}};
  for (const auto& r : in)
    if (S > 0 && r.n > 0 && bytes_overlap(new_lens, 4 * S, r.p, r.n)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  for (int l0 = 0; l0 < num_layers; l0 += PKV_LAYERS_PER_LAUNCH) {
    const int n = std::min(num_layers - l0, PKV_LAYERS_PER_LAUNCH);
    const CompactArgs a{block_tables, context_lens, base_lens, keep_start_loc, keep, new_lens,
                        ref_counts, num_seqs, num_keep, num_kv_heads, max_blocks_per_seq,
                        num_blocks, 2 * n, l0 == 0, device_errors};
    const Caches c = caches_of(k_caches, v_caches, l0, n);
    cudaStream_t on = static_cast<cudaStream_t>(stream);
    const int r = row_bytes == 64    ? launch_compact_rows<64>(c, a, on)
                  : row_bytes == 128 ? launch_compact_rows<128>(c, a, on)
                                     : launch_compact_rows<256>(c, a, on);
    if (r != PKV_OK) return r;
  }
  return PKV_OK;
}

}  // extern "C"

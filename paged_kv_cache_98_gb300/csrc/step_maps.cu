// Step maps: block tables, context lengths, query offsets, slots and positions
// of a batch, built from the requests' lengths (openeuler.csdn.net PagedAttention
// notes, "Block Table 数据结构": token i of a sequence lives at
// slot = table[i / 16] * 16 + i % 16).
//
//   ctx_s  = cached_s + q_s                 have_s = ceil(cached_s / 16)
//   need_s = ceil(ctx_s / 16)               grow_s = need_s - have_s
//   qsl_s  = sum_{r<s} q_r                  off_s  = sum_{r<s} grow_r
// Block b of sequence s is request_tables[rows_s][b] for b < have_s and
// new_blocks[off_s + b - have_s] for have_s <= b < need_s.
//
// One launch.  Every CTA takes both prefix sums over all sequences itself (12
// bytes per sequence out of L2) instead of waiting for another CTA or a second
// launch; then warps copy table rows and threads fill tokens.  Nothing read is
// written in the same launch: the request tables are read below have_s and
// written from have_s on, so CTAs need no order among themselves.
//
// Bound by the launch and the latency of that prefix pass (its loads, then the copies
// that wait for the sums), not by its bytes: one behind the other in a graph, where an empty
// launch takes 0.6 us, 3.3 us for 8 decode rows, 5.6 us for 1000 mixed sequences with 3.4 MB
// of tables (0.5 us of traffic).  Four sequences per thread, so that 1000 take one round
// (2 us less than with one each).

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSeqs = PKV_STEP_MAPS_MAX_SEQS;
constexpr int kPer = 4;  // sequences per thread and round of the prefix sums

struct MapParams {
  int32_t* block_tables;
  int32_t* context_lens;
  int32_t* query_start_loc;
  int64_t* slot_mapping;
  int32_t* positions;
  int32_t* request_tables;
  const int32_t* rows;
  const int32_t* cached_lens;
  const int32_t* q_lens;
  const int32_t* new_blocks;
  int num_seqs, num_rows, max_blocks, num_tokens, num_new, num_blocks;
  int chunks;  // kChunk-entry pieces of a table row
  uint32_t* errors;
};

constexpr int kChunk = 256;  // table entries per warp and work item

struct Seq {
  int row, cached, q;  // row -1: a padding sequence, without context or queries
};

__device__ __forceinline__ Seq load_seq(const MapParams& p, int s, bool report) {
  Seq x;
  x.row = __ldg(p.rows + s);
  x.cached = __ldg(p.cached_lens + s);
  x.q = __ldg(p.q_lens + s);
  const bool pad = x.row < 0;
  const long long ctx = (long long)x.cached + x.q;
  const bool bad = !pad && (x.row >= p.num_rows || x.cached < 0 || x.q < 0 ||
                            ctx > (long long)p.max_blocks * kBlockSize);
  if (bad && report) flag_error(p.errors, PKV_DEVERR_CONTEXT);
  if (pad || bad) x = {-1, 0, 0};
  return x;
}

__device__ __forceinline__ int blocks_of(int tokens) {
  return (tokens + kBlockSize - 1) / kBlockSize;
}

__global__ void __launch_bounds__(kThreads) step_maps_kernel(const MapParams p) {
  extern __shared__ int smem[];
  int* qsl = smem;                   // [S + 1], clamped to num_tokens
  int* off = smem + p.num_seqs + 1;  // [S + 1], clamped to num_new
  __shared__ long long part_q[kWarps], part_g[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.num_seqs;
  const bool first = blockIdx.x == 0;

  // 64-bit sums: a batch of bad lengths must not wrap into a good-looking one.  Each
  // thread takes kPer consecutive sequences, whose loads are on their way together.
  long long base_q = 0, base_g = 0;
  for (int s0 = 0; s0 < S; s0 += kThreads * kPer) {
    const int sb = s0 + tid * kPer;
    Seq x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      x[i] = {-1, 0, 0};
      if (sb + i < S) x[i] = load_seq(p, sb + i, first);
    }
    long long q = 0, g = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      q += x[i].q;
      g += blocks_of(x[i].cached + x[i].q) - blocks_of(x[i].cached);
    }
    long long iq = q, ig = g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(kFull, iq, o), b = __shfl_up_sync(kFull, ig, o);
      if (lane >= o) {
        iq += a;
        ig += b;
      }
    }
    if (lane == 31) {
      part_q[warp] = iq;
      part_g[warp] = ig;
    }
    __syncthreads();
    long long wq = 0, wg = 0, tq = 0, tg = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        wq += part_q[w];
        wg += part_g[w];
      }
      tq += part_q[w];
      tg += part_g[w];
    }
    long long rq = base_q + wq + iq - q, rg = base_g + wg + ig - g;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (sb + i < S) {
        const int ctx = x[i].cached + x[i].q;
        qsl[sb + i] = (int)min(rq, (long long)p.num_tokens);
        off[sb + i] = (int)min(rg, (long long)p.num_new);
        if (first) p.context_lens[sb + i] = ctx;
        rq += x[i].q;
        rg += blocks_of(ctx) - blocks_of(x[i].cached);
      }
    }
    base_q += tq;
    base_g += tg;
    __syncthreads();  // part_* free for the next round
  }
  if (tid == 0) {
    qsl[S] = (int)min(base_q, (long long)p.num_tokens);
    off[S] = (int)min(base_g, (long long)p.num_new);
    if (first && base_q > p.num_tokens) flag_error(p.errors, PKV_DEVERR_CONTEXT);
    if (first && base_g > p.num_new) flag_error(p.errors, PKV_DEVERR_BLOCK_ID);
  }
  __syncthreads();
  if (first)
    for (int s = tid; s <= S; s += kThreads) p.query_start_loc[s] = qsl[s];

  // ---- table rows: kChunk entries of a sequence's row per warp -------------------------------
  const uint32_t items = (uint32_t)S * (uint32_t)p.chunks;  // (below 2^31, checked on the host)
  for (uint32_t it = blockIdx.x * kWarps + warp; it < items; it += gridDim.x * kWarps) {
    const int s = (int)(it / (uint32_t)p.chunks), c = (int)(it - (uint32_t)s * p.chunks);
    const Seq x = load_seq(p, s, false);
    const int have = blocks_of(x.cached), need = blocks_of(x.cached + x.q);
    const int b1 = min(need, (c + 1) * kChunk);
    int32_t* dst = p.block_tables + (size_t)s * p.max_blocks;
    int32_t* src = p.request_tables + (size_t)(x.row < 0 ? 0 : x.row) * p.max_blocks;
    const int o = off[s] - have;
    int32_t id[kChunk / 32];
#pragma unroll
    for (int i = 0; i < kChunk / 32; ++i) {
      const int b = c * kChunk + 32 * i + lane;
      id[i] = -1;
      if (b < b1) {
        if (b < have) id[i] = src[b];
        else if (o + b < p.num_new) id[i] = __ldg(p.new_blocks + o + b);
      }
    }
#pragma unroll
    for (int i = 0; i < kChunk / 32; ++i) {
      const int b = c * kChunk + 32 * i + lane;
      if (b < b1) {
        dst[b] = id[i];
        if (b >= have) src[b] = id[i];
        if (id[i] < 0 || id[i] >= p.num_blocks) flag_error(p.errors, PKV_DEVERR_BLOCK_ID);
      }
    }
  }

  // ---- tokens: slot and position, -1 behind the last sequence ------------------------------------
  const int total = qsl[S];
  // (64 bits: the index steps past num_tokens by up to a grid)
  for (long long i = (long long)blockIdx.x * kThreads + tid; i < p.num_tokens;
       i += gridDim.x * kThreads) {
    const int t = (int)i;
    int64_t slot = -1;
    int pos = -1;
    if (t < total) {
      int lo = 0, hi = S - 1;  // largest s with qsl[s] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (qsl[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const Seq x = load_seq(p, lo, false);
      pos = x.cached + (t - qsl[lo]);
      const int b = pos / kBlockSize, have = blocks_of(x.cached);
      int id = -1;
      if (b < have)
        id = p.request_tables[(size_t)x.row * p.max_blocks + b];
      else if (off[lo] + b - have < p.num_new)
        id = __ldg(p.new_blocks + off[lo] + b - have);
      if (id >= 0 && id < p.num_blocks) slot = (int64_t)id * kBlockSize + pos % kBlockSize;
    }
    p.slot_mapping[t] = slot;
    p.positions[t] = pos;
  }
}

}  // namespace

int launch_step_maps(int32_t* block_tables, int32_t* context_lens, int32_t* query_start_loc,
                     int64_t* slot_mapping, int32_t* positions, int32_t* request_tables,
                     const int32_t* rows, const int32_t* cached_lens, const int32_t* q_lens,
                     const int32_t* new_blocks, int num_seqs, int num_rows, int max_blocks,
                     int num_tokens, int num_new, int num_blocks, uint32_t* errors,
                     cudaStream_t stream) {
  MapParams p{block_tables, context_lens, query_start_loc, slot_mapping, positions,
              request_tables, rows, cached_lens, q_lens, new_blocks, num_seqs, num_rows,
              max_blocks, num_tokens, num_new, num_blocks,
              (max_blocks + kChunk - 1) / kChunk, errors};
  const size_t smem = 2 * ((size_t)num_seqs + 1) * sizeof(int);
  if (smem > 48 * 1024 - 512 &&
      cudaFuncSetAttribute(step_maps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           2 * (kMaxSeqs + 1) * (int)sizeof(int)) != cudaSuccess)
    return PKV_ERR_CUDA;
  const long long warps = (long long)num_seqs * p.chunks;
  if (warps >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
  long long ctas = (warps + kWarps - 1) / kWarps;
  const long long for_tokens = ((long long)num_tokens + kThreads - 1) / kThreads;
  if (for_tokens > ctas) ctas = for_tokens;
  const long long cap = 2LL * sm_count();
  if (ctas > cap) ctas = cap;
  if (ctas < 1) ctas = 1;
  step_maps_kernel<<<(unsigned)ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv

// Requests whose block lists and reference counts live on the GPU: rows forked from their
// parents, blocks taken and given back.  Declarations and semantics are in
// include/pagedkv.h.

#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// ---- fork ------------------------------------------------------------------------------
// T'[i] = T[p_i], L'[i] = L[p_i], and count[b] += children(p) - 1 for every entry b of an
// old row p: a move (one child) touches no count.  So the work goes by old rows: a CTA has
// up to kForkRows of them and kForkChunk of their entries, looks through the parents for
// their children, copies the chunk for each, and adds children - 1 to its blocks' counts
// (integers: the order of the atomics does not matter).  Bound by the reads and writes of
// the tables for long ones, by launch and two dependent reads for short ones (64 rows of up to
// 94 entries: 1.8 us in a graph).
constexpr int kForkThreads = 256;
constexpr int kForkChunk = 1024;   // entries of a row a CTA handles: four a thread
constexpr int kForkTile = 2048;    // parents looked through at a time
constexpr int kForkRows = 64;
constexpr int kForkCtas = 1216;    // rows share CTAs beyond this many (eight a processor)

struct ForkArgs {
  int32_t *tables_out, *lens_out;
  const int32_t *tables, *lens;
  int32_t* counts;
  const int32_t* parents;
  int num_out, num_in, width, num_blocks;
  int rows;   // old rows of a CTA
  int lanes;  // threads that copy one row's chunk together, a power of two: 32 .. 256
  uint32_t* errors;
};

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkArgs a) {
  __shared__ int s_child[kForkTile], s_of[kForkTile];  // a child and its parent among the CTA's rows
  __shared__ int s_len[kForkRows], s_n[kForkRows], s_children[kForkRows];
  __shared__ int s_matches;
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * a.rows, rows = min(a.rows, a.num_in - r0);
  const int e0 = blockIdx.y * kForkChunk;
  const bool first = blockIdx.y == 0;
  int any = 0;
  if (tid < rows) {
    const int cap = a.width * kBlockSize;
    int len = __ldg(a.lens + r0 + tid);
    if (len < 0 || len > cap) {
      if (first) flag_error(a.errors, PKV_DEVERR_CONTEXT);
      len = len < 0 ? 0 : cap;
    }
    s_len[tid] = len;
    s_n[tid] = any = min(max((len + kBlockSize - 1) / kBlockSize - e0, 0), kForkChunk);
    s_children[tid] = 0;
  }
  if (!__syncthreads_or(any) && !first) return;
  const int group = tid / a.lanes, groups = kForkThreads / a.lanes, lane = tid % a.lanes;
  for (int t0 = 0; t0 < a.num_out; t0 += kForkTile) {
    if (tid == 0) s_matches = 0;
    __syncthreads();
    const int t1 = min(t0 + kForkTile, a.num_out);
    for (int i = t0 + tid; i < t1; i += kForkThreads) {
      const int p = __ldg(a.parents + i), r = p - r0;
      if (p >= r0 && r < rows) {
        const int k = atomicAdd(&s_matches, 1);
        s_child[k] = i;
        s_of[k] = r;
        atomicAdd(&s_children[r], 1);
        if (first) a.lens_out[i] = s_len[r];
      } else if (first && blockIdx.x == 0 && (p < 0 || p >= a.num_in)) {
        a.lens_out[i] = 0;
        if (p >= 0) flag_error(a.errors, PKV_DEVERR_CONTEXT);
      }
    }
    __syncthreads();
    const int matches = s_matches;
    for (int k = group; k < matches; k += groups) {
      const int r = s_of[k], n = s_n[r];
      const int32_t* src = a.tables + (size_t)(r0 + r) * a.width + e0;
      int32_t* dst = a.tables_out + (size_t)s_child[k] * a.width + e0;
      int v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = lane + u * a.lanes < n ? __ldg(src + lane + u * a.lanes) : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (lane + u * a.lanes < n) dst[lane + u * a.lanes] = v[u];
    }
    __syncthreads();  // the list has been read
  }
  for (int r = group; r < rows; r += groups) {
    const int more = s_children[r] - 1, n = s_n[r];
    const int32_t* src = a.tables + (size_t)(r0 + r) * a.width + e0;
    for (int e = lane; e < n; e += a.lanes) {
      const int b = __ldg(src + e);
      if (b < 0 || b >= a.num_blocks) flag_error(a.errors, PKV_DEVERR_BLOCK_ID);
      else if (more != 0) atomicAdd(a.counts + b, more);
    }
  }
}

// The same with one old row a CTA, whose entries its threads hold: they are read once, while
// the parents are looked through.  (512 rows of up to 8192 entries: 9 us with tables in L2, 12
// from memory, where samples in groups of eight share the front of their lists and their
// counts change eight times.  Eight rows a CTA, which add up what they change of a shared count,
// take 8 and 12, but 9 instead of 6 where nothing is shared, and 5.7 instead of 4.8 with 128 rows.)
__global__ void __launch_bounds__(kForkThreads) fork_row_kernel(const ForkArgs a) {
  constexpr int kDeep = kForkChunk / kForkThreads;
  __shared__ int s_child[kForkTile];
  __shared__ int s_matches;
  const int tid = threadIdx.x, row = blockIdx.x, e0 = blockIdx.y * kForkChunk + tid;
  const bool first = blockIdx.y == 0;
  const int cap = a.width * kBlockSize;
  int len = __ldg(a.lens + row);
  if (len < 0 || len > cap) {
    if (first && tid == 0) flag_error(a.errors, PKV_DEVERR_CONTEXT);
    len = len < 0 ? 0 : cap;
  }
  const int n = blocks_of(len);
  if (!first && e0 - tid >= n) return;
  const int32_t* src = a.tables + (size_t)row * a.width;
  int v[kDeep], children = 0;
#pragma unroll
  for (int u = 0; u < kDeep; ++u) {
    const int e = e0 + u * kForkThreads;
    v[u] = e < n ? __ldg(src + e) : 0;
  }
  for (int t0 = 0; t0 < a.num_out; t0 += kForkTile) {
    if (tid == 0) s_matches = 0;
    __syncthreads();
    const int t1 = min(t0 + kForkTile, a.num_out);
    for (int i = t0 + tid; i < t1; i += kForkThreads) {
      const int p = __ldg(a.parents + i);
      if (p == row) {
        s_child[atomicAdd(&s_matches, 1)] = i;
        if (first) a.lens_out[i] = len;
      } else if (first && row == 0 && (p < 0 || p >= a.num_in)) {
        a.lens_out[i] = 0;
        if (p >= 0) flag_error(a.errors, PKV_DEVERR_CONTEXT);
      }
    }
    __syncthreads();
    const int matches = s_matches;
    for (int k = 0; k < matches; ++k) {
      int32_t* dst = a.tables_out + (size_t)s_child[k] * a.width;
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (e0 + u * kForkThreads < n) dst[e0 + u * kForkThreads] = v[u];
    }
    children += matches;
    __syncthreads();  // the list has been read
  }
#pragma unroll
  for (int u = 0; u < kDeep; ++u) {
    if (e0 + u * kForkThreads >= n) continue;
    if (v[u] < 0 || v[u] >= a.num_blocks) flag_error(a.errors, PKV_DEVERR_BLOCK_ID);
    else if (children != 1) atomicAdd(a.counts + v[u], children - 1);
  }
}

// ---- resize ----------------------------------------------------------------------------
// One cluster of up to sixteen CTAs, which can wait for each other in hardware and read each
// other's shared memory, so that the call is one launch:
//   1  blocks behind the new lengths lose a reference
//   2  what each sequence needs: a copy of a shared partial last block (how many of its
//      holders grow, and the last of them: a hash table over the cluster's shared memory),
//      and the blocks it opens.  The last of holders that all grow needs no copy, as the others
//      leave; so if one of those is denied its copy, it marks the block, and the last one
//      stays as it is too
//   3  prefix sums of the needs in batch order, and of the free blocks in the order of
//      their ids; every CTA gets all the sequences' offsets
//   4  the warp that meets the r-th free block gives it to the sequence whose needs hold r.
//      The pool is dealt out to the warps in small pieces, since the blocks handed out are
//      those of its first ones
// Every sum is one of integers and the hash table only counts, takes maxima and is marked, so the
// result does not depend on the order of the atomics.  Bound by its dependent reads and
// five cluster barriers for small batches, by reading the counts twice (up to the last
// block handed out the second time) on sixteen processors for large pools: 35 us for 8000 sequences
// that give back or open blocks of a pool of 1000000, of which the scan takes 10.
constexpr int kResizeCtas = 16;  // at most; one where that is enough (kOneCta...)
constexpr int kResizeThreads = 1024;
constexpr int kResizeWarps = kResizeThreads / 32;
constexpr int kSat = 0x3fffffff;  // sums of needs end here; pools hold fewer blocks
constexpr int kPerThread =
    (PKV_STEP_MAPS_MAX_SEQS + kResizeCtas * kResizeThreads - 1) / (kResizeCtas * kResizeThreads);

struct ResizeArgs {
  int32_t *tables, *counts;
  const int32_t *rows, *cached, *lens;
  int32_t *granted, *new_blocks, *pairs;
  int num_seqs, num_rows, width, num_new, num_blocks;
  int slots;   // of the hash table, in each CTA: a power of two, twice the sequences in all
  int pieces;  // of the pool, and the blocks of each (a multiple of 128)
  int piece;
  uint32_t* errors;
};
constexpr int kPieces = 8192;  // at most
// A cluster costs more to start than one CTA, whose scan is longer: 64 sequences take 10.7 us
// with one CTA and 11.8 with sixteen from a pool of 8192 blocks, 12.4 and 12.1 of 32768, 15.0
// and 12.2 of 65536, 32.2 and 13.9 of 262144; 512 take 16.8 and 13.6 of 65536.
constexpr int kOneCtaSeqs = 512, kOneCtaBlocks = 16384;

__device__ __forceinline__ int sat_add(int x, int y) { return min(x + y, kSat); }

// Number of the four counts from id on (below end) that are 0, as bits.
__device__ __forceinline__ uint32_t free_bits(const int32_t* counts, int id, int end, bool vec) {
  uint32_t m = 0;
  if (vec && id + 4 <= end) {
    const int4 c = __ldcg(reinterpret_cast<const int4*>(counts + id));
    m = (c.x == 0 ? 1u : 0u) | (c.y == 0 ? 2u : 0u) | (c.z == 0 ? 4u : 0u) | (c.w == 0 ? 8u : 0u);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (id + u < end && __ldcg(counts + id + u) == 0) m |= 1u << u;
  }
  return m;
}

struct ResizeShared {
  int warp_want[kResizeWarps], warp_open[kResizeWarps], warp_free[kResizeWarps];
  int want[kResizeCtas], open[kResizeCtas];  // of every CTA
  int free;                                  // of the pool
};

__global__ void __launch_bounds__(kResizeThreads, 1) resize_kernel(const ResizeArgs a) {
  extern __shared__ __align__(16) int s_dyn[];  // (counts of pieces are read four at a time)
  __shared__ ResizeShared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = a.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  unsigned* s_begin = reinterpret_cast<unsigned*>(s_dyn);  // [S + 1]: 2 * first rank + (copies?)
  int* s_open = s_dyn + S + 1;                             // [S + 1]: blocks opened before
  int* s_key = s_open + S + 1 + 2 * (S + 1) % 4;           // [slots] a block, -1: none
  int* s_holders = s_key + a.slots;                        // [slots] sequences that grow in it
  int* s_latest = s_holders + a.slots;                     // [slots] the last of them
  int* s_free = s_latest + a.slots;                        // [pieces] free blocks before each piece
  // free blocks of this CTA's pieces: eight consecutive ones, then eight of the next CTA
  const int per_piece_cta = ((a.pieces + 8 * ctas - 1) / (8 * ctas)) * 8;
  int* s_count = s_free + ((a.pieces + 3) & ~3);
  for (int i = tid; i < a.slots; i += kResizeThreads) {
    s_key[i] = -1;
    s_holders[i] = 0;
    s_latest[i] = -1;
  }
  // ---- 1: this thread's sequences (consecutive in batch order), blocks given back ----------
  const int per_cta = (S + ctas - 1) / ctas;
  const int per = (per_cta + kResizeThreads - 1) / kResizeThreads;  // <= kPerThread
  const int i0 = cta * per_cta + tid * per;
  const int i1 = min(min(i0 + per, (cta + 1) * per_cta), S);
  int row[kPerThread], have[kPerThread], need[kPerThread], old_len[kPerThread], new_len[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    row[k] = -1;
    have[k] = need[k] = old_len[k] = new_len[k] = 0;
    const int i = i0 + k;
    if (i < i1) {
      const int r = __ldg(a.rows + i), c = __ldg(a.cached + i), l = __ldg(a.lens + i);
      const int cap = a.width * kBlockSize;
      if (r >= 0) {
        if (r < a.num_rows && c >= 0 && c <= cap && l >= 0 && l <= cap) {
          row[k] = r;
          old_len[k] = c;
          new_len[k] = l;
          have[k] = blocks_of(c);
          need[k] = blocks_of(l);
        } else {
          flag_error(a.errors, PKV_DEVERR_CONTEXT);
        }
      }
    }
    // the warp's sequences give their blocks back together, one entry a lane
    const unsigned back = max(have[k] - need[k], 0);  // (of 32 sequences: at most 2^31)
    unsigned incl = back;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned total = __shfl_sync(kFull, incl, 31);
    constexpr int kBatch = 4;  // entries in flight
    for (unsigned f0 = lane; f0 - lane < total; f0 += 32 * kBatch) {
      int32_t* at[kBatch];
      int b[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const unsigned f = f0 + 32 * u;
        int lo = 0;  // first lane with incl > f
#pragma unroll
        for (int o = 16; o; o >>= 1)
          if (__shfl_sync(kFull, incl, lo + o - 1) <= f) lo += o;
        lo = min(lo, 31);
        const int r = __shfl_sync(kFull, row[k], lo);
        const int e = __shfl_sync(kFull, need[k], lo) +
                      (int)(f - (__shfl_sync(kFull, incl, lo) - __shfl_sync(kFull, back, lo)));
        at[u] = f < total ? a.tables + (size_t)r * a.width + e : nullptr;
        b[u] = at[u] ? *at[u] : 0;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (!at[u]) continue;
        *at[u] = -1;
        if (b[u] >= 0 && b[u] < a.num_blocks) atomicSub(a.counts + b[u], 1);
        else flag_error(a.errors, PKV_DEVERR_BLOCK_ID);
      }
    }
  }
  cluster.sync();  // the counts are what is left, the hash tables are empty
  // ---- 2: needs --------------------------------------------------------------------------
  int slot[kPerThread], held[kPerThread], tail[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    slot[k] = -1;
    held[k] = tail[k] = 0;
    if (row[k] >= 0 && new_len[k] > old_len[k] && old_len[k] % kBlockSize != 0) {
      const int b = a.tables[(size_t)row[k] * a.width + old_len[k] / kBlockSize];
      if (b < 0 || b >= a.num_blocks) {
        flag_error(a.errors, PKV_DEVERR_BLOCK_ID);
      } else if ((held[k] = __ldcg(a.counts + b)) > 1) {
        tail[k] = b;
        // one table over the cluster (twice as many slots as sequences, so the search ends)
        const int all = a.slots * ctas;
        int h = (int)(((uint32_t)b * 2654435761u) >> 7) & (all - 1);
        for (int n = 0; n < all; ++n, h = (h + 1) & (all - 1)) {
          int* key = cluster.map_shared_rank(s_key, h / a.slots) + h % a.slots;
          const int was = atomicCAS(key, -1, b);
          if (was == -1 || was == b) break;
        }
        slot[k] = h;
        atomicAdd(cluster.map_shared_rank(s_holders, h / a.slots) + h % a.slots, 1);
        atomicMax(cluster.map_shared_rank(s_latest, h / a.slots) + h % a.slots, i0 + k);
      }
    }
  }
  // free blocks of this warp's pieces of the pool, for every CTA
  const bool vec = (reinterpret_cast<uintptr_t>(a.counts) & 15u) == 0;
  const int warps = ctas * kResizeWarps, me = warp * ctas + cta;
  constexpr int kScan = 8;  // pieces in flight
  for (int l0 = warp; l0 < per_piece_cta; l0 += kScan * kResizeWarps) {
    unsigned n[kScan];
#pragma unroll
    for (int u = 0; u < kScan; ++u) n[u] = 0;
    for (int d = 4 * lane; d < a.piece; d += 128)
#pragma unroll
      for (int u = 0; u < kScan; ++u) {
        const int l = l0 + u * kResizeWarps;
        const long long id = (long long)((l / 8 * ctas + cta) * 8 + l % 8) * a.piece + d;
        if (l < per_piece_cta && id < a.num_blocks) n[u] += __popc(free_bits(a.counts, (int)id, a.num_blocks, vec));
      }
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
      n[u] = __reduce_add_sync(kFull, n[u]);
      if (lane == 0 && l0 + u * kResizeWarps < per_piece_cta) s_count[l0 + u * kResizeWarps] = (int)n[u];
    }
  }
  cluster.sync();  // every holder has been counted
  // ---- 3: prefix sums ----------------------------------------------------------------------
  int want[kPerThread], opens[kPerThread], want_sum = 0, open_sum = 0;
  bool copies[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    copies[k] = false;
    if (slot[k] >= 0) {
      const int holders = cluster.map_shared_rank(s_holders, slot[k] / a.slots)[slot[k] % a.slots];
      const int latest = cluster.map_shared_rank(s_latest, slot[k] / a.slots)[slot[k] % a.slots];
      copies[k] = !(holders == held[k] && latest == i0 + k);
    }
    opens[k] = max(need[k] - have[k], 0);
    want[k] = opens[k] + (copies[k] ? 1 : 0);
    want_sum = sat_add(want_sum, want[k]);
    open_sum = sat_add(open_sum, opens[k]);
  }
  int want_incl = want_sum, open_incl = open_sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, want_incl, o), y = __shfl_up_sync(kFull, open_incl, o);
    if (lane >= o) {
      want_incl = sat_add(want_incl, x);
      open_incl = sat_add(open_incl, y);
    }
  }
  if (lane == 31) {
    sm.warp_want[warp] = want_incl;
    sm.warp_open[warp] = open_incl;
  }
  // free blocks before each piece: eight pieces a thread, from the CTA that counted them
  static_assert(kPieces <= 8 * kResizeThreads, "eight pieces a thread");
  int mine[8] = {0, 0, 0, 0, 0, 0, 0, 0}, free_sum = 0;
  if (8 * tid < a.pieces) {
    const int4* from = reinterpret_cast<const int4*>(cluster.map_shared_rank(s_count, tid % ctas) + tid / ctas * 8);
    const int4 x = from[0], y = from[1];
    mine[0] = x.x; mine[1] = x.y; mine[2] = x.z; mine[3] = x.w;
    mine[4] = y.x; mine[5] = y.y; mine[6] = y.z; mine[7] = y.w;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) free_sum += mine[u];
  int free_incl = free_sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, free_incl, o);
    if (lane >= o) free_incl += x;
  }
  if (lane == 31) sm.warp_free[warp] = free_incl;
  __syncthreads();
  if (warp == 0) {  // the warps' sums become what is before each of them
    int wi = sm.warp_want[lane], oi = sm.warp_open[lane], fi = sm.warp_free[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(kFull, wi, d), y = __shfl_up_sync(kFull, oi, d),
                z = __shfl_up_sync(kFull, fi, d);
      if (lane >= d) {
        wi = sat_add(wi, x);
        oi = sat_add(oi, y);
        fi += z;
      }
    }
    // (saturated sums cannot be subtracted from: what is before comes from the lane before)
    const int wb = __shfl_up_sync(kFull, wi, 1), ob = __shfl_up_sync(kFull, oi, 1),
              fb = __shfl_up_sync(kFull, fi, 1);
    sm.warp_want[lane] = lane ? wb : 0;
    sm.warp_open[lane] = lane ? ob : 0;
    sm.warp_free[lane] = lane ? fb : 0;
    if (lane == 31) sm.free = fi;
    const int wt = __shfl_sync(kFull, wi, 31), ot = __shfl_sync(kFull, oi, 31);
    if (lane < ctas) {
      ResizeShared* to = cluster.map_shared_rank(&sm, lane);
      to->want[cta] = wt;
      to->open[cta] = ot;
    }
  }
  cluster.sync();
  {
    int at = sm.warp_free[warp] + free_incl - free_sum;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (8 * tid + u < a.pieces) s_free[8 * tid + u] = at;
      at += mine[u];
    }
  }
  const int free_all = sm.free;
  int want_at = 0, open_at = 0, want_all = 0, open_all = 0;
  for (int c = 0; c < ctas; ++c) {
    if (c == cta) {
      want_at = want_all;
      open_at = open_all;
    }
    want_all = sat_add(want_all, sm.want[c]);
    open_all = sat_add(open_all, sm.open[c]);
  }
  {
    const int x = __shfl_up_sync(kFull, want_incl, 1), y = __shfl_up_sync(kFull, open_incl, 1);
    want_at = sat_add(sat_add(want_at, sm.warp_want[warp]), lane ? x : 0);
    open_at = sat_add(sat_add(open_at, sm.warp_open[warp]), lane ? y : 0);
  }
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int i = i0 + k;
    if (i < i1) {
      const unsigned begin = 2u * (unsigned)want_at + (copies[k] ? 1u : 0u);
      s_begin[i] = begin;
      s_open[i] = open_at;
      want_at = sat_add(want_at, want[k]);
      open_at = sat_add(open_at, opens[k]);
      const bool ok = want[k] == 0 || want_at <= free_all;
      if (!ok) {
        flag_error(a.errors, PKV_DEVERR_NO_BLOCKS);
        // it goes on holding its block, whatever the block's last holder counts on (the numbers
        // of holders have been read: a barrier ago)
        if (copies[k]) cluster.map_shared_rank(s_holders, slot[k] / a.slots)[slot[k] % a.slots] = -1;
      }
      a.granted[i] = row[k] < 0 ? 0 : ok ? new_len[k] : old_len[k];
      if (!(ok && copies[k])) {
        a.pairs[2 * i] = -1;
        a.pairs[2 * i + 1] = -1;
      } else {
        atomicSub(a.counts + tail[k], 1);  // (others hold it: it does not become free)
      }
    }
  }
  if (tid == 0) {  // (each CTA's own; not among those copied)
    s_begin[S] = 2u * (unsigned)want_all;
    s_open[S] = open_all;
  }
  cluster.sync();  // the offsets are there, and the marks
  // one that keeps its block while another still holds it does not grow (if it needs blocks, it is
  // behind one that got none, and has none either)
#pragma unroll
  for (int k = 0; k < kPerThread; ++k)
    if (slot[k] >= 0 && !copies[k] &&
        cluster.map_shared_rank(s_holders, slot[k] / a.slots)[slot[k] % a.slots] < 0)
      a.granted[i0 + k] = old_len[k];
  if (ctas > 1) {
    constexpr int kCopy = 4;
    for (int i0 = tid; i0 < S; i0 += kCopy * kResizeThreads) {
      unsigned b[kCopy];
      int o[kCopy];
#pragma unroll
      for (int u = 0; u < kCopy; ++u) {
        const int i = i0 + u * kResizeThreads, of = i / per_cta;
        if (i < S && of != cta) {
          b[u] = cluster.map_shared_rank(s_begin, of)[i];
          o[u] = cluster.map_shared_rank(s_open, of)[i];
        }
      }
#pragma unroll
      for (int u = 0; u < kCopy; ++u) {
        const int i = i0 + u * kResizeThreads;
        if (i < S && i / per_cta != cta) {
          s_begin[i] = b[u];
          s_open[i] = o[u];
        }
      }
    }
    cluster.sync();  // (also: nobody leaves while its memory is read)
  }
  // ---- 4: blocks handed out ------------------------------------------------------------------
  // sequences whose needs end within the free blocks: up to the last offset that does
  auto last_at_most = [&](int n, int r) {  // the last i <= n whose offset is at most r
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int)(s_begin[mid] >> 1) <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  const int end = last_at_most(S, free_all);
  const int limit = (int)(s_begin[end] >> 1), opened = s_open[end];
  for (int n = opened + cta * kResizeThreads + tid; n < a.num_new; n += ctas * kResizeThreads)
    a.new_blocks[n] = -1;
  if (opened > a.num_new && cta == 0 && tid == 0) flag_error(a.errors, PKV_DEVERR_BLOCK_ID);
  for (int k = me; k < a.pieces && s_free[k] < limit; k += warps) {
    const int id0 = k * a.piece, id1 = min(id0 + a.piece, a.num_blocks);
    int r = s_free[k];
    for (int id = id0 + 4 * lane; r < limit && id - 4 * lane < id1; id += 128) {
      const uint32_t bits = id < id1 ? free_bits(a.counts, id, id1, vec) : 0u;
      int incl = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
      }
      int mine = r + incl - __popc(bits);
      r += __shfl_sync(kFull, incl, 31);
      for (uint32_t m = bits; m != 0 && mine < limit; m &= m - 1, ++mine) {
        const int b = id + __ffs(m) - 1;
        const int i = last_at_most(S - 1, mine);
        const unsigned begin = s_begin[i];
        const int k = mine - (int)(begin >> 1), copy = (int)(begin & 1u);
        const int cached = __ldg(a.cached + i);
        // (a copy replaces the last entry, the others go behind it)
        const int e = k < copy ? cached / kBlockSize : blocks_of(cached) + k - copy;
        int32_t* at = a.tables + (size_t)__ldg(a.rows + i) * a.width + e;
        a.counts[b] = 1;
        if (k < copy) {
          a.pairs[2 * i] = *at;
          a.pairs[2 * i + 1] = b;
        } else {
          const int n = s_open[i] + k - copy;
          if (n < a.num_new) a.new_blocks[n] = b;
        }
        *at = b;
      }
    }
  }
}

bool apart(const void* p, unsigned long long np, const void* q, unsigned long long nq) {
  return np == 0 || nq == 0 || !bytes_overlap(p, np, q, nq);
}
bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_fork_requests(int32_t* tables_out, int32_t* lens_out, const int32_t* tables,
                      const int32_t* lens, int32_t* ref_counts, const int32_t* parents,
                      int num_out, int num_in, int max_blocks_per_seq, int block_size,
                      int num_blocks, uint32_t* device_errors, void* stream) {
  using namespace pkv;
  if (num_out < 0 || num_in < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_out > 0 && (!tables_out || !lens_out || !parents)) return PKV_ERR_INVALID_ARG;
  if (num_in > 0 && (!tables || !lens || !ref_counts)) return PKV_ERR_INVALID_ARG;
  if (!words(tables_out) || !words(lens_out) || !words(tables) || !words(lens) ||
      !words(ref_counts) || !words(parents) || !words(device_errors))
    return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (num_out > PKV_FORK_MAX_ROWS || num_in > PKV_FORK_MAX_ROWS) return PKV_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * kBlockSize > (1LL << 30)) return PKV_ERR_UNSUPPORTED;
  const unsigned long long row = 4ull * max_blocks_per_seq, no = num_out, ni = num_in;
  const struct { const void* p; unsigned long long n; } out[] = {
      {tables_out, no * row}, {lens_out, 4 * no}, {ref_counts, ni > 0 ? 4ull * num_blocks : 0}},
      in[] = {{tables, ni * row}, {lens, 4 * ni}, {parents, 4 * no}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (!apart(out[i].p, out[i].n, out[j].p, out[j].n)) return PKV_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j)
      if (!apart(out[i].p, out[i].n, in[j].p, in[j].n)) return PKV_ERR_INVALID_ARG;
  }
  if (num_out == 0 && num_in == 0) return PKV_OK;
  ForkArgs a{tables_out, lens_out, tables, lens, ref_counts, parents, num_out, num_in,
             max_blocks_per_seq, num_blocks, 1, 32, device_errors};
  cudaStream_t on = static_cast<cudaStream_t>(stream);
  const int chunks = (max_blocks_per_seq + kForkChunk - 1) / kForkChunk;
  if (chunks > 65535) return PKV_ERR_UNSUPPORTED;
  if (num_in > 0 && num_in <= kForkCtas) {
    fork_row_kernel<<<dim3(num_in, chunks), kForkThreads, 0, on>>>(a);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  }
  a.rows = num_in > kForkCtas ? (num_in + kForkCtas - 1) / kForkCtas : 1;
  while (a.lanes < kForkThreads && 4 * a.lanes < max_blocks_per_seq) a.lanes *= 2;
  const int ctas = num_in > 0 ? (num_in + a.rows - 1) / a.rows : 1;
  static_assert((PKV_FORK_MAX_ROWS + kForkCtas - 1) / kForkCtas <= kForkRows, "rows of a CTA");
  fork_kernel<<<dim3(ctas, chunks), kForkThreads, 0, on>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int pkv_resize_requests(int32_t* request_tables, int32_t* ref_counts, const int32_t* rows,
                        const int32_t* cached_lens, const int32_t* new_lens,
                        int32_t* granted_lens, int32_t* new_blocks, int32_t* block_pairs,
                        int num_seqs, int num_request_rows, int max_blocks_per_seq,
                        int num_new_blocks, int block_size, int num_blocks,
                        uint32_t* device_errors, void* stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_request_rows <= 0 || max_blocks_per_seq <= 0 || num_new_blocks < 0 ||
      num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!request_tables || !ref_counts || !rows || !cached_lens || !new_lens ||
                       !granted_lens || !block_pairs))
    return PKV_ERR_INVALID_ARG;
  if (num_new_blocks > 0 && !new_blocks) return PKV_ERR_INVALID_ARG;
  if (!words(request_tables) || !words(ref_counts) || !words(rows) || !words(cached_lens) ||
      !words(new_lens) || !words(granted_lens) || !words(new_blocks) || !words(block_pairs) ||
      !words(device_errors))
    return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > PKV_STEP_MAPS_MAX_SEQS || num_blocks >= kSat) return PKV_ERR_UNSUPPORTED;
  if ((long long)max_blocks_per_seq * kBlockSize > (1LL << 30)) return PKV_ERR_UNSUPPORTED;
  const unsigned long long S = num_seqs;
  const struct { const void* p; unsigned long long n; } out[] = {
      {request_tables, S > 0 ? 4ull * num_request_rows * max_blocks_per_seq : 0},
      {ref_counts, S > 0 ? 4ull * num_blocks : 0}, {granted_lens, 4 * S},
      {new_blocks, 4ull * num_new_blocks}, {block_pairs, 8 * S}},
      in[] = {{rows, 4 * S}, {cached_lens, 4 * S}, {new_lens, 4 * S}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (!apart(out[i].p, out[i].n, out[j].p, out[j].n)) return PKV_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j)
      if (!apart(out[i].p, out[i].n, in[j].p, in[j].n)) return PKV_ERR_INVALID_ARG;
  }
  if (num_seqs == 0 && num_new_blocks == 0) return PKV_OK;
  ResizeArgs a{request_tables, ref_counts, rows, cached_lens, new_lens, granted_lens, new_blocks,
               block_pairs, num_seqs, num_request_rows, max_blocks_per_seq, num_new_blocks,
               num_seqs > 0 ? num_blocks : 0, 64, 0, 128, device_errors};
  const int ctas = num_seqs <= kOneCtaSeqs && num_blocks <= kOneCtaBlocks ? 1 : kResizeCtas;
  while (a.slots * ctas < 2 * num_seqs) a.slots *= 2;
  while ((long long)a.piece * kPieces < a.num_blocks) a.piece *= 2;
  a.pieces = (a.num_blocks + a.piece - 1) / a.piece;
  const size_t smem = 4 * (2 * ((size_t)num_seqs + 1) + 2 + 3 * (size_t)a.slots + (a.pieces + 3) / 4 * 4 +
                           (a.pieces + 8 * ctas - 1) / (8 * ctas) * 8);
  constexpr size_t kMostSmem = 4 * (2 * (PKV_STEP_MAPS_MAX_SEQS + 1) +
                                    3 * (2 * PKV_STEP_MAPS_MAX_SEQS / kResizeCtas) + kPieces +
                                    kPieces / kResizeCtas + 16);
  static_assert(kMostSmem + sizeof(ResizeShared) <= 232448, "shared memory budget of one CTA");
  static std::atomic<unsigned long long> configured{0};
  if (!smem_once(resize_kernel, kMostSmem, configured)) return PKV_ERR_CUDA;
  // (more than eight CTAs to a cluster have to be asked for)
  if (ctas > 8 && cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                      cudaSuccess)
    return PKV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kResizeThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, resize_kernel, a) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"

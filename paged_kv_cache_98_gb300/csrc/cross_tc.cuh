// Cross attention on the tcgen05 tensor cores: ragged query rows over the paged states of
// an encoder, every query seeing every state of its sequence (head_dim 64 or 128, 16-bit
// or E4M3 caches, any group size up to 16).
//
// A row is a (query token, head of the group) pair, a query tile is 128 rows of whole
// tokens, a key tile 128 states.  The mathematics is that of prefill_tc.cuh:
//   S = Q K^T in TMEM, P = 2^(s - m) back over S as 16-bit pairs, O += P V,
// where m only has to be near the row's maximum, since P, sums and O are floating-point
// numbers: it starts 4 below the maximum of the first 64 states' scores and moves (and O is
// rescaled) only when the weights of 64 states add up to more than 2^15; out = O / sum(P).
// The sum is that of the rounded weights.  With bf16 ones (16 rows over 300 / 1500 / 16000
// normal states, heads of 128) the error of out is 1.26 / 1.33 / 1.38 times that of an exact
// result's rounding, at most 1.5 / 1.7 / 1.6 times in a call, instead of 1.36 / 1.41 / 1.40 and
// 1.7 / 1.9 / 1.6 with sums of the weights as they were, for 219 us instead of 209 with six
// prompts of 300 to 1500 tokens (both on this kernel); decode waits for memory.
//
// Work.  A unit is a sequence, KV head and one or two query tiles.  With two, K and V of a
// key tile feed both, each tile having its own softmax warpgroup; with one (a token, a
// request's beams, the odd tile of a prompt) the warpgroups take the even and the odd key
// tiles, each into an O of its own, and the one with the last tile joins the two (the other
// goes on to the next unit meanwhile).
// Sequences differ in both lengths and there may be one unit or many thousand, so units
// are not dealt out: all key tiles of the call lie one behind the other on a line of work
// (a tile counts kCost1 or kCost2, what a unit costs once kCostUnit), which is cut into
// one equal part for each CTA, one CTA a processor.  Cuts fall inside units, also where
// queries are few and inputs long; what a CTA has of a cut unit goes to the workspace as a
// normalised partial and its log-sum-exp, at most two per CTA, and a second kernel, launched
// as a dependent, joins the parts of a unit.  The line is walked with integers that every
// CTA computes for itself, so the result depends on the batch alone.
//
// Two CTAs of a cluster that share four query tiles, each loading half of every K and V tile
// and multicasting it to both, were built and measured: 741 against 747 us for four prompts of
// 1024 tokens over 16384 states (before the sums of rounded weights), and slower with ragged
// prompts (in a unit of few tiles one CTA waits for the other).  Loads alone take 515 us of
// those, MMAs alone 495.
//
// Bounds, and what was measured (calls in a graph, join included; heads of 128 on 8): HBM for
// few queries (1.5 GB of states 234 us, 6.5 TB/s); for prompts the softmax's exponentials and
// conversions beside the MMAs (four of 1024 tokens over 16384 states 762 us, 1440 TFLOP/s; six
// ragged ones 219 us, 1145); on E4M3 caches the converters' and the softmax's instructions
// (260 MB of codes 107 us); latency for small calls (eight tokens, 16 heads of 64, 23 MB: 20 us).
// A key tile takes its 1.03 us however few rows it has, which bounds few queries where its bytes
// take less (heads of 64: 16 sequences of 8192 states on 8 heads, 268 MB, 58 us).
//
// Warps: 0-3 softmax of tile a (or even key tiles), 4-7 of tile b (odd), 8 and 9 issue the
// MMAs of either (8 owns TMEM), 10 and 11 load, 10 also makes the items from the line of work
// and loads the V rows of partial last blocks, 12-15 (E4M3 caches) widen K tiles to the
// query's type and V tiles to fp16 where they land.
#ifndef PKV_CROSS_TC_CUH
#define PKV_CROSS_TC_CUH

#include "cross.h"
#include "prefill_mods.cuh"

namespace pkv {
namespace cross_tc {
namespace {
using namespace pre_tc;
using pre_mods::issue_mods_scores;
using pre_mods::wait_for;
using pre_mods::widen16;

constexpr int kSoft = 8;       // softmax warps
constexpr int kIssuer = 8, kIssuers = 2, kTma = 10, kTmaWarps = 2, kConvert = 12, kConverts = 4;
constexpr int cross_threads(bool fp8) { return fp8 ? 512 : 384; }
// Registers: the launch holds 168 for each of 384 threads or 128 for each of 512; the
// softmax warps take over what the others return.
constexpr int cross_launch_regs(bool fp8) { return fp8 ? 128 : 168; }
constexpr int cross_soft_regs(bool fp8) { return fp8 ? 168 : 200; }
constexpr int cross_other_regs(bool fp8) { return fp8 ? 88 : 104; }
constexpr bool cross_regs_fit(bool fp8) {
  return 256 * cross_soft_regs(fp8) + (cross_threads(fp8) - 256) * cross_other_regs(fp8) <=
         cross_threads(fp8) * cross_launch_regs(fp8);
}
static_assert(cross_regs_fit(false) && cross_regs_fit(true),
              "setmaxnreg may only share out what the launch holds");

// The line of work, in quarters of a key tile's time with one query tile (measured: 1.03 us
// with one, 1.6 with two, and 3 to 4 us for a unit once).
constexpr int kCost1 = 4;
constexpr int kCost2 = 6;
constexpr int kCostUnit = 14;  // at most half of a CTA's part of the tiles: every part
                               // begins with a unit, or what is left of one, anyway
constexpr int kLeast = 8;  // of a CTA's part (at least kCost2, so that every part inside a unit
                           // holds the start of a tile)
constexpr float kMostSum = 32768.0f;   // of 64 weights, before m moves (fp16 holds any of them)
constexpr float kLift = 4.0f;          // m is 2^4 below the maximum that it is taken from: fp16
                                       // weights then reach 2^-28 of the largest
constexpr int kItems = 4;              // made ahead

// Type of the products P V: the query's, but fp16 on an E4M3 cache, whose codes it holds as
// they are; the weights are rounded to 2^-12 of theirs then, not to the 2^-9 of bf16.
template <class QT, bool kFP8>
using ProductType = typename std::conditional<kFP8, F16, QT>::type;

struct CrossItem {
  int live;            // 0: the end
  int seq, kvh, len, q0;
  int t0[2], nt[2];    // first token (within the sequence) and tokens of the query tiles
  int kt0, kt1;        // key tiles (none: no states, the rows are zeros)
  int part;            // slot of the partial, -1: all of the unit
  int tail;            // 16-state step of tile kt1 - 1 with the partial last block, else -1
};

template <int D, bool kFP8>
struct CrossSmem {
  static constexpr int kTile = 128 * D * 2;                   // bytes of a 16-bit tile
  static constexpr int kCodes = 16384;                        // place of E4M3 codes in a stage
  static constexpr int kStage = kFP8 && D == 64 ? 24576 : kTile;
  static constexpr int kSt = 131072 / kStage;                 // 4, 5 or 8 stages
  static constexpr int kTail = kBlockSize * D * 2;
  alignas(1024) uint8_t ring[kSt][kStage];
  alignas(1024) uint8_t q[2][kTile];
  alignas(1024) uint8_t tail[2][kTail];
  long long start[kMaxSeqs + 1];  // of each sequence on the line of work
  int qlen[kMaxSeqs], len[kMaxSeqs], q0[kMaxSeqs];
  long long scan[16];
  int scan_units[16];
  int cost_unit;
  float2 other[128];  // maxima and sums of the warpgroup that does not join
  CrossItem item[kItems];
  uint64_t item_full[kItems], item_read[kItems];
  uint64_t landed[kSt], full[kSt], empty[kSt];
  uint64_t q_full[2], q_empty[2];
  uint64_t turn[2];
  uint64_t s_ready[2], p_half[2], p_ready[2], o_half[2], o_done[2], o_free[2];
  uint64_t other_ready;
  uint64_t tail_full[2], tail_free[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  uint32_t issued;  // places of the ring that producer 0 has come to
  int abort;
};

__device__ __forceinline__ int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }

// The next item, for a whole warp; false when the wait gave up.
template <class SM>
__device__ __forceinline__ bool take(SM& sm, uint32_t n, CrossItem& x, volatile int* abort,
                                     unsigned long long lim) {
  const int slot = n % kItems;
  if (!__all_sync(kFull, wait_for(&sm.item_full[slot], (n / kItems) & 1, abort, lim))) return false;
  x = sm.item[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.item_read[slot]);
  return true;
}

// ---- the line of work --------------------------------------------------------------------
// Lengths of the sequences and where each begins on the line; ends with the CTA
// synchronised.
template <int D, bool kFP8>
__device__ __forceinline__ void cross_setup(const AttnParams& p, const CrossArgs& c,
                                            CrossSmem<D, kFP8>& sm) {
  using SM = CrossSmem<D, kFP8>;
  constexpr int kThreads = cross_threads(kFP8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < SM::kSt; ++s) {
      mbar_init(&sm.landed[s], 1);
      mbar_init(&sm.full[s], kFP8 ? kConverts : 1);
      mbar_init(&sm.empty[s], kIssuers);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.q_full[x], 1);
      mbar_init(&sm.q_empty[x], kIssuers);
      mbar_init(&sm.s_ready[x], 1);
      mbar_init(&sm.turn[x], 1);
      mbar_init(&sm.p_half[x], 4);
      mbar_init(&sm.p_ready[x], 4);
      mbar_init(&sm.o_half[x], 1);
      mbar_init(&sm.o_done[x], 1);
      mbar_init(&sm.o_free[x], 4);
      mbar_init(&sm.tail_full[x], 1);
      mbar_init(&sm.tail_free[x], kIssuers);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      // the softmax warps, the issuers, the other producer and the converters
      mbar_init(&sm.item_read[i], kSoft + kIssuers + kTmaWarps - 1 + (kFP8 ? kConverts : 0));
    }
    mbar_init(&sm.other_ready, 4);
    mbar_init(&sm.mma_done, kIssuers);
    sm.abort = 0;
    sm.issued = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  const int S = p.num_seqs, tid = threadIdx.x;
  const int chunk = (S + kThreads - 1) / kThreads;
  const int cap = min(p.max_blocks_per_seq * kBlockSize, p.max_context);
  const int rpt = kRowsM / p.group;
  auto work = [&](int q, int len) -> long long {  // of its key tiles
    const int tiles = (q + rpt - 1) / rpt;
    return (long long)p.num_kv_heads * tiles_of(len) * ((long long)(tiles >> 1) * kCost2 + (tiles & 1) * kCost1);
  };
  // (a launch has below 2^31 units: its query heads)
  auto units = [&](int q) { return p.num_kv_heads * (((q + rpt - 1) / rpt + 1) >> 1); };
  long long local = 0;
  int mine = 0;
  for (int i = 0; i < chunk; ++i) {
    const int sq = tid * chunk + i;
    if (sq < S) {
      const int q0 = __ldg(p.query_start_loc + sq), q1 = __ldg(p.query_start_loc + sq + 1);
      int len = __ldg(p.context_lens + sq), q = q1 - q0;
      if (len < 0 || len > cap || q0 < 0 || q1 < q0 || q1 > p.num_rows || q > c.max_q) {
        if (blockIdx.x == 0) flag_error(p.errors, PKV_DEVERR_CONTEXT);
        len = len < 0 ? 0 : min(len, cap);
        q = q0 < 0 || q1 < q0 || q1 > p.num_rows ? 0 : min(q, c.max_q);
      }
      sm.qlen[sq] = q;
      sm.len[sq] = len;
      sm.q0[sq] = q0;
      local += work(q, len);
      mine += units(q);
    }
  }
  long long incl = local;
  int incl_u = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, incl, o);
    const int z = __shfl_up_sync(kFull, incl_u, o);
    if (lane >= o) {
      incl += y;
      incl_u += z;
    }
  }
  if (lane == 31) {
    sm.scan[warp] = incl;
    sm.scan_units[warp] = incl_u;
  }
  __syncthreads();
  long long run = incl - local, total = 0;
  int run_u = incl_u - mine;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      run += sm.scan[w];
      run_u += sm.scan_units[w];
    }
    total += sm.scan[w];
  }
  const int unit = (int)max(min(total / (2 * (int)gridDim.x), (long long)kCostUnit), 1LL);
  for (int i = 0; i < chunk; ++i) {
    const int sq = tid * chunk + i;
    if (sq < S) {
      sm.start[sq] = run + (long long)unit * run_u;
      run += work(sm.qlen[sq], sm.len[sq]);
      run_u += units(sm.qlen[sq]);
    }
  }
  if (tid == kThreads - 1) {  // (the last thread's run ends at the total)
    sm.start[S] = run + (long long)unit * run_u;
    sm.cost_unit = unit;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
}

// This CTA's part of the line, walked by one warp.
struct Walk {
  long long T, w, w1;  // the line, where the walk is and ends
  int parts, s;        // parts of the line, the sequence at w
  int4 cut0, cut1;     // the unit that the part ends in
};

template <int D, bool kFP8>
__device__ __forceinline__ Walk walk_begin(const AttnParams& p, const CrossSmem<D, kFP8>& sm) {
  Walk k;
  k.T = sm.start[p.num_seqs];
  k.parts = (int)max(min((long long)gridDim.x, k.T / kLeast), 1LL);
  const int part = blockIdx.x;
  k.w = part < k.parts ? k.T * part / k.parts : 0;
  k.w1 = part < k.parts ? k.T * (part + 1) / k.parts : 0;
  k.cut0 = k.cut1 = make_int4(-1, 0, 0, 0);
  k.s = 0;
  if (k.w < k.w1) {  // the last sequence that begins at or before w
    int hi = p.num_seqs - 1;
    while (k.s < hi) {
      const int mid = (k.s + hi + 1) >> 1;
      if (sm.start[mid] <= k.w) k.s = mid; else hi = mid - 1;
    }
  }
  return k;
}

// The next item of the part (none: live is 0).
template <int D, bool kFP8>
__device__ __forceinline__ CrossItem walk_on(const AttnParams& p, const CrossSmem<D, kFP8>& sm, Walk& v) {
  const int rpt = kRowsM / p.group, hkv = p.num_kv_heads, once = sm.cost_unit;
  CrossItem x = {};
  while (v.w < v.w1) {
    const int q = sm.qlen[v.s], len = sm.len[v.s], nk = tiles_of(len);
    const int tiles = (q + rpt - 1) / rpt;
    const long long u2 = (long long)nk * kCost2 + once, u1 = (long long)nk * kCost1 + once;
    const long long twos = (long long)hkv * (tiles >> 1), off = v.w - sm.start[v.s];
    const bool two = off < twos * u2;
    const long long k = two ? off / u2 : twos + (off - twos * u2) / u1;
    const long long u0 = sm.start[v.s] + (two ? k * u2 : twos * u2 + (k - twos) * u1);
    const long long u = two ? u2 : u1;
    const int cost = two ? kCost2 : kCost1;
    // tiles whose place on the line is in [w, w1)
    auto tile_at = [&](long long at) {
      const long long d = at - u0 - once;
      return d <= 0 ? 0 : (int)min((d + cost - 1) / cost, (long long)nk);
    };
    const int a = v.w <= u0 ? 0 : tile_at(v.w), b = v.w1 >= u0 + u ? nk : tile_at(v.w1);
    const bool begins = v.w <= u0;
    const int seq = v.s;
    v.w = u0 + u;
    while (v.s + 1 < p.num_seqs && sm.start[v.s + 1] <= v.w) ++v.s;
    if (a >= b && !(nk == 0 && begins)) continue;
    x.live = 1;
    x.seq = seq;
    x.kvh = (int)(k % hkv);
    x.len = len;
    x.q0 = sm.q0[seq];
    x.t0[0] = 2 * (int)(k / hkv) * rpt;
    x.t0[1] = x.t0[0] + rpt;
    x.nt[0] = min(rpt, q - x.t0[0]);
    x.nt[1] = two ? min(rpt, q - x.t0[1]) : 0;
    x.kt0 = a;
    x.kt1 = b;
    x.part = a == 0 && b == nk ? -1 : 2 * (int)blockIdx.x + (a == 0 ? 1 : 0);
    x.tail = !kFP8 && b == nk && (len & (kBlockSize - 1)) != 0 ? ((len - 1) % kTileKeys) / kBlockSize : -1;
    if (a == 0 && b < nk) {
      // the unit goes on in the parts up to the one with its last tile
      const long long last = u0 + once + (long long)(nk - 1) * cost;
      v.cut0 = make_int4((int)(((last + 1) * v.parts + v.T - 1) / v.T - 1), x.q0 + x.t0[0], x.nt[0], x.nt[1]);
      v.cut1 = make_int4(x.kvh, 0, 0, 0);
    }
    break;
  }
  return x;
}

// ---- loads ---------------------------------------------------------------------------------
// Order of a unit's tiles in the ring, as the issuer takes them: K0, K1, V0, K2, V1, ...
template <int D, bool kFP8>
__device__ __forceinline__ void cross_producer(const AttnParams& p, const CrossArgs& c,
                                               CrossSmem<D, kFP8>& sm, const CUtensorMap& tm_k,
                                               const CUtensorMap& tm_v, const CUtensorMap& tm_q,
                                               int kv_rows, int pw) {
  using SM = CrossSmem<D, kFP8>;
  constexpr int kSt = SM::kSt;
  constexpr int kRow = D * (kFP8 ? 1 : 2);          // bytes of a cache row
  constexpr int kBoxRow = kRow < 128 ? kRow : 128;  // bytes of a row in a box
  constexpr int kLoad = kTileKeys * kRow;
  uint64_t* const bars = kFP8 ? sm.landed : sm.full;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const int lane = threadIdx.x & 31, g = p.group;
  const bool my_lane = (lane & 1) == pw;            // blocks pw, pw + 2, ... of a tile
  uint8_t* const ring = &sm.ring[0][0];
  uint32_t pos = 0, nq = 0, ntail = 0;
  bool ok = true;
  CrossItem x = {};
  auto fetch = [&](int ch) -> int {                 // table entry of block 32 ch + lane
    const int b = 32 * ch + lane;
    return b < (x.len + kBlockSize - 1) / kBlockSize
               ? __ldg(p.block_tables + (size_t)x.seq * p.max_blocks_per_seq + b)
               : kBeyond;
  };
  auto to_row = [&](int blk) -> int {
    if (blk == kBeyond) return kv_rows;             // past the pool: the box reads zeros
    if (blk >= 0 && blk < p.num_blocks) return (blk * p.num_kv_heads + x.kvh) * kBlockSize;
    flag_error(p.errors, PKV_DEVERR_BLOCK_ID);
    return kv_rows;
  };
  auto issue = [&](int t, int row, bool is_v) -> bool {
    const int st = pos % kSt;
    // test hook: these boxes are never issued, so every wait for the tile runs out
    const bool skip = blockIdx.x == 0 && p.skip_copy > 0 && pos + 1 == (uint32_t)p.skip_copy;
    bool good = true;
    if (lane == 0) {
      if (pos >= (uint32_t)kSt) good = wait_for(&sm.empty[st], ((pos / kSt) - 1) & 1, abort, lim);
      if (good && !skip && pw == 0) mbar_arrive_expect_tx(&bars[st], kLoad);
      if (good && pw == 0) {
        __threadfence_block();
        *static_cast<volatile uint32_t*>(&sm.issued) = pos + 1;
      }
    }
    if (!__shfl_sync(kFull, (int)good, 0)) return false;
    if (!skip && (lane >> 3) == (t & 3) && my_lane) {
      uint8_t* dst = ring + (size_t)st * SM::kStage + (kFP8 ? SM::kCodes : 0) +
                     (lane & 7) * (kBlockSize * kBoxRow);
      const CUtensorMap* map = is_v ? &tm_v : &tm_k;
      tc::tma_load_2d(dst, map, 0, row, &bars[st]);
      if (kRow > 128) tc::tma_load_2d(dst + kHalf, map, 64, row, &bars[st]);
    }
    __syncwarp();
    ++pos;
    return true;
  };
  // V rows of the step that holds the partial last block, rows past the states as zeros (in the
  // product 0 * NaN would be NaN), with the ring's swizzle
  auto load_tail = [&]() -> bool {
    const int buf = ntail & 1;
    bool good = true;
    if (lane == 0 && ntail >= 2) good = wait_for(&sm.tail_free[buf], ((ntail >> 1) - 1) & 1, abort, lim);
    if (!__shfl_sync(kFull, (int)good, 0)) return false;
    constexpr int kChunks = D / 8;  // 16-byte chunks of a row
    const int b = (x.len - 1) / kBlockSize;
    const int blk = __ldg(p.block_tables + (size_t)x.seq * p.max_blocks_per_seq + b);
    const bool in = blk >= 0 && blk < p.num_blocks;
#pragma unroll
    for (int i = 0; i < kBlockSize * kChunks / 32; ++i) {
      const int e = lane + 32 * i, r = e / kChunks, ch = e % kChunks;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (in && b * kBlockSize + r < x.len)
        v = __ldg(reinterpret_cast<const uint4*>(
                      p.v_cache + (((size_t)blk * p.num_kv_heads + x.kvh) * kBlockSize + r) * (kChunks * 16)) + ch);
      *reinterpret_cast<uint4*>(&sm.tail[buf][0] + (ch >> 3) * (SM::kTail / 2) + r * 128 +
                                (((ch & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.tail_full[buf]);
    ++ntail;
    return true;
  };
  Walk walk = {};
  if (pw == 0) walk = walk_begin<D, kFP8>(p, sm);
  for (uint32_t n = 0; ok; ++n) {
    if (pw == 0) {  // makes the items, for the others too
      x = walk_on<D, kFP8>(p, sm, walk);
      bool good = true;
      if (lane == 0) {
        const int slot = n % kItems;
        if (n >= kItems) good = wait_for(&sm.item_read[slot], ((n / kItems) - 1) & 1, abort, lim);
        if (good) {
          sm.item[slot] = x;
          mbar_arrive(&sm.item_full[slot]);
        }
      }
      ok = __shfl_sync(kFull, (int)good, 0) != 0;
    } else {
      ok = take(sm, n, x, abort, lim);
    }
    if (!ok || !x.live) break;
    if (x.kt0 == x.kt1) continue;
    if (pw == 0) {
      bool good = true;
      for (int qt = 0; qt < 2 && x.nt[qt] > 0; ++qt, ++nq) {
        const int b = nq & 1;
        if (lane == 0 && good) {
          if (nq >= 2) good = wait_for(&sm.q_empty[b], ((nq >> 1) - 1) & 1, abort, lim);
          if (good) {
            uint8_t* dq = &sm.q[b][0];
            mbar_arrive_expect_tx(&sm.q_full[b], c.box_tokens * g * D * 2);
            const int tok = x.q0 + x.t0[qt];
            tc::tma_load_3d(dq, &tm_q, 0, x.kvh * g, tok, &sm.q_full[b]);
            if (D > 64) tc::tma_load_3d(dq + kHalf, &tm_q, 64, x.kvh * g, tok, &sm.q_full[b]);
          }
        }
      }
      ok = __shfl_sync(kFull, (int)good, 0) != 0;
    }
    // block rows of two chunks of 32 blocks (four key tiles), which K and V tiles are in,
    // and the next one's entries, read ahead
    int c0 = -1, c1 = -1, row0 = kv_rows, row1 = kv_rows;
    int pre = x.kt0 >> 2, pre_raw = fetch(pre);
    auto row_for = [&](int t) -> int {
      const int ch = t >> 2;
      if (c0 == ch) return row0;
      if (c1 == ch) return row1;
      const int r = to_row(pre == ch ? pre_raw : fetch(ch));
      if (c0 < c1) {
        c0 = ch;
        row0 = r;
      } else {
        c1 = ch;
        row1 = r;
      }
      pre = ch + 1;
      pre_raw = 4 * pre < x.kt1 ? fetch(pre) : kBeyond;
      return r;
    };
    if (ok) ok = issue(x.kt0, row_for(x.kt0), false);
    for (int t = x.kt0; ok && t < x.kt1; ++t) {
      if (t + 1 < x.kt1) ok = issue(t + 1, row_for(t + 1), false);
      if (ok && pw == 0 && t == x.kt1 - 1 && x.tail >= 0) ok = load_tail();
      if (ok) ok = issue(t, row_for(t), true);
    }
  }
  if (pw == 0 && lane == 0 && c.cuts) {
    c.cuts[2 * blockIdx.x] = walk.cut0;
    c.cuts[2 * blockIdx.x + 1] = walk.cut1;
  }
  if (!ok && lane == 0) {
    flag_error(p.errors, PKV_DEVERR_TIMEOUT);
    // tiles and queries still on their way land before the CTA goes away
    for (uint32_t y = pos > (uint32_t)kSt ? pos - kSt : 0; y < pos; ++y)
      mbar_wait(&bars[y % kSt], (y / kSt) & 1, 10000000ull);
    if (pw == 0)
      for (uint32_t y = nq > 2 ? nq - 2 : 0; y < nq; ++y)
        mbar_wait(&sm.q_full[y & 1], (y >> 1) & 1, 10000000ull);
  }
}

// Converter cw of an E4M3 cache: each tile that has landed, in ring order, from codes
// [128 rows][D bytes] at kCodes of its stage to 16-bit elements, [D / 64 halves][128 rows]
// [128 bytes] with the 128-byte swizzle; V rows past the states as zeros.  (head_dim 128:
// row r of the codes lies where row r of the second half will, and a warp reads whole rows
// before it writes them.)
template <class QT, int D>
__device__ __forceinline__ void cross_converter(const AttnParams& p, CrossSmem<D, true>& sm, int cw) {
  using SM = CrossSmem<D, true>;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  constexpr int kLanes = D / 16;      // 16-code chunks, and lanes, per row
  constexpr int kRows = 32 / kLanes;  // rows a turn
  const int lane = threadIdx.x & 31, ch = lane % kLanes;
  uint32_t pos = 0;
  bool ok = true;
  CrossItem x = {};
  auto convert = [&](auto type, int rows) -> bool {
    using T = decltype(type);
    const int st = pos % SM::kSt;
    if (!__all_sync(kFull, wait_for(&sm.landed[st], (pos / SM::kSt) & 1, abort, lim))) return false;
    ++pos;
    uint8_t* tile = &sm.ring[st][0];
    auto codes = [&](int u) {
      const int r = kRows * u + lane / kLanes;
      return *reinterpret_cast<const uint4*>(tile + SM::kCodes + r * D +
                                             ((D == 128 ? ch ^ (r & 7) : ch) << 4));
    };
    // two turns' codes at a time (beams 124 us with one, 110 with two, 126 with four, whose code
    // the instruction cache has no room for beside the softmax's)
    constexpr int kTurns = kTileKeys / kRows / kConverts;
    constexpr int kDeep = kTurns < 2 ? kTurns : 2;
#pragma unroll 1
    for (int u0 = cw; u0 < kTileKeys / kRows; u0 += kConverts * kDeep) {
      uint4 w[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) w[i] = codes(u0 + i * kConverts);
      __syncwarp();  // the rows have been read
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int r = kRows * (u0 + i * kConverts) + lane / kLanes;
        if (r >= rows) w[i] = make_uint4(0, 0, 0, 0);
        // (the halves' lanes store their two chunks in opposite order: eight lanes hit eight
        // different bank groups)
        const bool up = ch >> 2;
        const uint32_t v[4] = {up ? w[i].z : w[i].x, up ? w[i].w : w[i].y, up ? w[i].x : w[i].z,
                               up ? w[i].y : w[i].w};
        uint4 a, b;
        widen16<T>(v, &a, &b);
        uint8_t* d = tile + (ch >> 2) * kHalf + r * 128;
        const int k0 = (2 * (ch & 3) + (up ? 1 : 0)) ^ (r & 7);
        *reinterpret_cast<uint4*>(d + (k0 << 4)) = a;
        *reinterpret_cast<uint4*>(d + ((k0 ^ 1) << 4)) = b;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.full[st]);
    return true;
  };
  for (uint32_t n = 0; ok; ++n) {
    ok = take(sm, n, x, abort, lim);
    if (!ok || !x.live) break;
    auto rows = [&](int t) { return min(x.len - t * kTileKeys, kTileKeys); };
    if (x.kt0 < x.kt1) ok = convert(QT{}, kTileKeys);
    for (int t = x.kt0; ok && t < x.kt1; ++t) {
      if (t + 1 < x.kt1) ok = convert(QT{}, kTileKeys);
      if (ok) ok = convert(ProductType<QT, true>{}, rows(t));
    }
  }
  if (!ok && lane == 0) flag_error(p.errors, PKV_DEVERR_TIMEOUT);
}

// Half of a tile's product, O (at d) (+)= P (TMEM at a, 16 states per 8 columns) V: the steps of
// 16 states from kFrom on; step ts takes its V rows from the tail buffer.
template <int kFrom>
__device__ __forceinline__ void issue_half(uint32_t d, uint32_t a, uint64_t dv, uint64_t dtail, int ts,
                                           uint32_t acc0, uint32_t idesc) {
#pragma unroll
  for (int kk = kFrom; kk < kFrom + kTileKeys / 32; ++kk) {
    const uint64_t b = kk == ts ? dtail : dv + (uint64_t)((kk * (kBlockSize * 128)) >> 4);
    mma_f16_tmem_a(d, a + kk * 8, b, idesc, acc0 | (kk != kFrom ? 1u : 0u));
  }
}

// ---- MMA issuers -----------------------------------------------------------------------------
// One thread for each softmax warpgroup: with two query tiles P_y(t) V(t), S_y(t+1) for every
// key tile t; with one, of every other key tile, t = y first.  (One for both left the tensor
// pipe idle while it waited and committed: without any softmax a key tile took 3100 cycles of
// which 2050 are MMAs.)
//
// A stage is empty when both issuers have released it; whoever uses it alone does so twice.
// An issuer that does not use a stage for a while waits for the producer to have come to its
// tile's place first: a barrier tells one phase from the one before, not from the one before
// that, so the wait for a tile may only begin when the one before in its stage has landed.
// Places of a unit's tiles in the ring: K0, K1, V0, K2, V1, ..., V(n-1).
__device__ __forceinline__ uint32_t k_place(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ uint32_t v_place(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

template <class QT, int D, bool kFP8>
__device__ __forceinline__ bool issue_group(const AttnParams& p, CrossSmem<D, kFP8>& sm, uint32_t tmem, int y) {
  using SM = CrossSmem<D, kFP8>;
  constexpr int kSt = SM::kSt;
  constexpr uint32_t kAB = std::is_same<QT, BF16>::value ? 1u : 0u;
  constexpr uint32_t kPV = std::is_same<ProductType<QT, kFP8>, BF16>::value ? 1u : 0u;
  constexpr uint32_t kIdescS = tc::idesc_f16(kAB, 0, 0, 128, kTileKeys);
  constexpr uint32_t kIdescO = tc::idesc_f16(kPV, 0, 1, 128, D);
  constexpr uint64_t kStage = SM::kStage >> 4;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_for(bar, parity, abort, lim); };
  const uint64_t dq0 = tc::smem_desc(smem_u32(&sm.q[0][0]), 16, 1024, tc::kLayoutSw128);
  const uint64_t dk0 = tc::smem_desc(smem_u32(&sm.ring[0][0]), 16, 1024, tc::kLayoutSw128);
  const uint64_t dv0 = tc::smem_desc(smem_u32(&sm.ring[0][0]), kHalf, 1024, tc::kLayoutSw128);
  const uint64_t dt0 = tc::smem_desc(smem_u32(&sm.tail[0][0]), SM::kTail / 2, 1024, tc::kLayoutSw128);
  const uint32_t s_col = tmem + y * 128, o_col = tmem + kColO + y * 128;
  uint32_t base = 0, np = 0, nit = 0, nq = 0, ntail = 0;  // ring place of the unit, P consumed, ...
  uint32_t seen = 0;    // places that the producer has come to, as last read
  auto issued = [&](uint32_t at) -> bool {
    for (uint64_t t0 = 0; (int32_t)(seen - at) <= 0;) {
      seen = *static_cast<volatile uint32_t*>(&sm.issued);
      if ((int32_t)(seen - at) > 0) break;
      if (*abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > lim) {
        *abort = 1;
        return false;
      }
    }
    return true;
  };
  uint32_t turns = 0;   // handed over by the other issuer
  bool others = false;  // (the first issuer) the last product of two query tiles is the other's
  CrossItem x = {};
  for (uint32_t n = 0;; ++n) {
    const int slot = n % kItems;
    if (!wait(&sm.item_full[slot], (n / kItems) & 1)) return false;
    x = sm.item[slot];
    mbar_arrive(&sm.item_read[slot]);
    if (!x.live) return true;
    const int tiles = x.kt1 - x.kt0;
    if (tiles == 0) continue;  // nothing to multiply: the rows are zeros
    const bool two = x.nt[1] > 0;
    auto full = [&](uint32_t place, int& st) -> bool {
      const uint32_t at = base + place;
      st = at % kSt;
      if (!issued(at)) return false;
      return wait(&sm.full[st], (at / kSt) & 1);
    };
    auto release = [&](int st) {
      tc::mma_commit(&sm.empty[st]);
      if (!two) tc::mma_commit(&sm.empty[st]);
    };
    const int step = two ? 1 : 2, first = two ? 0 : y;
    // Of a pair of query tiles an issuer waits for its own only, and yet never takes the phase
    // before last of the other's buffer when it comes to the next tile there.  Issuer 1 has gone
    // on to its product behind issuer 0's (the turn), so the pair's first tile has landed.
    // For issuer 0 a tile of its own lies between (were it of a pair, the next would be issuer 1's),
    // loaded when both had given the pair back: issuer 1 did so behind the second tile's landing.
    const int qb = (nq + (two ? y : 0)) & 1;
    if (!wait(&sm.q_full[qb], ((nq + (two ? y : 0)) >> 1) & 1)) return false;
    int kst, vst;
    auto scores = [&](int i) -> bool {
      if (!full(k_place(i), kst)) return false;
      tc::fence_after_sync();
      issue_mods_scores<D>(s_col, dq0 + qb * (SM::kTile >> 4), dk0 + kst * kStage, kIdescS);
      tc::mma_commit(&sm.s_ready[y]);
      return true;
    };
    if (first < tiles) {
      if (!scores(first)) return false;
      release(kst);
    }
    if (first + step >= tiles) {
      tc::mma_commit(&sm.q_empty[nq & 1]);
      if (two) tc::mma_commit(&sm.q_empty[(nq + 1) & 1]);
    }
    for (int i = first; i < tiles; i += step) {
      if (!wait(&sm.p_half[y], np & 1)) return false;
      if (i == first && nit >= 1 && !wait(&sm.o_free[y], (nit - 1) & 1))
        return false;  // the previous item's O has been read out
      if (!full(v_place(i, tiles), vst)) return false;
      const int ts = i == tiles - 1 ? x.tail : -1;
      const uint64_t dv = dv0 + vst * kStage, dt = dt0 + (ntail & 1) * (SM::kTail >> 4);
      if (ts >= 0 && !wait(&sm.tail_full[ntail & 1], (ntail >> 1) & 1)) return false;
      // with two query tiles the products take turns, in the order of the tiles: the two
      // softmax warpgroups then stay half a period apart, one at work while the other's
      // MMAs run (1054 against 807 us with 16384 states)
      if (two && (y == 1 || others)) {
        if (!wait(&sm.turn[y], turns & 1)) return false;
        ++turns;
      }
      others |= two;
      tc::fence_after_sync();
      // 64 states' weights while the softmax is at the others'
      issue_half<0>(o_col, s_col, dv, dt, ts, i != first, kIdescO);
      tc::mma_commit(&sm.o_half[y]);
      if (!wait(&sm.p_ready[y], np & 1)) return false;
      ++np;
      tc::fence_after_sync();
      issue_half<kTileKeys / 32>(o_col, s_col, dv, dt, ts, 1, kIdescO);
      if (i + step < tiles) {
        if (!scores(i + step)) return false;
        if (two) mbar_arrive(&sm.turn[y ^ 1]);
        release(vst);
        release(kst);
        if (i + 2 * step >= tiles) {  // the item's last scores
          tc::mma_commit(&sm.q_empty[nq & 1]);
          if (two) tc::mma_commit(&sm.q_empty[(nq + 1) & 1]);
        }
      } else {
        if (two) mbar_arrive(&sm.turn[y ^ 1]);
        tc::mma_commit(&sm.o_done[y]);
        release(vst);
      }
    }
    if (first < tiles) ++nit;
    if (x.tail >= 0) {
      // (waited for also where the other one used it: the buffer's phases keep their order)
      if (!wait(&sm.tail_full[ntail & 1], (ntail >> 1) & 1)) return false;
      tc::mma_commit(&sm.tail_free[ntail & 1]);
      ++ntail;
    }
    nq += two ? 2 : 1;
    base += 2 * tiles;
  }
}

template <class QT, int D, bool kFP8>
__device__ __forceinline__ void cross_issuer(const AttnParams& p, CrossSmem<D, kFP8>& sm, uint32_t tmem, int y) {
  y = __shfl_sync(kFull, y, 0);  // (the same in every lane for the compiler, too)
  if (tc::elect_one()) {
    if (!issue_group<QT, D, kFP8>(p, sm, tmem, y)) flag_error(p.errors, PKV_DEVERR_TIMEOUT);
    tc::mma_commit(&sm.mma_done);
    mbar_wait(&sm.mma_done, 0, 100000000ull);
  }
  __syncwarp();
}

// Weights 2^z of 32 states, rounded to 16 bits, as 16 packed pairs, and the fp32 sums of what
// they were rounded to: out = sum(p v) / sum(p) is then a mean with weights a rounding off, and
// a state that has all but all the weight is given back as it is.  (Sums that take the 16-bit
// halves as they are: 766 us for four prompts of 1024 tokens over 16384 states, 779 with
// halves widened before.)
template <class PT>
__device__ __forceinline__ void weights(const float* z, float* pk, float2* sums) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const uint32_t u = pack2<PT>(fast_exp2(z[e]), fast_exp2(z[e + 1]));
    float2& t = sums[(e >> 1) & 3];
    if constexpr (std::is_same<PT, BF16>::value)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.f32.bf16 %0, lo, %0;\n\tadd.f32.bf16 %1, hi, %1;\n\t}"
          : "+f"(t.x), "+f"(t.y) : "r"(u));
    else
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.f32.f16 %0, lo, %0;\n\tadd.f32.f16 %1, hi, %1;\n\t}"
          : "+f"(t.x), "+f"(t.y) : "r"(u));
    pk[e >> 1] = __uint_as_float(u);
  }
}

// ---- softmax and epilogue ------------------------------------------------------------------
// Thread = row of a query tile.  Warpgroup y: query tile y, or (one query tile) the even or
// odd key tiles.
template <class QT, int D, bool kFP8>
__device__ __forceinline__ void cross_softmax(const AttnParams& p, const CrossArgs& c,
                                              CrossSmem<D, kFP8>& sm, uint32_t tmem) {
  using OutT = typename QT::T;
  using PT = ProductType<QT, kFP8>;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int y = warp >> 2, g = p.group, r = threadIdx.x & 127;
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_col = tmem + lane_off + y * 128;
  const uint32_t o_col = tmem + lane_off + kColO + y * 128;
  const uint32_t o_other = tmem + lane_off + kColO + (y ^ 1) * 128;
  const float qs = p.q_scale == 0.0f ? 1e-30f : p.q_scale;  // (2^(s * 1e-30) rounds to 1)
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(kFull, wait_for(bar, parity, abort, lim)) != 0;
  };
  uint32_t ns = 0, nit = 0, nother = 0;  // steps and items of this warpgroup; joins
  bool ok = true;
  for (uint32_t n = 0;; ++n) {
    // the item stays in shared memory until the warp is done with it (its fields would cost
    // the loop registers)
    ok = wait(&sm.item_full[n % kItems], (n / kItems) & 1);
    const CrossItem& x = sm.item[n % kItems];
    if (!ok || !x.live) break;
    auto done = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_read[n % kItems]);
    };
    const bool two = x.nt[1] > 0;
    const int qt = two ? y : 0, kt0 = x.kt0, kt1 = x.kt1;
    const int rows = x.nt[qt] * g;                    // rows past the tokens are never stored
    const bool idle = 32 * (warp & 3) >= rows;        // the warp has no others
    // the row's place in the output, in heads
    auto head_of = [&]() { return (x.q0 + x.t0[qt] + r / g) * p.num_heads + x.kvh * g + r % g; };
    if (kt0 == kt1) {  // no states
      if (r < rows && (two || y == 0)) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<OutT*>(p.out) + (size_t)head_of() * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
      }
      done();
      continue;
    }
    const int step = two ? 1 : 2, first = two ? kt0 : kt0 + y;
    if (first >= kt1) {  // one key tile: the other warpgroup's
      done();
      continue;
    }
    int left = x.len - first * kTileKeys;             // states from the tile on
    float m_run = -INFINITY;
    float2 l2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) l2[i] = make_float2(0.0f, 0.0f);
    for (int t = first; t < kt1; t += step, left -= step * kTileKeys, ++ns) {
      ok = wait(&sm.s_ready[y], ns & 1);
      if (!ok) break;
      if (!idle) {
        tc::fence_after_sync();
        if (left < kTileKeys) {
          // the last tile: scores past the states become those of weight zero, where they are
          // (tests in the loop below would cost every tile 128 selections)
          const float none = qs > 0.0f ? -INFINITY : INFINITY;
#pragma unroll 1
          for (int k = left & ~31; k < kTileKeys; k += 32) {
            float sv[32];
            tc::tmem_ld32(s_col + k, sv);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[e] = k + e < left ? sv[e] : none;
            tc::tmem_st32(s_col + k, sv);
          }
          tc::tmem_wait_st();
        }
        // 64 states at a time: weights 2^(s * scale - m) with m as it is.  Their sum tells
        // whether that m will do for all rows of the warp, as it nearly always does; else m
        // moves for those that it does not do for, what they have so far is scaled to it, and
        // the weights are taken again.  (The maximum of every tile first costs 570 of a
        // step's 2000 cycles.)
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float pk[32];
          float2 t2[4];
          const uint32_t s_at = s_col + 64 * half;
#pragma unroll 1
          for (int again = 0;; again = 1) {
            const float m = m_run == -INFINITY ? 0.0f : m_run;
            const float2 f2 = make_float2(qs, qs), m2 = make_float2(-m, -m);
            auto exponents = [&](float* sv) {  // of 32 scores, in place
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 v = __ffma2_rn(make_float2(sv[e], sv[e + 1]), f2, m2);
                sv[e] = v.x;
                sv[e + 1] = v.y;
              }
            };
            float sv[2][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) t2[i] = make_float2(0.0f, 0.0f);
            tc::tmem_ld32(s_at, sv[0]);
            tc::tmem_wait_ld();
            tc::tmem_ld32(s_at + 32, sv[1]);
            exponents(sv[0]);
            weights<PT>(sv[0], pk, t2);
            tc::tmem_wait_ld();
            exponents(sv[1]);
            weights<PT>(sv[1], pk + 16, t2);
            const float sum = ((t2[0].x + t2[0].y) + (t2[1].x + t2[1].y)) +
                              ((t2[2].x + t2[2].y) + (t2[3].x + t2[3].y));
            // (what rows past the tokens hold does not matter)
            const bool off = r < rows && (m_run == -INFINITY || sum > kMostSum);
            // (once over is enough: only scores of 2^27 and more, whose differences fp32 does
            // not hold, could exceed their own maximum)
            if (again || !__any_sync(kFull, off)) break;
            float mz = -INFINITY;
#pragma unroll 1
            for (int k = 0; k < 64; k += 32) {
              float z[32];
              tc::tmem_ld32(s_at + k, z);
              tc::tmem_wait_ld();
              exponents(z);
#pragma unroll
              for (int e = 0; e < 32; e += 2) mz = fmax3(mz, z[e], z[e + 1]);
            }
            const bool move = off && mz > -INFINITY;
            mz -= kLift;
            // (a row without a weight so far has zeros)
            const float alpha = !move ? 1.0f : m_run == -INFINITY ? 0.0f : fast_exp2(-mz);
            if (move) m_run = m + mz;
#pragma unroll
            for (int i = 0; i < 4; ++i) l2[i] = __fmul2_rn(l2[i], make_float2(alpha, alpha));
            // O holds the tiles before this one (its scores were issued behind their product),
            // and the first half of this one
            if (half == 1 || t > first) {
              if (half == 1) {
                ok = wait(&sm.o_half[y], ns & 1);
                if (!ok) break;
                tc::fence_after_sync();
              }
#pragma unroll 1
              for (int k = 0; k < D; k += 32) {
                float ov[32];
                tc::tmem_ld32(o_col + k, ov);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                tc::tmem_st32(o_col + k, ov);
              }
            }
          }
          if (!ok) break;
          // P over scores that have been read
          tc::tmem_st32(s_col + 32 * half, pk);
#pragma unroll
          for (int i = 0; i < 4; ++i) l2[i] = __fadd2_rn(l2[i], t2[i]);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (half == 0 && lane == 0) mbar_arrive(&sm.p_half[y]);
        }
        if (!ok) break;
      } else if (lane == 0) {
        mbar_arrive(&sm.p_half[y]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_ready[y]);
    }
    if (!ok) break;
    ok = wait(&sm.o_done[y], nit & 1);
    ++nit;
    if (!ok) break;
    tc::fence_after_sync();
    float l = ((l2[0].x + l2[0].y) + (l2[1].x + l2[1].y)) + ((l2[2].x + l2[2].y) + (l2[3].x + l2[3].y));
    float a0 = 1.0f, a1 = 0.0f;
    const bool join = !two && kt1 - kt0 > 1;
    if (join) {
      if (y != ((kt1 - kt0 - 1) & 1)) {  // its maxima, sums and O are for the other warpgroup
        sm.other[r] = make_float2(m_run, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.other_ready);
        ++nother;
        done();
        continue;
      }
      ok = wait(&sm.other_ready, nother & 1);
      ++nother;
      if (!ok) break;
      tc::fence_after_sync();
      const float2 o = sm.other[r];
      const float m = fmaxf(m_run, o.x), mm = m == -INFINITY ? 0.0f : m;
      a0 = fast_exp2(m_run - mm);
      a1 = fast_exp2(o.x - mm);
      l = l * a0 + o.y * a1;
      m_run = m;
    }
    const bool none = l == 0.0f;  // (every score -inf)
    const float inv = p.v_scale / l;
    a0 *= inv;
    a1 *= inv;
    // 32 dimensions of the row from k on, divided and (one query tile) joined
    auto result = [&](int k, float* ov) {
      tc::tmem_ld32(o_col + k, ov);
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) ov[e] *= a0;
      if (join) {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          float ow[16];
          tc::tmem_ld16(o_other + k + h, ow);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) ov[h + e] = fmaf(ow[e], a1, ov[h + e]);
        }
      }
    };
    const int part = x.part;
    if (!idle) {
      if (part >= 0) {
        const int at = part * c.part_rows + qt * 128 + r;
        float4* o = reinterpret_cast<float4*>(p.o_part + (size_t)at * D);
        if (r < rows) p.lse[at] = none ? -INFINITY : m_run + log2f(l);
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          float ov[32];
          result(k, ov);
          if (r < rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              o[(k + e) / 4] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                    : make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
          }
        }
      } else {
        // four lanes exchange their rows' 16-byte pieces, so that they store 64 contiguous
        // bytes of one row at a time
        const int head = r < rows ? head_of() : -1;
        int place[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) place[i] = __shfl_sync(kFull, head, (lane & 28) + i);
        const bool up2 = lane & 2, up1 = lane & 1;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          float ov[32];
          result(k, ov);
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = make_uint4(pack2<QT>(ov[8 * i], ov[8 * i + 1]), pack2<QT>(ov[8 * i + 2], ov[8 * i + 3]),
                              pack2<QT>(ov[8 * i + 4], ov[8 * i + 5]), pack2<QT>(ov[8 * i + 6], ov[8 * i + 7]));
          auto swap = [&](uint4& a, uint4& b, bool up, int mask) {  // a of the upper lane for b of the lower
            uint4 t = up ? a : b;
            t.x = __shfl_xor_sync(kFull, t.x, mask);
            t.y = __shfl_xor_sync(kFull, t.y, mask);
            t.z = __shfl_xor_sync(kFull, t.z, mask);
            t.w = __shfl_xor_sync(kFull, t.w, mask);
            if (up) a = t; else b = t;
          };
          swap(w[0], w[2], up2, 2);
          swap(w[1], w[3], up2, 2);
          swap(w[0], w[1], up1, 1);
          swap(w[2], w[3], up1, 1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (place[i] >= 0)
              *reinterpret_cast<uint4*>(static_cast<OutT*>(p.out) + (size_t)place[i] * D + k +
                                        8 * (lane & 3)) = w[i];
        }
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.o_free[y]);
      if (join) mbar_arrive(&sm.o_free[y ^ 1]);
    }
    done();
  }
  if (!ok && lane == 0) flag_error(p.errors, PKV_DEVERR_TIMEOUT);
}

template <class QT, int D, bool kFP8>
__global__ void __launch_bounds__(cross_threads(kFP8), 1)
    cross_kernel(const AttnParams p, const CrossArgs c, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                 int kv_rows) {
  extern __shared__ uint8_t smem_raw[];
  using SM = CrossSmem<D, kFP8>;
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  if (warp >= kTma && warp < kTma + kTmaWarps && (threadIdx.x & 31) == 0) {
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
    tc::prefetch_tmap(&tm_q);
  }
  cross_setup<D, kFP8>(p, c, sm);
  const uint32_t tmem = sm.tmem_base;
  if (warp >= kSoft) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(cross_other_regs(kFP8)));
    if (warp < kIssuer + kIssuers) cross_issuer<QT, D, kFP8>(p, sm, tmem, warp - kIssuer);
    else if (warp < kTma + kTmaWarps)
      cross_producer<D, kFP8>(p, c, sm, tm_k, tm_v, tm_q, kv_rows, warp - kTma);
    else if constexpr (kFP8) cross_converter<QT, D>(p, sm, warp - kConvert);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(cross_soft_regs(kFP8)));
    cross_softmax<QT, D, kFP8>(p, c, sm, tmem);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the unit that CTA blockIdx.x's part of the line ends in, if it ends
// inside one: weights 2^(lse - max) of the parts, which that CTA wrote as its second partial
// and the CTAs up to the last one as their first.  A warp per row.
constexpr int kJoinThreads = 256;
template <class QT, int D>
__global__ void __launch_bounds__(kJoinThreads) cross_join_kernel(const AttnParams p, const CrossArgs c) {
  using OutT = typename QT::T;
  tc::grid_dependency_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int4 cut = __ldcg(c.cuts + 2 * b);
  if (cut.x < 0) return;
  const int kvh = __ldcg(&c.cuts[2 * b + 1].x);
  const int last = cut.x, g = p.group, rpt = kRowsM / g;
  const int warps = gridDim.y * (kJoinThreads / 32);
  for (int at = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); at < c.part_rows; at += warps) {
    const int qt = at >> 7, r = at & 127;
    if (r >= (qt ? cut.w : cut.z) * g) continue;
    auto slot = [&](int i) { return (size_t)(2 * (b + i) + (i == 0 ? 1 : 0)) * c.part_rows + at; };
    const int parts = last - b + 1;
    constexpr int kLanes = D / 4, kAhead = 4;
    auto value = [&](int i) {
      return i < parts && lane < kLanes
                 ? __ldcg(reinterpret_cast<const float4*>(p.o_part + slot(i) * D) + lane)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 v[kAhead];  // on their way while the weights are found
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = value(u);
    const float lse = lane < parts ? __ldcg(p.lse + slot(lane)) : -INFINITY;
    float m = lse;
    for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, __ldcg(p.lse + slot(i)));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float mine = exp2f(lse - m);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.0f;
    for (int i0 = 0; i0 < parts; i0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u;
        if (i >= parts) break;
        const float w = i < 32 ? __shfl_sync(kFull, mine, i) : exp2f(__ldcg(p.lse + slot(i)) - m);
        sum += w;
        acc.x = fmaf(w, v[u].x, acc.x);
        acc.y = fmaf(w, v[u].y, acc.y);
        acc.z = fmaf(w, v[u].z, acc.z);
        acc.w = fmaf(w, v[u].w, acc.w);
      }
      if (i0 + kAhead < parts) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) v[u] = value(i0 + kAhead + u);
      }
    }
    if (lane < kLanes) {
      const float inv = 1.0f / sum;
      OutT* o = static_cast<OutT*>(p.out) +
                ((size_t)(cut.y + qt * rpt + r / g) * p.num_heads + kvh * g + r % g) * D + 4 * lane;
      const uint2 w = make_uint2(pack2<QT>(acc.x * inv, acc.y * inv), pack2<QT>(acc.z * inv, acc.w * inv));
      *reinterpret_cast<uint2*>(o) = w;
    }
  }
}

template <class QT, int D, bool kFP8>
int launch_cross_typed(const AttnParams& p, const CrossArgs& c, int ctas, cudaStream_t stream) {
  const bool bf16 = std::is_same<QT, BF16>::value;
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  CUtensorMap tk, tv, tq;
  const int type = kFP8 ? PKV_FP8_E4M3 : (bf16 ? PKV_BF16 : PKV_F16);
  if (!make_map_rows(&tk, p.k_cache, kv_rows, D, type, kBlockSize) ||
      !make_map_rows(&tv, p.v_cache, kv_rows, D, type, kBlockSize) ||
      !make_map_heads(&tq, p.q, (uint64_t)p.num_rows, (uint32_t)p.num_heads, D, bf16,
                      (uint32_t)p.group, (uint32_t)c.box_tokens))
    return PKV_ERR_CUDA;
  using SM = CrossSmem<D, kFP8>;
  constexpr size_t smem = sizeof(SM) + 1024;
  static_assert(smem <= 232448, "shared memory budget of one CTA");
  static_assert(offsetof(SM, ring) % 1024 == 0 && offsetof(SM, q) % 1024 == 0 &&
                    offsetof(SM, tail) % 1024 == 0 && SM::kStage % 1024 == 0 && SM::kTail % 1024 == 0,
                "swizzled buffers must start on 1024-byte boundaries");
  auto kern = cross_kernel<QT, D, kFP8>;
  // the kernel's register shares add up to what its launch holds; with fewer its
  // warpgroups would wait for registers without end
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != cross_launch_regs(kFP8)) return PKV_ERR_CUDA;
  static std::atomic<unsigned long long> configured{0};
  if (!smem_once(kern, smem, configured)) return PKV_ERR_CUDA;
  kern<<<ctas, cross_threads(kFP8), smem, stream>>>(p, c, tk, tv, tq, (int)kv_rows);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  if (!c.cuts) return PKV_OK;
  // a CTA of the join for each of the kernel's and up to 32 rows
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, (c.part_rows + 31) / 32);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_join_kernel<QT, D>, p, c) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D>
int launch_cross_dim(const AttnParams& p, const CrossArgs& c, int q_dtype, int kv_dtype, int ctas,
                     cudaStream_t stream) {
  const bool fp8 = kv_dtype == PKV_FP8_E4M3;
  if (q_dtype == PKV_BF16)
    return fp8 ? launch_cross_typed<BF16, D, true>(p, c, ctas, stream)
               : launch_cross_typed<BF16, D, false>(p, c, ctas, stream);
  return fp8 ? launch_cross_typed<F16, D, true>(p, c, ctas, stream)
             : launch_cross_typed<F16, D, false>(p, c, ctas, stream);
}

}  // namespace
}  // namespace cross_tc
}  // namespace pkv

#endif  // PKV_CROSS_TC_CUH

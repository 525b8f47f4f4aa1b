// Biased chunked prefill on the tcgen05 tensor cores (head_dim 64 or 128, fp16/bf16
// or E4M3 caches, any group size up to 16): capped scores, a distance bias, and an
// interval of visible keys per query row (score_mods.cuh).  The mathematics and
// the layouts are those of prefill_tc.cuh; what differs:
//
//  * What a modified score costs is instructions of the softmax (one thread per row, two
//    warps per scheduler), whose code is long and fetched anew at each step; so there is
//    one kernel per set of modifiers, scores are modified in place (the exponentials' code
//    stands once), and a step is 64 keys, half of a loaded tile.  Four warps per scheduler,
//    two per row with 32 keys each and their maxima exchanged, were slower (a cap on the
//    mixed batch's chunks 122 against 110 us), and so were steps of 128 keys (124).
//  * A query tile has two score buffers, so that its softmax has the next step's scores at
//    hand.  Two issuers share the MMAs (all from one: cap 128 against 109, packed documents
//    171 against 124 us; an issuer's single thread needs 1500 cycles for a tile's step; four
//    of them slow the softmax beside them: cap 119).  Score MMAs of 64 keys take 72 % of the
//    time of 128; that and the issuers bound the kernel without modifiers (85 us on the
//    chunks, as the plain kernel's 83).
//  * An item (two query tiles of whole tokens) walks the keys from its first row's first
//    one to its last row's last one; blocks before and behind those are not read.  A
//    step that every row of a warp sees is not masked; one that none sees costs no
//    exponentials, only zeros for P.
//  * A running CTA takes over the next item not launched yet instead of owning a fixed
//    share.  Items are short (the packed documents': 11 steps), so what each costs once
//    counts: one warp makes them ahead of the others, and four lanes gather 64 bytes of a
//    row before they store (134 -> 120 us for the documents).
//  * A distance bias grows towards the query, so the running max would move, and O
//    be rescaled, at nearly every step of a walk towards it; those kernels walk from the
//    last key back.
//  * A key hidden from a row has weight zero, but in the product 0 * inf is NaN: rows whose
//    output is not finite are looked at again after the main loop (redo_rows), by the warp
//    that wrote them, so that a hidden infinity never reaches them.  Finite inputs never
//    take that path.
//  * E4M3 caches: five more warps turn each K or V tile into the query's 16-bit type
//    (exactly) where it lands, once for both query tiles, and everything
//    behind is as for 16-bit caches: no rounding but theirs, and no pass over the query.
//    8-bit products instead need the query and P as two E4M3 terms each to be as good
//    (one term of P alone is 2 % of the output's norm), and that splitting is on the
//    softmax warps: 211 us against 132 for the same prompts on a 16-bit cache.
//
// Measured (calls one behind the other, on changing inputs): window 1024 and cap 50 on 4
// chunks of 512 behind 2048 tokens, 32 query heads, 8 KV heads, 60 us (572 TFLOP/s of the
// visible products); documents packed into 8191 tokens with a bias 118 us (685); six
// prompts with two-way prefixes on an E4M3 cache 135 us (674).  head_dim 64, from cold
// caches: those chunks 56 us with window and cap, 71 without (keys only; head_dim 128: 78).
#ifndef PKV_PREFILL_MODS_CUH
#define PKV_PREFILL_MODS_CUH

#include "prefill_tc.cuh"
#include "score_mods.cuh"

namespace pkv {
namespace pre_mods {
namespace {
using namespace pre_tc;

// Modifiers that a kernel is built for, as bits: tests in the tile loop instead
// would have every case pay the registers of all.
constexpr int kModCap = 1, kModBias = 2;

// Waits for a barrier's phase, at most limit_ns or until the CTA gives up; the clock is
// only read once the wait has been long (reading it takes longer than most waits).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         unsigned long long limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !mbar_test(bar, parity); ++it) {
    if ((it & 63u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort) return false;
      if (now - t0 > limit_ns) {
        *abort = 1;
        return false;
      }
    }
  }
  return true;
}

constexpr int kTileWarps = 4;  // softmax warps of a query tile
constexpr int kSoftWarps = 2 * kTileWarps;
constexpr int kIssuers = 2;
// What the issuers share out: scores and products of both query tiles, or the query
// tiles.  By role, the products' order keeps the two softmax warpgroups in step; that
// suits them while they are not bound by the pipes they share, in items of many steps, not
// with a cap (118 us against 109 on the mixed batch's chunks; with a bias, too, 130 against
// 126) or where converter warps work beside them (E4M3 prompts 142 against 138).  Measured
// without a cap, by role against by tile, keys only and with a bias: those chunks 82
// against 92 and 87 against 98; with a window of 1024 50 / 51 and 51 / 55, of 256 equal;
// 8191 tokens with a window of 64 49 / 48 and 59 / 53 (32 KV heads 78 / 70 and 82 / 75);
// cut into documents of 50 tokens 50 / 49 and 59 / 55, of 200 59 / 56 and 68 / 63, of 800
// 82 / 86 and 94 / 91, of 2000 136 / 146 and 148 / 156, of 5000 231 / 256 and 247 / 268.
// So by role where items are long by the call's own sizes: no window, or one of at least
// 512.  How long first keys leave them is not known at the launch; they are taken for
// short ones, which costs documents of thousands of tokens 5 to 13 %.
constexpr int kLongWindow = 512;
template <bool kFP8, int kMods>
__device__ __forceinline__ bool by_role(const AttnParams& p) {
  return !kFP8 && (kMods & kModCap) == 0 && p.key_start == nullptr &&
         (p.window == 0 || p.window >= kLongWindow);
}
constexpr int kWarpMma = kSoftWarps, kWarpTma = kSoftWarps + kIssuers;
// Warps beside softmax and issuers, and threads of the CTA: two producers, or (E4M3
// caches) one and five that convert its tiles.
constexpr int kConverters = 5;
constexpr int mod_producers(bool fp8) { return fp8 ? 1 : 2; }
constexpr int mod_extra(bool fp8) { return mod_producers(fp8) + (fp8 ? kConverters : 0); }
constexpr int mod_threads(bool fp8) { return 32 * (kSoftWarps + kIssuers + mod_extra(fp8)); }
// Registers per thread: the launch gives 168 to each of 384 threads, enough for all, and
// 128 to each of 512 (E4M3 caches), of which the two softmax warpgroups take over what
// the others return.  (Stated for both: without, the compiler lays the 16-bit kernels out
// 3 % slower.)
constexpr int soft_regs(bool fp8) { return fp8 ? 152 : 168; }
constexpr int other_regs(bool fp8) { return fp8 ? 104 : 168; }
constexpr int launch_regs(bool fp8) { return fp8 ? 128 : 168; }
constexpr bool regs_fit(bool fp8) {
  return 32 * kSoftWarps * soft_regs(fp8) + (mod_threads(fp8) - 32 * kSoftWarps) * other_regs(fp8) <=
         mod_threads(fp8) * launch_regs(fp8);
}
static_assert(regs_fit(false) && regs_fit(true) && mod_threads(false) == 384 && mod_threads(true) == 512,
              "setmaxnreg may only share out what the launch holds");
constexpr int kChunk = 32;  // keys whose weights are packed and stored together
constexpr int kStepKeys = kTileKeys / 2;  // keys of a step: half a loaded tile
constexpr int kAhead = 4;   // items made before the slowest warp takes them
// Items that a softmax warp can list for redo_rows.  A CTA whose list could not take what
// it has under way and one more leaves the rest of the grid to others: when it asks for
// item n + 1, its warps have listed items up to n - 2 - kAhead.
constexpr int kRedo = 32;
constexpr int kUnderWay = kAhead + 3;

// Two query tiles of a sequence and KV head, and the keys they see.
struct ModItem {
  int k;               // its number in the launch, -1: no further item
  int seq, kvh, ctx, q0;
  int bidir;           // keys every query of the sequence sees (0: causal)
  int t0[2], nt[2];    // first token (within the chunk) and tokens of tiles a, b
  int pos0[2];         // absolute position of each tile's first token
  int h0, nh;          // halves [h0, nh) of key tiles (64 keys) of the item
  int kt0, nk;         // the key tiles [kt0, nk) they lie in (nk 0: no row sees a key)
  int last[2];         // last step of each query tile (-1: its rows see nothing)
  int lo_block, end_block;  // blocks any row sees
  int tail_step;       // MMA step of key tile nk - 1 holding the partial last block, in half
                       // nh - 1, else -1 (E4M3 caches: -1)
};

template <bool kFP8>
struct ModSmem {
  alignas(1024) uint8_t ring[kStages][kTileBytes];
  alignas(1024) uint8_t q[2][kTileBytes];
  alignas(1024) uint8_t tail[kTailBytes];  // V rows of a partial block (16-bit caches)
  int seq_start[kMaxSeqs + 1];  // prefix of items per sequence (one KV head's)
  int seq_qlen[kMaxSeqs];
  int seq_ctx[kMaxSeqs];
  int seq_q0[kMaxSeqs];
  int scan[mod_threads(kFP8) / 32];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t staged[kStages];  // an E4M3 tile has landed in the second half of its stage
  uint64_t q_full;
  uint64_t q_empty;
  uint64_t s_ready[2][2];  // per query tile and score buffer
  uint64_t p_ready[2][2];
  uint64_t o_done[2][2];  // the product of that buffer's P
  uint64_t o_free[2];
  uint64_t tail_full;
  uint64_t tail_free;
  uint64_t mma_done[kIssuers];
  alignas(16) unsigned long long answer[2];  // to the request for a further item
  uint64_t answer_full;
  ModItem item[kAhead];  // item n of the CTA in slot n % kAhead
  uint64_t item_full[kAhead];
  uint64_t item_read[kAhead];
  uint32_t tmem_base;
  int abort;
  // items with rows that came out not finite, by softmax warp (its rows as bits)
  int redo_n[kSoftWarps];
  int redo_item[kSoftWarps][kRedo];
  uint32_t redo_rows[kSoftWarps][kRedo];
};

// Loads go through an item's key tiles, kt0 + i being the i-th one (backwards under a
// bias: nk - 1 - i), the products through their halves, step v = 0 .. nh - h0 - 1.
template <int kMods>
__device__ __forceinline__ int tile_of(const ModItem& x, int i) {
  return (kMods & kModBias) ? x.nk - 1 - i : x.kt0 + i;
}
template <int kMods>
__device__ __forceinline__ int half_of(const ModItem& x, int v) {
  return (kMods & kModBias) ? x.nh - 1 - v : x.h0 + v;
}

// Item k of the launch, or (k past the last one) an item without keys or rows.
template <int kMods, bool kFP8>
__device__ __forceinline__ void make_item(const AttnParams& p, const ModSmem<kFP8>& sm, int k, int total,
                                          ModItem& it) {
  if (k >= total) {
    it = ModItem{};
    it.k = k;
    it.last[0] = it.last[1] = it.tail_step = -1;
    return;
  }
  it.k = k;
  it.kvh = k % p.num_kv_heads;
  const int pair = k / p.num_kv_heads;
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.seq_start[mid] <= pair) lo = mid; else hi = mid - 1;
  }
  const int rpt = kRowsM / p.group;  // tokens per query tile
  const int qlen = sm.seq_qlen[lo];
  it.seq = lo;
  it.ctx = sm.seq_ctx[lo];
  it.q0 = sm.seq_q0[lo];
  it.bidir = p.bidir_lens ? min(__ldg(p.bidir_lens + lo), it.ctx) : 0;
  // the sequence's last pair of tiles, the longest without a window, first
  const int mp = sm.seq_start[lo + 1] - 1 - pair;
  int lo_min = INT_MAX, hi_max = 0, end[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    it.t0[x] = (2 * mp + x) * rpt;
    it.nt[x] = max(0, min(rpt, qlen - it.t0[x]));
    it.pos0[x] = it.ctx - qlen + it.t0[x];
    end[x] = 0;
    if (it.nt[x] > 0) {
      // the first row has the tile's smallest first key, the last row that sees a
      // key its largest end
      const int* start = p.key_start ? p.key_start + it.q0 + it.t0[x] : nullptr;
      int pos = it.pos0[x] + it.nt[x] - 1;
      int h = max(pos + 1, it.bidir), first = 0;
      while (start && pos >= it.pos0[x] && __ldg(start + (pos - it.pos0[x])) >= h) {
        --pos;
        h = pos >= it.pos0[x] ? max(pos + 1, it.bidir) : 0;
      }
      if (start) first = max(first, __ldg(start));
      if (p.window > 0) first = max(first, it.pos0[x] - p.window + 1);
      if (first < h) {
        end[x] = (h - 1) / kStepKeys + 1;
        lo_min = min(lo_min, first);
        hi_max = max(hi_max, h);
      }
    }
  }
  it.nh = max(end[0], end[1]);
  it.nk = (it.nh + 1) / 2;
  it.h0 = it.nk > 0 ? lo_min / kStepKeys : 0;
  it.kt0 = it.h0 / 2;
  it.lo_block = it.nk > 0 ? lo_min / kBlockSize : 0;
  it.end_block = (hi_max + kBlockSize - 1) / kBlockSize;
#pragma unroll
  for (int x = 0; x < 2; ++x)
    it.last[x] = end[x] > 0 ? ((kMods & kModBias) ? it.nh : end[x]) - 1 - it.h0 : -1;
  const bool partial = !kFP8 && (it.ctx & (kBlockSize - 1)) != 0;
  it.tail_step = partial && (it.ctx - 1) / kStepKeys == it.nh - 1
                     ? ((it.ctx - 1) % kTileKeys) / kBlockSize
                     : -1;
}

// Items differ in length (documents, windows, causal chunks), so a CTA does not own a
// fixed share: the grid has a CTA per item, and a running CTA takes over the next one
// not launched yet (clusterlaunchcontrol) each time it begins one.  Round robin over
// 152 CTAs left the longest 30 % above the mean for the packed documents.
//
// Producer warp 0 makes the items, for all warps: it asks for the one after next when it
// begins one, and leaves each in shared memory, ahead of the warps that need it (made by
// every warp for itself, an item cost the softmax 2500 cycles of index arithmetic and
// dependent loads).  No request follows one that found the grid empty; an item -1 ends
// every warp's loop.
template <bool kFP8>
__device__ __forceinline__ void ask_next(ModSmem<kFP8>& sm) {
  mbar_arrive_expect_tx(&sm.answer_full, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::
          "r"(smem_u32(&sm.answer[0])),
      "r"(smem_u32(&sm.answer_full))
      : "memory");
}

// The answer to request m, for one thread: an item's number, -1 where there is none, -2
// when the wait gave up.
template <bool kFP8>
__device__ __forceinline__ int next_item(ModSmem<kFP8>& sm, uint32_t m, volatile int* abort,
                                         unsigned long long lim) {
  if (!wait_for(&sm.answer_full, m & 1, abort, lim)) return -2;
  const unsigned long long a = *static_cast<volatile unsigned long long*>(&sm.answer[0]);
  const unsigned long long b = *static_cast<volatile unsigned long long*>(&sm.answer[1]);
  uint32_t yes, index;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "mov.b128 r, {%2, %3};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(yes), "=r"(index)
      : "l"(a), "l"(b));
  fence_proxy_async_smem();  // read before a later answer overwrites it
  return yes ? (int)index : -1;
}

// The n-th item of this CTA, for a warp, or (kOne) for one thread of it; false when the
// wait gave up.
template <bool kOne, bool kFP8>
__device__ __forceinline__ bool take_item(ModSmem<kFP8>& sm, uint32_t n, ModItem& x, volatile int* abort,
                                          unsigned long long lim) {
  const int slot = n % kAhead;
  bool ok = wait_for(&sm.item_full[slot], (n / kAhead) & 1, abort, lim);
  if (!kOne) ok = __all_sync(kFull, ok);
  if (!ok) return false;
  x = sm.item[slot];
  if (!kOne) __syncwarp();
  if (kOne || (threadIdx.x & 31) == 0) mbar_arrive(&sm.item_read[slot]);
  return true;
}

// Largest magnitude of three values.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The scores of a step's 64 keys from k0 on, modified in place.  a > 0 takes a raw
// score to base-2 units, C = cap log2(e) is the cap in them.  Returns the factor
// still to be applied, which the exponential's own multiply-add carries: a where the
// score is only masked, 1 after a cap or a bias.
//
// The cap is C tanh(a s / C).  For a row whose scores all stay below half the cap, the
// usual case, it is s T(s^2), T(u) = a (1 + k3 c^2 u + k5 c^4 u^2 + ...),
// c = a / C: the polynomial of tanh with the scales folded into its coefficients, five
// operations on packed pairs and no exponential beside the softmax's own.  Otherwise
// C - 2 C / (2^(2 c log2(e) s) + 1): two more MUFU results per score, off by at most
// 2^-22 C, as much as the product behind the row's largest score is.  Each row chooses for
// itself (by a vote of the warp, a neighbour's large score, or what Q holds past the tile's
// tokens, would have cost the others their precision): a warp with rows of both kinds
// runs both.  Keys hidden from the row have no say either: where a score is large, the
// largest that the row sees is found from tensor memory, in a rolled loop (the hidden ones
// zeroed in registers instead, code beside the path that is taken, cost 5 us of 59 with a
// window).  The mixed batch's chunks: 106 us with the polynomial, 140
// without, 80 uncapped.  (One of degree 9 that holds up to 3/4 of the cap took 8 us more;
// folding either into the exponential's argument saves operations, but has the code of the
// exponentials twice, and was slower by 15.)
template <int kMods>
__device__ __forceinline__ float modify_scores(const AttnParams& p, float* sv, float a, float slope,
                                               uint32_t s_at, int pos, int k0, int lo, int hi,
                                               bool valid) {
  if constexpr (kMods == 0) return a;
  if constexpr ((kMods & kModCap) != 0) {
    const float c = a / p.cap_log2, C = p.cap_log2;
    float top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kStepKeys; i += 2)
      top[(i >> 1) & 3] = absmax3(top[(i >> 1) & 3], sv[i], sv[i + 1]);
    float most = absmax3(fmaxf(top[0], top[1]), top[2], top[3]) * c;
    if (__any_sync(kFull, !(most <= kTanhPoly) && (lo > k0 || hi < k0 + kStepKeys))) {
      // a large one may be hidden: the largest that the row sees, from the scores read again
      most = 0.0f;
#pragma unroll 1
      for (int i = 0; i < kStepKeys; i += 16) {
        float s[16];
        tc::tmem_ld16(s_at + i, s);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (k0 + i + e >= lo && k0 + i + e < hi) most = fmaxf(most, fabsf(s[e]));
      }
      most *= c;
    }
    if ((most <= kTanhPoly || !valid) && c <= 256.0f) {
      const float c2 = c * c;
      const float t1 = a * c2, t2 = t1 * c2, t3 = t2 * c2;
      const float2 q0 = make_float2(a, a), q1 = make_float2(t1 * kTanh3, t1 * kTanh3),
                   q2 = make_float2(t2 * kTanh5, t2 * kTanh5),
                   q3 = make_float2(t3 * kTanh7, t3 * kTanh7);
#pragma unroll
      for (int i = 0; i < kStepKeys; i += 2) {
        const float2 x = make_float2(sv[i], sv[i + 1]), u = __fmul2_rn(x, x);
        const float2 t = __ffma2_rn(u, __ffma2_rn(u, __ffma2_rn(u, q3, q2), q1), q0);
        const float2 y = __fmul2_rn(x, t);
        sv[i] = y.x;
        sv[i + 1] = y.y;
      }
    } else {
      const float k = 2.0f * kLog2e * c;
#pragma unroll
      for (int i = 0; i < kStepKeys; ++i) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fast_exp2(sv[i] * k) + 1.0f));
        sv[i] = fmaf(r, -2.0f * C, C);
      }
    }
    __syncwarp();
  }
  if constexpr ((kMods & kModBias) != 0) {
    // distance bias of key k0 + i: -slope |pos - k0 - i|; without the absolute value
    // where every row of the warp is behind the tile
    const float f = (kMods & kModCap) != 0 ? 1.0f : a;
    const float d0 = (float)(pos - k0), b0 = -slope * d0;
    if (__all_sync(kFull, pos >= k0 + kStepKeys - 1)) {
#pragma unroll
      for (int i = 0; i < kStepKeys; ++i) sv[i] = fmaf(sv[i], f, fmaf(slope, (float)i, b0));
    } else {
#pragma unroll
      for (int i = 0; i < kStepKeys; ++i) sv[i] = fmaf(sv[i], f, -slope * fabsf(d0 - (float)i));
    }
  }
  return 1.0f;
}

// Scores: S (128 rows x 64 keys, fp32 in TMEM at d) = Q K^T over D dimensions, 16 an MMA,
// within 64-dimension halves of 16 KB.
template <int D>
__device__ __forceinline__ void issue_mods_scores(uint32_t d, uint64_t dq, uint64_t dk,
                                                  uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
    tc::mma_f16(d, dq + off, dk + off, idesc, kk > 0);
  }
}

// Output: O (at d) (+)= P (TMEM at a, 16 keys per 8 columns) V, 16 keys an MMA; the one
// numbered ts (if >= 0) takes its V rows from the tail buffer.
__device__ __forceinline__ void issue_mods_pv(uint32_t d, uint32_t a, uint64_t dv, uint64_t dtail,
                                              int ts, uint32_t acc0, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < kStepKeys / 16; ++kk) {
    const uint64_t b = kk == ts ? dtail : dv + (uint64_t)((kk * (kBlockSize * 128)) >> 4);
    mma_f16_tmem_a(d, a + kk * 8, b, idesc, acc0 | (kk != 0 ? 1u : 0u));
  }
}

// One row (a query token's head) from its own keys alone, in fp32 (the plain online
// softmax, exp2f), into those elements of its output that are not finite.  Four lanes
// share the row, D / 4 dimensions each; gmask is their mask.
template <class QT, bool kFP8, int D>
__device__ __forceinline__ void exact_row(const AttnParams& p, int seq, int row, int h, int pos,
                                          int lo, int hi, unsigned gmask) {
  constexpr int kElem = kFP8 ? 1 : 2, kDims = D / 4;
  using T = typename QT::T;
  const int quarter = threadIdx.x & 3, kvh = h / p.group;
  const float slope = p.alibi ? __ldg(p.alibi + h) * kLog2e : 0.0f;
  const size_t at = ((size_t)row * p.num_heads + h) * D + quarter * kDims;
  float qf[kDims], acc[kDims], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < kDims / 8; ++c)
    to_float(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + at) + c), qf + 8 * c,
             QT());
#pragma unroll
  for (int d = 0; d < kDims; ++d) acc[d] = 0.0f;
  for (int j = lo; j < hi; ++j) {
    const int blk = __ldg(p.block_tables + (size_t)seq * p.max_blocks_per_seq + j / kBlockSize);
    const bool bok = blk >= 0 && blk < p.num_blocks;
    const size_t off = ((((size_t)(bok ? blk : 0) * p.num_kv_heads + kvh) * kBlockSize +
                         j % kBlockSize) * D + quarter * kDims) * kElem;
    float kv[kDims], dot = 0.0f;
    if (bok) {
      const uint4* kp = reinterpret_cast<const uint4*>(p.k_cache + off);
#pragma unroll
      for (int c = 0; c < kDims * kElem / 16; ++c) {
        if constexpr (kFP8) to_float(__ldg(kp + c), kv + 16 * c, E4M3());
        else to_float(__ldg(kp + c), kv + 8 * c, QT());
      }
#pragma unroll
      for (int d = 0; d < kDims; ++d) dot = fmaf(qf[d], kv[d], dot);
    }
    dot += __shfl_xor_sync(gmask, dot, 1);
    dot += __shfl_xor_sync(gmask, dot, 2);
    float sc = dot * p.q_scale;
    if (p.softcap > 0.0f) sc = p.cap_log2 * cap_tanh(sc / p.cap_log2);
    sc = fmaf(-slope, fabsf((float)(pos - j)), sc);
    if (!(sc <= m)) {  // (a NaN score too: the row's result is NaN)
      const float a = exp2f(m - sc);
      l *= a;
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] *= a;
      m = sc;
    }
    // (a score of -inf has no weight, also where no other has come yet)
    const float w = sc == -INFINITY ? 0.0f : exp2f(sc - m);
    l += w;
    if (l != l) break;  // so is every output of the row (the four lanes agree)
    if (bok) {
      const uint4* vp = reinterpret_cast<const uint4*>(p.v_cache + off);
#pragma unroll
      for (int c = 0; c < kDims * kElem / 16; ++c) {
        if constexpr (kFP8) to_float(__ldg(vp + c), kv + 16 * c, E4M3());
        else to_float(__ldg(vp + c), kv + 8 * c, QT());
      }
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] = fmaf(w, kv[d], acc[d]);
    }
  }
  const float inv = p.v_scale / l;
  T* op = static_cast<T*>(p.out) + at;
#pragma unroll
  for (int d = 0; d < kDims; ++d) {
    const float o = acc[d] * inv;
    if (fabsf(o) < INFINITY && !(fabsf((float)op[d]) < INFINITY)) store_out(op + d, o);
  }
}

// What an element of V is, from its bits: 0 finite, 1 NaN, 2 and 3 the infinities.
template <class QT, bool kFP8>
__device__ __forceinline__ int odd_kind(uint32_t bits) {
  if constexpr (kFP8) {
    return (bits & 0x7fu) == 0x7fu ? 1 : 0;
  } else {
    constexpr uint32_t kExp = std::is_same<QT, BF16>::value ? 0x7f80u : 0x7c00u;
    if ((bits & kExp) != kExp) return 0;
    return (bits & 0x7fffu) != kExp ? 1 : (bits & 0x8000u) ? 3 : 2;
  }
}

// The rows listed by softmax warp `warp`: their softmax sums are numbers, but an element of
// the output is not.  Where a V that the row sees is not finite in that dimension, so is
// the element, as the weights are positive; else a V of the item that is hidden from the
// row has reached it, and the row is computed again from its own keys (exact_row).
//
// Which it is takes one pass over the V rows of the item: each lane has D / 32 dimensions
// and keeps the last key so far with a NaN and with either infinity.  Rows see intervals of
// keys whose ends do not decrease, so the pass stops at each row's end in turn and asks
// whether such a key is at or behind its first one.  The pass costs about what loading the
// item did.  Rows are computed again only beside a V that their neighbours in the item see
// and they do not, a tile's worth or two for each such V.  A prompt of 8192 tokens, 32 query
// and 8 KV heads: 0.37 ms, with one infinite V in its first token 3.4 ms (the pass over
// every item), with a NaN in token 5000 18.9 ms (beside that the 63 tokens before it, their
// 5000 keys one by one).
template <class QT, bool kFP8, int kMods, int D>
__device__ __noinline__ void redo_rows(const AttnParams& p, const ModSmem<kFP8>& sm, int total, int warp) {
  using T = typename QT::T;
  constexpr int kElem = kFP8 ? 1 : 2, kDims = D / 32, kBits = 8 * kElem;
  const int lane = threadIdx.x & 31, g = p.group, qt = warp / kTileWarps;
  const int r0 = 32 * (warp % kTileWarps);  // the warp's first row of the tile
  const unsigned gmask = 0xFu << (lane & 28);
  const int n = sm.redo_n[warp];
  ModItem x;
  for (int i = 0; i < n; ++i) {
    make_item<kMods, kFP8>(p, sm, sm.redo_item[warp][i], total, x);
    const uint32_t rows = sm.redo_rows[warp][i];
    const int t0 = qt ? x.t0[1] : x.t0[0], pos0 = qt ? x.pos0[1] : x.pos0[0];
    const int32_t* table = p.block_tables + (size_t)x.seq * p.max_blocks_per_seq;
    int last[3][kDims];  // last key with a NaN, +inf, -inf
    uint32_t unseen[kDims];  // rows whose element is not finite without a key of theirs
#pragma unroll
    for (int e = 0; e < kDims; ++e) {
      last[0][e] = last[1][e] = last[2][e] = -1;
      unseen[e] = 0;
    }
    int j = x.lo_block * kBlockSize;
    auto scan_to = [&](int end) {  // keys [j, end), whole blocks where they last
      while (j < end) {
        const int b = j / kBlockSize, f = j % kBlockSize, m = min(kBlockSize, end - b * kBlockSize);
        const int blk = __ldg(table + b);
        if (blk >= 0 && blk < p.num_blocks) {  // (else zeros)
          const uint8_t* v = p.v_cache + ((size_t)blk * p.num_kv_heads + x.kvh) * (kBlockSize * D * kElem) +
                             lane * (kDims * kElem);
          unsigned long long w[kBlockSize];
#pragma unroll
          for (int t = 0; t < kBlockSize; ++t) {
            const uint8_t* s = v + t * (D * kElem);
            w[t] = 0;
            if (t >= f && t < m) {
              if constexpr (kDims * kElem == 8) w[t] = __ldg(reinterpret_cast<const unsigned long long*>(s));
              else if constexpr (kDims * kElem == 4) w[t] = __ldg(reinterpret_cast<const uint32_t*>(s));
              else w[t] = __ldg(reinterpret_cast<const unsigned short*>(s));
            }
          }
#pragma unroll
          for (int t = 0; t < kBlockSize; ++t)
#pragma unroll
            for (int e = 0; e < kDims; ++e) {
              const int kind = odd_kind<QT, kFP8>((uint32_t)(w[t] >> (e * kBits)) & ((1u << kBits) - 1u));
              if (kind == 1) last[0][e] = b * kBlockSize + t;
              if (kind == 2) last[1][e] = b * kBlockSize + t;
              if (kind == 3) last[2][e] = b * kBlockSize + t;
            }
        }
        j = b * kBlockSize + m;
      }
    };
    for (uint32_t todo = rows; todo != 0; todo &= todo - 1) {
      const int rw = __ffs(todo) - 1, tok = (r0 + rw) / g;
      const int row = x.q0 + t0 + tok, h = x.kvh * g + (r0 + rw) % g;
      int lo, hi;
      key_interval(p, row, pos0 + tok, x.ctx, x.bidir, &lo, &hi);
      scan_to(hi);
      T* o = static_cast<T*>(p.out) + ((size_t)row * p.num_heads + h) * D + lane * kDims;
#pragma unroll
      for (int e = 0; e < kDims; ++e) {
        if (fabsf((float)o[e]) < INFINITY) continue;
        const bool nan = last[0][e] >= lo, up = last[1][e] >= lo, down = last[2][e] >= lo;
        if (!nan && !up && !down) unseen[e] |= 1u << rw;
        else store_out(o + e, nan || up == down ? NAN : up ? INFINITY : -INFINITY);
      }
    }
    scan_to(min(x.end_block * kBlockSize, x.ctx));
    uint32_t again = 0;
#pragma unroll
    for (int e = 0; e < kDims; ++e)  // (no such V in the whole item: the sum itself overflowed)
      if (last[0][e] >= 0 || last[1][e] >= 0 || last[2][e] >= 0) again |= unseen[e];
    again = __reduce_or_sync(kFull, again);
    __syncwarp();
    for (int c = lane >> 2; c < __popc(again); c += 8) {
      const int rw = (int)__fns(again, 0, c + 1), tok = (r0 + rw) / g;
      const int row = x.q0 + t0 + tok, h = x.kvh * g + (r0 + rw) % g;
      int lo, hi;
      key_interval(p, row, pos0 + tok, x.ctx, x.bidir, &lo, &hi);
      exact_row<QT, kFP8, D>(p, x.seq, row, h, pos0 + tok, lo, hi, gmask);
    }
    __syncwarp();
  }
}

// Barriers, tensor memory, and the per-sequence tables; ends with the CTA synchronised.
template <bool kFP8, int kMods>
__device__ __forceinline__ void mods_setup(const AttnParams& p, ModSmem<kFP8>& sm, const CUtensorMap& tm_k,
                                           const CUtensorMap& tm_v, const CUtensorMap& tm_q) {
  constexpr int kModThreads = mod_threads(kFP8);
  const int users = by_role<kFP8, kMods>(p) ? 1 : 2;  // issuers that give back K, V, Q and tail
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], kFP8 ? kConverters : mod_producers(false));
      mbar_init(&sm.empty[s], users);
      mbar_init(&sm.staged[s], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, users);
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sm.s_ready[x][b], 1);
        mbar_init(&sm.p_ready[x][b], kTileWarps);
        mbar_init(&sm.o_done[x][b], 1);
      }
      mbar_init(&sm.o_free[x], kTileWarps);
      mbar_init(&sm.mma_done[x], 1);
    }
    for (int w = 0; w < kSoftWarps; ++w) sm.redo_n[w] = 0;
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_read[i], kSoftWarps + kIssuers + mod_extra(kFP8) - 1);
    }
    mbar_init(&sm.answer_full, 1);
    mbar_init(&sm.tail_full, 1);
    mbar_init(&sm.tail_free, users);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp >= kWarpTma && lane == 0) {
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
    tc::prefetch_tmap(&tm_q);
  }
  if (warp == kWarpMma) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  const int S = p.num_seqs, tid = threadIdx.x;
  const int chunk = (S + kModThreads - 1) / kModThreads;
  const int cap = min(p.max_blocks_per_seq * kBlockSize, p.max_context);
  const int per_item = 2 * (kRowsM / p.group);  // tokens
  int local = 0;
  for (int i = 0; i < chunk; ++i) {
    const int sq = tid * chunk + i;
    if (sq < S) {
      const int q0 = __ldg(p.query_start_loc + sq);
      int qlen = __ldg(p.query_start_loc + sq + 1) - q0;
      int ctx = __ldg(p.context_lens + sq);
      if (ctx < 0 || ctx > cap || qlen < 0 || qlen > ctx || q0 < 0 || qlen > p.num_rows - q0) {
        flag_error(p.errors, PKV_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : min(ctx, cap);
        qlen = qlen < 0 ? 0 : min(qlen, ctx);
        if (q0 < 0 || qlen > p.num_rows - q0) qlen = 0;
      }
      sm.seq_qlen[sq] = qlen;
      sm.seq_ctx[sq] = ctx;
      sm.seq_q0[sq] = q0;
      local += (qlen + per_item - 1) / per_item;
    }
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += sm.scan[w];
  int run = base + incl - local;
  for (int i = 0; i < chunk; ++i) {
    const int sq = tid * chunk + i;
    if (sq < S) {
      sm.seq_start[sq] = run;
      run += (sm.seq_qlen[sq] + per_item - 1) / per_item;
    }
  }
  if (tid == kModThreads - 1) sm.seq_start[S] = base + incl;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
}

// TMA producer pw: per item the query tiles, then per step its key tile's K boxes, the
// tail rows of V where the tile holds the context's partial last block, and its V
// boxes, into the ring.  The boxes are dealt out to the producers block by block; an
// E4M3 tile, half as large, lands in the second half of its stage.
template <bool kFP8, int kMods, int D>
__device__ __forceinline__ void mods_producer(const AttnParams& p, ModSmem<kFP8>& sm,
                                              const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                              const CUtensorMap& tm_q, int kv_rows, int total,
                                              int pw) {
  constexpr int nst = kStages, kModProd = mod_producers(kFP8);
  constexpr int kRow = D * (kFP8 ? 1 : 2);       // bytes of a cache row
  constexpr int kLoadBytes = kTileKeys * kRow;
  constexpr int kBoxRow = kRow < 128 ? kRow : 128;  // bytes of a row in a box
  uint64_t* const landed = kFP8 ? sm.staged : sm.full;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const int lane = threadIdx.x & 31, g = p.group;
  const int mine = (8 - pw + kModProd - 1) / kModProd;  // blocks per tile
  const bool my_lane = (lane & 7) % kModProd == pw;
  uint8_t* const ring = &sm.ring[0][0];
  uint32_t pos = 0, n = 0;
  int nitem = 0, ntail = 0, nquery = 0;  // items with keys, tails, items whose Q is asked for
  bool ok = true;
  ModItem x;
  // table entry of block 32 c + lane (kBeyond outside the visible blocks), read ahead
  // of its use, checked when used
  auto fetch = [&](int c) -> int {
    const int b = 32 * c + lane;
    return b >= x.lo_block && b < x.end_block
               ? __ldg(p.block_tables + (size_t)x.seq * p.max_blocks_per_seq + b)
               : kBeyond;
  };
  auto to_row = [&](int blk) -> int {
    if (blk == kBeyond) return kv_rows;
    if (blk >= 0 && blk < p.num_blocks) return (blk * p.num_kv_heads + x.kvh) * kBlockSize;
    flag_error(p.errors, PKV_DEVERR_BLOCK_ID);
    return kv_rows;
  };
  auto issue = [&](int t, int row, bool is_v) -> bool {
    const int st = pos % nst;
    // test hook: these boxes are never issued, so every wait for the tile runs out
    const bool skip = pw == 0 && blockIdx.x == 0 && p.skip_copy > 0 && pos + 1 == (uint32_t)p.skip_copy;
    bool good = true;
    if (lane == 0) {
      if (pos >= (uint32_t)nst) good = wait_for(&sm.empty[st], ((pos / nst) - 1) & 1, abort, lim);
      if (good && !skip) mbar_arrive_expect_tx(&landed[st], mine * (kLoadBytes / 8));
    }
    if (!__shfl_sync(kFull, (int)good, 0)) return false;
    if (!skip && (lane >> 3) == (t & 3) && my_lane) {
      uint8_t* dst = ring + (size_t)st * kTileBytes + (kFP8 ? kHalf : 0) +
                     (lane & 7) * (kBlockSize * kBoxRow);
      const CUtensorMap* map = is_v ? &tm_v : &tm_k;
      tc::tma_load_2d(dst, map, 0, row, &landed[st]);
      if (kRow > 128) tc::tma_load_2d(dst + kHalf, map, 64, row, &landed[st]);
    }
    __syncwarp();
    ++pos;
    return true;
  };
  // V rows of the MMA step that holds the partial last block, rows past the context
  // as zeros, with the ring's swizzle
  auto load_tail = [&]() -> bool {
    bool good = true;
    if (lane == 0 && ntail >= 1) good = wait_for(&sm.tail_free, (ntail - 1) & 1, abort, lim);
    if (!__shfl_sync(kFull, (int)good, 0)) return false;
    constexpr int kRowChunks = D / 8;  // 16-byte chunks per row
    const int key0 = (x.nk - 1) * kTileKeys + x.tail_step * kBlockSize;
#pragma unroll
    for (int i = 0; i < kBlockSize * kRowChunks / 32; ++i) {
      const int c = lane + 32 * i;
      const int r = c / kRowChunks, ch = c % kRowChunks;
      const int key = key0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (key < x.ctx && key / kBlockSize < x.end_block) {
        const int blk =
            __ldg(p.block_tables + (size_t)x.seq * p.max_blocks_per_seq + key / kBlockSize);
        if (blk >= 0 && blk < p.num_blocks)
          v = __ldg(reinterpret_cast<const uint4*>(
                        p.v_cache + (((size_t)blk * p.num_kv_heads + x.kvh) * kBlockSize +
                                     (key & (kBlockSize - 1))) * (kRowChunks * 16)) + ch);
      }
      *reinterpret_cast<uint4*>(&sm.tail[0] + (ch >> 3) * (kTailBytes / 2) + r * 128 +
                                (((ch & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.tail_full);
    ++ntail;
    return true;
  };
  uint32_t asked = 0;
  for (; ok; ++n) {
    bool good = true;
    if (pw == 0) {
      int k = n == 0 ? (int)blockIdx.x : -1;
      if (lane == 0 && n > 0 && asked == n) k = next_item(sm, n - 1, abort, lim);
      k = __shfl_sync(kFull, k, 0);
      if (k == -2) {
        ok = false;
        break;
      }
      if (k >= 0) {
        // (not for more items than the lists of redo_rows can take)
        const int listed = lane < kSoftWarps ? *static_cast<volatile int*>(&sm.redo_n[lane]) : 0;
        if (__all_sync(kFull, listed + kUnderWay <= kRedo)) {
          if (lane == 0) ask_next(sm);
          ++asked;
        }
        make_item<kMods, kFP8>(p, sm, k, total, x);
      }
      if (lane == 0) {
        const int slot = n % kAhead;
        if (n >= kAhead) good = wait_for(&sm.item_read[slot], ((n / kAhead) - 1) & 1, abort, lim);
        if (good) {
          if (k >= 0) sm.item[slot] = x;
          else sm.item[slot].k = -1;
          mbar_arrive(&sm.item_full[slot]);
        }
      }
      ok = __shfl_sync(kFull, (int)good, 0) != 0;
      if (!ok || k < 0) break;
    } else {
      ok = take_item<false>(sm, n, x, abort, lim);
      if (!ok || x.k < 0) break;
    }
    if (x.nk == 0) continue;
    if (pw == 0 && lane == 0) {
      if (nitem >= 1) good = wait_for(&sm.q_empty, (nitem - 1) & 1, abort, lim);
      if (good) {
        const int nq = x.nt[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(&sm.q_full, nq * (kRowsM / g * g * D * 2));
        ++nquery;
        for (int qt = 0; qt < nq; ++qt) {
          uint8_t* dq = &sm.q[qt][0];
          const int tok = x.q0 + x.t0[qt];
          tc::tma_load_3d(dq, &tm_q, 0, x.kvh * g, tok, &sm.q_full);
          if (D > 64) tc::tma_load_3d(dq + kHalf, &tm_q, 64, x.kvh * g, tok, &sm.q_full);
        }
      }
    }
    ok = __shfl_sync(kFull, (int)good, 0) != 0;
    // block rows of the 32-block chunk (four key tiles) in use; the next one read ahead
    constexpr int kStep = (kMods & kModBias) ? -1 : 1;
    int cur_c = tile_of<kMods>(x, 0) >> 2, cur_row = to_row(fetch(cur_c));
    int pre_raw = fetch(cur_c + kStep);
    for (int i = 0; ok && i < x.nk - x.kt0; ++i) {
      const int t = tile_of<kMods>(x, i);
      if ((t >> 2) != cur_c) {
        cur_c = t >> 2;
        cur_row = to_row(pre_raw);
        pre_raw = fetch(cur_c + kStep);
      }
      ok = issue(t, cur_row, false);
      if (ok && pw == 0 && t == x.nk - 1 && x.tail_step >= 0) ok = load_tail();
      if (ok) ok = issue(t, cur_row, true);
    }
    ++nitem;
  }
  if (!ok && lane == 0) {
    flag_error(p.errors, PKV_DEVERR_TIMEOUT);
    // an answer, Q and tiles still on their way land before the CTA goes away
    if (pw == 0 && asked > 0) mbar_wait(&sm.answer_full, (asked - 1) & 1, 10000000ull);
    if (nquery > 0) mbar_wait(&sm.q_full, (nquery - 1) & 1, 10000000ull);
    for (uint32_t y = pos > (uint32_t)nst ? pos - nst : 0; y < pos; ++y)
      mbar_wait(&landed[y % nst], (y / nst) & 1, 10000000ull);
  }
}

// 16 E4M3 codes as 16-bit elements (each code is one of either type), a pair by one
// conversion to fp16, and for bf16 by way of fp32.  (Moving the fields and
// multiplying the exponents' offset in, with a test for NaN codes, takes more
// instructions, and they are what a converter's time goes by: 167 against 151 us.)
template <class QT>
__device__ __forceinline__ void widen16(const uint32_t* u, uint4* a, uint4* b) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((u[i >> 1] >> (16 * (i & 1))) & 0xffffu), __NV_E4M3);
    if constexpr (std::is_same<QT, BF16>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
      o[i] = pack2<BF16>(f.x, f.y);
    } else {
      o[i] = *reinterpret_cast<const uint32_t*>(&hr);
    }
  }
  *a = make_uint4(o[0], o[1], o[2], o[3]);
  *b = make_uint4(o[4], o[5], o[6], o[7]);
}

// Converter cw of five on an E4M3 cache: each tile that has landed, in ring order, from
// [128 rows][D B] in the second half of its stage to [D / 64 halves][128 rows][128 B], the
// V rows past the context as zeros; all with the 128-byte swizzle, but for the 64-byte
// rows of D = 64, which land as they are.  Row r of the codes lies where row r of the
// second half of the elements will (or beside all of them), so a warp that reads whole
// rows before it writes them needs no order with the others.
template <class QT, int kMods, int D>
__device__ __forceinline__ void mods_converter(const AttnParams& p, ModSmem<true>& sm, int total,
                                               int cw) {
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  constexpr int kLanes = D / 16;         // 16-code chunks, and lanes, per row
  constexpr int kRows = 32 / kLanes;     // rows a turn
  const int lane = threadIdx.x & 31, c = lane % kLanes;
  uint32_t pos = 0;
  bool ok = true;
  ModItem x;
  auto convert = [&](int rows) -> bool {
    const int st = pos % kStages;
    bool good = true;
    if (lane == 0) good = wait_for(&sm.staged[st], (pos / kStages) & 1, abort, lim);
    if (!__shfl_sync(kFull, (int)good, 0)) return false;
    ++pos;
    uint8_t* tile = &sm.ring[st][0];
    // the next turn's codes are read ahead (rolled: beside the softmax's code the
    // instruction cache has little room, see above)
    auto codes = [&](int u) {
      const int r = kRows * u + lane / kLanes;
      return *reinterpret_cast<const uint4*>(tile + kHalf + r * D +
                                             ((D == 128 ? c ^ (r & 7) : c) << 4));
    };
    uint4 w = codes(cw);
#pragma unroll 1
    for (int u = cw; u < kTileKeys / kRows; u += kConverters) {
      const int r = kRows * u + lane / kLanes;
      uint4 nw = w;
      if (u + kConverters < kTileKeys / kRows) nw = codes(u + kConverters);
      if (rows < kTileKeys && r >= rows) w = make_uint4(0, 0, 0, 0);
      // chunks 2 (c % 4) and 2 (c % 4) + 1 of half c / 4; the halves' lanes store them
      // in opposite order, so that eight lanes hit eight different bank groups (D = 64:
      // the swizzle of two rows does that)
      const bool up = c >> 2;
      const uint32_t v[4] = {up ? w.z : w.x, up ? w.w : w.y, up ? w.x : w.z, up ? w.y : w.w};
      uint4 a, b;
      widen16<QT>(v, &a, &b);
      __syncwarp();  // the rows have been read
      uint8_t* d = tile + (c >> 2) * kHalf + r * 128;
      const int k0 = (2 * (c & 3) + (up ? 1 : 0)) ^ (r & 7);
      *reinterpret_cast<uint4*>(d + (k0 << 4)) = a;
      *reinterpret_cast<uint4*>(d + ((k0 ^ 1) << 4)) = b;
      w = nw;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.full[st]);
    return true;
  };
  for (uint32_t n = 0; ok; ++n) {
    ok = take_item<false>(sm, n, x, abort, lim);
    if (!ok || x.k < 0) break;
    for (int i = 0; ok && i < x.nk - x.kt0; ++i)
      ok = convert(kTileKeys) && convert(x.ctx - tile_of<kMods>(x, i) * kTileKeys);
  }
  if (!ok && lane == 0) flag_error(p.errors, PKV_DEVERR_TIMEOUT);
}

// MMA issuers, one thread each.  A query tile has two score buffers, so that its softmax
// has the next step's scores at hand; scores of step v go where P of step v - 2 was,
// behind its product.  (One issuer for all was the bottleneck: 1500 cycles for a query
// tile's step, most of them waits, commits and their latencies, not MMAs.)
//
// By role: the scores of both query tiles.
template <class QT, bool kFP8, int kMods, int D>
__device__ __forceinline__ bool issue_all_scores(const AttnParams& p, ModSmem<kFP8>& sm, uint32_t tmem) {
  constexpr uint32_t kAB = std::is_same<QT, BF16>::value ? 1u : 0u;
  constexpr uint32_t kIdesc = tc::idesc_f16(kAB, 0, 0, 128, kStepKeys);
  constexpr uint64_t kStage = kTileBytes >> 4;          // in descriptor units
  constexpr uint64_t kInTile = (kStepKeys * 128) >> 4;  // a tile's second half of keys
  constexpr int kBack = (kMods & kModBias) != 0;
  static_assert((kStages & (kStages - 1)) == 0, "ring positions wrap");
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const uint64_t dq[2] = {tc::smem_desc(smem_u32(&sm.q[0][0]), 16, 1024, tc::kLayoutSw128),
                          tc::smem_desc(smem_u32(&sm.q[1][0]), 16, 1024, tc::kLayoutSw128)};
  const uint64_t dk = tc::smem_desc(smem_u32(&sm.ring[0][0]), 16, 1024, tc::kLayoutSw128);
  uint32_t at = 0, ns[2] = {0, 0}, nitem = 0;  // ring position of the K tile, steps issued, items
  ModItem x;
  for (uint32_t n = 0;; ++n) {
    if (!take_item<true>(sm, n, x, abort, lim)) return false;
    if (x.k < 0) return true;
    if (x.nk == 0) continue;
    const int steps = x.nh - x.h0, last[2] = {x.last[0], x.last[1]};
    int half = half_of<kMods>(x, 0);
    bool fresh = true;  // the step's tile has not been waited for
    if (!wait_for(&sm.q_full, nitem & 1, abort, lim)) return false;
#pragma unroll 1
    for (int v = 0; v < steps; ++v) {
      if (fresh && !wait_for(&sm.full[at % kStages], (at / kStages) & 1, abort, lim)) return false;
#pragma unroll
      for (int qt = 0; qt < 2; ++qt) {
        if (v > last[qt]) continue;
        const uint32_t b = ns[qt] & 1;
        if (ns[qt] >= 2 && !wait_for(&sm.o_done[qt][b], ((ns[qt] >> 1) - 1) & 1, abort, lim))
          return false;
        ++ns[qt];
        tc::fence_after_sync();
        issue_mods_scores<D>(tmem + qt * 128 + b * kStepKeys, dq[qt],
                             dk + (at % kStages) * kStage + (half & 1) * kInTile, kIdesc);
        tc::mma_commit(&sm.s_ready[qt][b]);
      }
      fresh = v + 1 == steps || (half & 1) != kBack;  // the tile's last step
      if (fresh) {
        tc::mma_commit(&sm.empty[at % kStages]);
        at += 2;
      }
      half += kBack ? -1 : 1;
    }
    tc::mma_commit(&sm.q_empty);
    ++nitem;
  }
}

// By role: the products of both query tiles.
template <class QT, bool kFP8, int kMods, int D>
__device__ __forceinline__ bool issue_all_products(const AttnParams& p, ModSmem<kFP8>& sm, uint32_t tmem) {
  constexpr uint32_t kAB = std::is_same<QT, BF16>::value ? 1u : 0u;
  constexpr uint32_t kIdesc = tc::idesc_f16(kAB, 0, 1, 128, D);
  constexpr uint64_t kStage = kTileBytes >> 4;
  constexpr uint64_t kInTile = (kStepKeys * 128) >> 4;
  constexpr int kBack = (kMods & kModBias) != 0;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const uint64_t dv = tc::smem_desc(smem_u32(&sm.ring[0][0]), kHalf, 1024, tc::kLayoutSw128);
  const uint64_t dtail =
      tc::smem_desc(smem_u32(&sm.tail[0]), kTailBytes / 2, 1024, tc::kLayoutSw128);
  uint32_t at = 1, np[2] = {0, 0};        // ring position of the V tile, P consumed
  uint32_t nit[2] = {0, 0}, ntail = 0;    // items with steps of a query tile, tails
  ModItem x;
  for (uint32_t n = 0;; ++n) {
    if (!take_item<true>(sm, n, x, abort, lim)) return false;
    if (x.k < 0) return true;
    if (x.nk == 0) continue;
    const int steps = x.nh - x.h0, last[2] = {x.last[0], x.last[1]};
    const int tail_half = x.tail_step >= 0 ? x.nh - 1 : -1;
    int half = half_of<kMods>(x, 0);
    bool fresh = true;
#pragma unroll 1
    for (int v = 0; v < steps; ++v) {
      if (fresh && !wait_for(&sm.full[at % kStages], (at / kStages) & 1, abort, lim)) return false;
      if (half == tail_half && !wait_for(&sm.tail_full, ntail & 1, abort, lim)) return false;
#pragma unroll
      for (int qt = 0; qt < 2; ++qt) {
        if (v > last[qt]) continue;
        const uint32_t b = np[qt] & 1;
        if (!wait_for(&sm.p_ready[qt][b], (np[qt] >> 1) & 1, abort, lim)) return false;
        if (v == 0 && nit[qt] > 0 && !wait_for(&sm.o_free[qt], (nit[qt] - 1) & 1, abort, lim))
          return false;  // the previous item's O has been read out
        ++np[qt];
        tc::fence_after_sync();
        issue_mods_pv(tmem + kColO + qt * 128, tmem + qt * 128 + b * kStepKeys,
                      dv + (at % kStages) * kStage + (half & 1) * kInTile, dtail,
                      half == tail_half ? x.tail_step & 3 : -1, v != 0, kIdesc);
        tc::mma_commit(&sm.o_done[qt][b]);
      }
      fresh = v + 1 == steps || (half & 1) != kBack;
      if (fresh) {
        tc::mma_commit(&sm.empty[at % kStages]);
        at += 2;
      }
      half += kBack ? -1 : 1;
    }
    if (x.tail_step >= 0) {
      tc::mma_commit(&sm.tail_free);
      ++ntail;
    }
    nit[0] += last[0] >= 0;
    nit[1] += last[1] >= 0;
  }
}

// By query tile: scores and products of tile qt.  (qt is the same in every lane by a
// shuffle: MMA operands that the compiler takes for different ones come out wrong.)
template <class QT, bool kFP8, int kMods, int D>
__device__ __forceinline__ bool issue_tile(const AttnParams& p, ModSmem<kFP8>& sm, uint32_t tmem, int qt) {
  constexpr uint32_t kAB = std::is_same<QT, BF16>::value ? 1u : 0u;
  constexpr uint32_t kIdescS = tc::idesc_f16(kAB, 0, 0, 128, kStepKeys);
  constexpr uint32_t kIdescO = tc::idesc_f16(kAB, 0, 1, 128, D);
  constexpr uint64_t kStage = kTileBytes >> 4;
  constexpr uint64_t kInTile = (kStepKeys * 128) >> 4;
  constexpr int kBack = (kMods & kModBias) != 0;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const uint64_t dq = tc::smem_desc(smem_u32(&sm.q[qt][0]), 16, 1024, tc::kLayoutSw128);
  const uint64_t dk = tc::smem_desc(smem_u32(&sm.ring[0][0]), 16, 1024, tc::kLayoutSw128);
  const uint64_t dv = tc::smem_desc(smem_u32(&sm.ring[0][0]), kHalf, 1024, tc::kLayoutSw128);
  const uint64_t dtail =
      tc::smem_desc(smem_u32(&sm.tail[0]), kTailBytes / 2, 1024, tc::kLayoutSw128);
  const uint32_t s_col = tmem + qt * 128, o_col = tmem + kColO + qt * 128;
  uint32_t at_k = 0, at_v = 1;  // ring positions of the scores' K and the products' V tile
  uint32_t ns = 0, np = 0;      // score steps issued, P consumed
  uint32_t nit = 0, nitem = 0, ntail = 0;  // items with steps of this tile, items, tails
  bool ok = true;
  ModItem x;
  for (uint32_t n = 0; ok; ++n) {
    ok = take_item<true>(sm, n, x, abort, lim);
    if (!ok || x.k < 0) break;
    if (x.nk == 0) continue;
    const int steps = x.nh - x.h0, last = qt ? x.last[1] : x.last[0];
    const int tail_half = x.tail_step >= 0 ? x.nh - 1 : -1;
    int hs = half_of<kMods>(x, 0), hp = hs;  // halves of the scores' and the products' step
    bool new_k = true, new_v = true;         // their tile has not been waited for
    // scores of step v
    auto scores = [&](int v) -> bool {
      if (new_k) {
        if (!wait_for(&sm.full[at_k % kStages], (at_k / kStages) & 1, abort, lim)) return false;
        tc::fence_after_sync();
      }
      if (v <= last) {
        const uint32_t b = ns++ & 1;
        issue_mods_scores<D>(s_col + b * kStepKeys, dq,
                             dk + (at_k % kStages) * kStage + (hs & 1) * kInTile, kIdescS);
        tc::mma_commit(&sm.s_ready[qt][b]);
      }
      new_k = v + 1 == steps || (hs & 1) != kBack;
      if (new_k) {  // the tile's last step
        tc::mma_commit(&sm.empty[at_k % kStages]);
        at_k += 2;
      }
      hs += kBack ? -1 : 1;
      if (v + 1 == steps) tc::mma_commit(&sm.q_empty);
      return true;
    };
    ok = wait_for(&sm.q_full, nitem & 1, abort, lim);
    if (ok) tc::fence_after_sync();
#pragma unroll 1
    for (int v = -2; ok && v < steps; ++v) {
      if (v >= 0) {
        if (new_v) {
          ok = wait_for(&sm.full[at_v % kStages], (at_v / kStages) & 1, abort, lim);
          if (!ok) break;
        }
        if (hp == tail_half) {
          ok = wait_for(&sm.tail_full, ntail & 1, abort, lim);
          if (!ok) break;
        }
        if (v <= last) {
          const uint32_t b = np & 1;
          ok = wait_for(&sm.p_ready[qt][b], (np >> 1) & 1, abort, lim);
          if (ok && v == 0 && nit > 0)  // the previous item's O has been read out
            ok = wait_for(&sm.o_free[qt], (nit - 1) & 1, abort, lim);
          if (!ok) break;
          ++np;
          tc::fence_after_sync();
          issue_mods_pv(o_col, s_col + b * kStepKeys,
                        dv + (at_v % kStages) * kStage + (hp & 1) * kInTile, dtail,
                        hp == tail_half ? x.tail_step & 3 : -1, v != 0, kIdescO);
          tc::mma_commit(&sm.o_done[qt][b]);
        }
        new_v = v + 1 == steps || (hp & 1) != kBack;
        if (new_v) {
          tc::mma_commit(&sm.empty[at_v % kStages]);
          at_v += 2;
        }
        hp += kBack ? -1 : 1;
      }
      if (v + 2 < steps) ok = scores(v + 2);
    }
    if (ok && x.tail_step >= 0) {
      tc::mma_commit(&sm.tail_free);
      ++ntail;
    }
    if (last >= 0) ++nit;
    ++nitem;
  }
  return ok;
}

template <class QT, bool kFP8, int kMods, int D>
__device__ __forceinline__ void mods_issuer(const AttnParams& p, ModSmem<kFP8>& sm, uint32_t tmem, int i) {
  i = __shfl_sync(kFull, i, 0);
  if (tc::elect_one()) {
    bool ok;
    if (by_role<kFP8, kMods>(p))
      ok = i == 0 ? issue_all_scores<QT, kFP8, kMods, D>(p, sm, tmem)
                  : issue_all_products<QT, kFP8, kMods, D>(p, sm, tmem);
    else
      ok = issue_tile<QT, kFP8, kMods, D>(p, sm, tmem, i);
    if (!ok) flag_error(p.errors, PKV_DEVERR_TIMEOUT);
    tc::mma_commit(&sm.mma_done[i]);
    mbar_wait(&sm.mma_done[i], 0, 100000000ull);
  }
  __syncwarp();
}

// Softmax and epilogue: thread = row of query tile qt.
template <class QT, bool kFP8, int kMods, int D>
__device__ __forceinline__ void mods_softmax(const AttnParams& p, ModSmem<kFP8>& sm, uint32_t tmem, int total) {
  using OutT = typename QT::T;
  volatile int* abort = &sm.abort;
  const unsigned long long lim = wait_limit(p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qt = warp / kTileWarps, g = p.group;
  const int r = threadIdx.x & 127;  // row = TMEM lane
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_col = tmem + lane_off + qt * 128;
  const uint32_t o_col = tmem + lane_off + kColO + qt * 128;
  // scores are scaled inside the exponent; a negative scale is folded in by negating
  // them, a zero one taken as 1e-30
  const bool neg = p.q_scale < 0.0f;
  const float qa = fmaxf(fabsf(p.q_scale), 1e-30f);
  const int tok = r / g, head_in = r - tok * g;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {  // the warp's lanes agree
    return __all_sync(kFull, wait_for(bar, parity, abort, lim)) != 0;
  };
  uint32_t n = 0;
  uint32_t ns = 0;  // steps of this query tile
  bool ok = true;
  ModItem x;
  for (;; ++n) {
    ok = take_item<false>(sm, n, x, abort, lim);
    if (!ok || x.k < 0) break;
    const int nt = qt ? x.nt[1] : x.nt[0], t0 = qt ? x.t0[1] : x.t0[0];
    const int last = qt ? x.last[1] : x.last[0];
    const int pos = (qt ? x.pos0[1] : x.pos0[0]) + tok;
    // rows past the tile's tokens compute on whatever Q holds there; never stored
    const bool valid = r < nt * g;
    const int row = x.q0 + t0 + tok, h = x.kvh * g + head_in;
    const size_t head = (size_t)row * p.num_heads + h;
    OutT* orow = static_cast<OutT*>(p.out) + head * D;
    int lo = 0, hi = INT_MAX;
    if (valid) {
      key_interval(p, row, pos, x.ctx, x.bidir, &lo, &hi);
      // first keys that decrease from row to row: blocks before lo_block are not here
      if (lo < hi && (last < 0 || lo < x.lo_block * kBlockSize))
        flag_error(p.errors, PKV_DEVERR_CONTEXT);
    }
    const bool empty = lo >= hi;  // zeros, whatever O and l hold
    if (last < 0) {               // no row of the tile sees a key
      if (valid) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(orow)[i] = make_uint4(0, 0, 0, 0);
      }
      continue;
    }
    const float slope = (kMods & kModBias) && valid ? __ldg(p.alibi + h) * kLog2e : 0.0f;
    float m_run = -INFINITY;
    float2 l2[4];  // partial row sums (independent chains, packed pairs)
#pragma unroll
    for (int i = 0; i < 4; ++i) l2[i] = make_float2(0.0f, 0.0f);
    for (int v = 0; v <= last; ++v, ++ns) {
      const int k0 = half_of<kMods>(x, v) * kStepKeys, b = ns & 1;
      const uint32_t s_at = s_col + b * kStepKeys;
      ok = wait(&sm.s_ready[qt][b], (ns >> 1) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      if (__all_sync(kFull, hi <= k0 || lo >= k0 + kStepKeys || empty)) {
        // no row of the warp sees a key of the step
        float z[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) z[c] = 0.0f;
#pragma unroll
        for (int c = 0; c < kStepKeys / kChunk; ++c) tc::tmem_st16(s_at + 16 * c, z);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[qt][b]);
        continue;
      }
      float sv[kStepKeys];
#pragma unroll
      for (int c = 0; c < kStepKeys; c += 32) tc::tmem_ld32(s_at + c, sv + c);
      tc::tmem_wait_ld();
      if (neg) {
#pragma unroll
        for (int c = 0; c < kStepKeys; ++c) sv[c] = -sv[c];
      }
      const float f = modify_scores<kMods>(p, sv, qa, slope, s_at, pos, k0, lo, hi, valid);
      if (!__all_sync(kFull, lo <= k0 && hi >= k0 + kStepKeys)) {
        // an interval of some row of the warp ends in this tile: hidden keys become -inf
#pragma unroll
        for (int c = 0; c < kStepKeys; ++c)
          sv[c] = k0 + c >= lo && k0 + c < hi ? sv[c] : -INFINITY;
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) mx[c] = -INFINITY;
#pragma unroll
      for (int c = 0; c < kStepKeys; c += 2)
        mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], sv[c], sv[c + 1]);
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
      // move the running max (and rescale O) only on a large increase
      const bool fresh = m_run == -INFINITY;  // no key seen so far
      const bool need = mt > m_run + kRescaleAt;
      float alpha = 1.0f;
      if (need) {
        alpha = fresh ? 0.0f : fast_exp2(m_run - mt);
        m_run = mt;
#pragma unroll
        for (int c = 0; c < 4; ++c) l2[c] = __fmul2_rn(l2[c], make_float2(alpha, alpha));
      }
      const float m = m_run == -INFINITY ? 0.0f : m_run;  // 2^(-inf - 0) = 0
      // weights, over the scores read (hidden keys are -inf: weight 0)
#pragma unroll
      for (int c = 0; c < kStepKeys / kChunk; ++c) {
        float pk[16];
        const float2 f2 = make_float2(f, f), m2 = make_float2(-m, -m);
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) {
          const float2 y = __ffma2_rn(make_float2(sv[kChunk * c + e], sv[kChunk * c + e + 1]), f2, m2);
          const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          l2[(e >> 1) & 3] = __fadd2_rn(l2[(e >> 1) & 3], w);
          pk[e >> 1] = __uint_as_float(pack2<QT>(w.x, w.y));
        }
        tc::tmem_st16(s_at + 16 * c, pk);
      }
      // the product of this step adds onto O: rescale it first, once the one before is done
      if (v > 0 && __any_sync(kFull, need)) {
        ok = wait(&sm.o_done[qt][(ns - 1) & 1], ((ns - 1) >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float ov[32];
          tc::tmem_ld32(o_col + c, ov);
          tc::tmem_wait_ld();
          // (a row that had seen no key: zeros, although 0 * inf may be there)
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = fresh && need ? 0.0f : ov[e] * alpha;
          tc::tmem_st32(o_col + c, ov);
        }
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_ready[qt][b]);
    }
    if (!ok) break;
    // ---- epilogue: O / l ------------------------------------------------------------------
    const float l = ((l2[0].x + l2[0].y) + (l2[1].x + l2[1].y)) +
              ((l2[2].x + l2[2].y) + (l2[3].x + l2[3].y));
    ok = wait(&sm.o_done[qt][(ns - 1) & 1], ((ns - 1) >> 1) & 1);
    if (!ok) break;
    tc::fence_after_sync();
    const float inv = valid && !empty ? p.v_scale / l : 0.0f;
    // four lanes exchange their rows' 16-byte pieces, so that they store 64 contiguous
    // bytes of one row at a time (a piece of 32 rows in each store instead cost 5300 cycles
    // an item); the four rows' places in the output, -1 where there is none
    int place[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      place[i] = __shfl_sync(kFull, valid ? row * p.num_heads + h : -1, (lane & 28) + i);
    const bool up2 = lane & 2, up1 = lane & 1;
    float2 z = make_float2(0.0f, 0.0f);  // NaN behind an output that is not finite
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float ov[32];
      tc::tmem_ld32(o_col + c, ov);
      tc::tmem_wait_ld();
      uint32_t w1[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 o2 = __fmul2_rn(make_float2(ov[e], ov[e + 1]), make_float2(inv, inv));
        z = __ffma2_rn(o2, make_float2(0.0f, 0.0f), z);
        w1[e >> 1] = empty ? 0u : pack2<QT>(o2.x, o2.y);
      }
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = make_uint4(w1[4 * i], w1[4 * i + 1], w1[4 * i + 2], w1[4 * i + 3]);
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
          *reinterpret_cast<uint4*>(static_cast<OutT*>(p.out) + (size_t)place[i] * D + c +
                                    8 * (lane & 3)) = w[i];
    }
    // (where the sum of the weights is no number, a score that the row sees is none)
    const bool odd = valid && !empty && l > 0.0f && l < INFINITY && (z.x != z.x || z.y != z.y);
    const uint32_t odd_rows = __ballot_sync(kFull, odd);
    if (odd_rows != 0 && lane == 0) {
      const int at = sm.redo_n[warp];  // (below kRedo: the producer sees to it)
      if (at < kRedo) {
        sm.redo_item[warp][at] = x.k;
        sm.redo_rows[warp][at] = odd_rows;
        *static_cast<volatile int*>(&sm.redo_n[warp]) = at + 1;
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.o_free[qt]);
  }
  if (!ok && lane == 0) flag_error(p.errors, PKV_DEVERR_TIMEOUT);
  __syncwarp();
  if (ok && sm.redo_n[warp] > 0) redo_rows<QT, kFP8, kMods, D>(p, sm, total, warp);
}

template <class QT, bool kFP8, int kMods, int D>
__global__ void __launch_bounds__(mod_threads(kFP8), 1)
    prefill_mods_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_q, int kv_rows) {
  extern __shared__ uint8_t smem_raw[];
  using SM = ModSmem<kFP8>;
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  mods_setup<kFP8, kMods>(p, sm, tm_k, tm_v, tm_q);
  const uint32_t tmem = sm.tmem_base;
  const int total = sm.seq_start[p.num_seqs] * p.num_kv_heads;
  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(other_regs(kFP8)));
    if (warp < kWarpTma)
      mods_issuer<QT, kFP8, kMods, D>(p, sm, tmem, warp - kWarpMma);
    else if (warp < kWarpTma + mod_producers(kFP8))
      mods_producer<kFP8, kMods, D>(p, sm, tm_k, tm_v, tm_q, kv_rows, total, warp - kWarpTma);
    else if constexpr (kFP8)
      mods_converter<QT, kMods, D>(p, sm, total, warp - kWarpTma - mod_producers(true));
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(soft_regs(kFP8)));
    mods_softmax<QT, kFP8, kMods, D>(p, sm, tmem, total);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <class QT, bool kFP8, int kMods, int D>
int launch_mods(const AttnParams& p, int total_q, cudaStream_t stream) {
  const bool bf16 = std::is_same<QT, BF16>::value;
  const uint64_t kv_rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
  const uint32_t g = (uint32_t)p.group, tokens = kRowsM / g, heads = (uint32_t)p.num_heads;
  CUtensorMap tk, tv, tq;
  const int type = kFP8 ? PKV_FP8_E4M3 : (bf16 ? PKV_BF16 : PKV_F16);
  if (!make_map_rows(&tk, p.k_cache, kv_rows, D, type, kBlockSize) ||
      !make_map_rows(&tv, p.v_cache, kv_rows, D, type, kBlockSize) ||
      !make_map_heads(&tq, p.q, (uint64_t)total_q, heads, D, bf16, g, tokens))
    return PKV_ERR_CUDA;
  using SM = ModSmem<kFP8>;
  const size_t smem = sizeof(SM) + 1024;
  static_assert(sizeof(SM) + 1024 <= 232448, "shared memory budget of one CTA");
  static_assert(offsetof(SM, ring) % 1024 == 0 && offsetof(SM, q) % 1024 == 0 &&
                    offsetof(SM, tail) % 1024 == 0,
                "swizzled buffers must start on 1024-byte boundaries");
  auto kern = prefill_mods_kernel<QT, kFP8, kMods, D>;
  // the kernel's register shares add up to what its launch holds; with fewer its
  // warpgroups would wait for registers without end
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
  if (fa.numRegs != launch_regs(kFP8)) return PKV_ERR_CUDA;
  static std::atomic<unsigned long long> configured{0};
  if (!smem_once(kern, smem, configured)) return PKV_ERR_CUDA;
  // launches of at most kMaxSeqs sequences each; their query rows stay absolute
  for (int s0 = 0; s0 < p.num_seqs; s0 += kMaxSeqs) {
    AttnParams c = p;
    c.num_seqs = p.num_seqs - s0 < kMaxSeqs ? p.num_seqs - s0 : kMaxSeqs;
    c.block_tables = p.block_tables + (size_t)s0 * p.max_blocks_per_seq;
    c.context_lens = p.context_lens + s0;
    c.query_start_loc = p.query_start_loc + s0;
    if (p.bidir_lens) c.bidir_lens = p.bidir_lens + s0;
    // a CTA per item: an upper bound of them (every sequence's pairs of query tiles, the
    // last of each perhaps short, times the KV heads); those past the last do nothing
    const long long pairs = total_q / (2 * (long long)tokens) + c.num_seqs;
    const long long items = pairs * p.num_kv_heads;
    if (items > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    kern<<<(unsigned)items, mod_threads(kFP8), smem, stream>>>(c, tk, tv, tq, (int)kv_rows);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

template <int kMods, int D>
int launch_mods_dim(const AttnParams& p, int q_dtype, int kv_dtype, int total_q,
                    cudaStream_t stream) {
  const bool fp8 = kv_dtype == PKV_FP8_E4M3;
  if (q_dtype == PKV_BF16)
    return fp8 ? launch_mods<BF16, true, kMods, D>(p, total_q, stream)
               : launch_mods<BF16, false, kMods, D>(p, total_q, stream);
  return fp8 ? launch_mods<F16, true, kMods, D>(p, total_q, stream)
             : launch_mods<F16, false, kMods, D>(p, total_q, stream);
}

}  // namespace
}  // namespace pre_mods
}  // namespace pkv

#endif  // PKV_PREFILL_MODS_CUH

// Rotary positions of Q and K fused with the cache write: Q is rotated into
// q_out, K is rotated into its cache slot, V is written to its slot.
//
// Pair i (i < rotary_dim / 2) of a row at position t turns by t * inv_freq[i]:
//   (a, b) -> f (a cos - b sin, b cos + a sin)
// with (a, b) = (x[i], x[i + rotary_dim / 2]) in the half layout and
// (x[2i], x[2i + 1]) in the interleaved one, f the attention factor of a scaled
// context; elements from rotary_dim on are copied.
//
// Angles.  t * inv_freq loses whole turns in fp32 long before 131,072 tokens,
// and fp64 runs at 1/60 of fp32 here.  The angle is taken modulo one turn in
// integers instead: the host gives phase[i] = frac(inv_freq[i] / 2 pi) * 2^64,
// and t * phase[i] mod 2^64 is the fraction of a turn, exact but for phase's own
// rounding, 2^-63 turns, so off by less than 2^-32 turns at any position.  Its top 32
// bits as a signed fraction go through sincospif.  No table is read, so there is none to
// size for the longest context.
//
// A warp takes a token, or a share of its rows.  A row is D / 8 lanes, one 16-byte
// chunk each, so two (D = 128) or four rows move at once, four times over before
// the first is needed; a lane's chunk is the same in every row, so its cosines and
// sines are computed once and stay in registers.  In the half layout the other
// element of a pair is in another lane's chunk and comes by shuffle (or, where the
// halves are not whole chunks, from global memory again).  Rotation in fp32, one
// rounding on the way out (to 16 bits, or straight to E4M3 after the division by the
// scale).
//
// Bound by HBM for many tokens: 8192 tokens of 64 query and 8 KV heads of 128 (fp16, half
// of each head turning), 336 MB, in 52.6 us, 6.4 TB/s (CTAs of 256 threads 55.5; an
// earlier form with a CTA per token and the angles in shared memory 71); by the launch
// for few: 64 tokens 3.6 us, one call behind the other in a graph, where an empty launch takes
// 0.6.  2080 tokens into an E4M3 cache, 47 MB, take 11.8 us that way and 14.3 alone, against
// 6.9 for their bytes: the launch makes one warp of each token there, three or four per
// scheduler, each with its angles and its codes to compute (issue slots 53 % busy), where
// the registers would hold five; more warps of fewer rows have not been measured.

#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;  // head_dim 128
constexpr int kDeep = 4;       // row groups loaded ahead

struct RotParams {
  uint8_t* q_out;
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slots;
  const int32_t* positions;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  int num_tokens, num_heads, num_kv_heads, pairs;
  int parts, rows_per_part;  // warps per token, and the rows (of Q, K, V in order) of each
  long long num_slots;
  float factor, k_scale, v_scale;
  uint32_t* errors;
  unsigned long long phase[kMaxPairs];
};

__device__ __forceinline__ uint32_t e4m3x4(const float* f, float scale) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(f[i], scale), __NV_SATFINITE, __NV_E4M3)
         << (8 * i);
  return w;
}

// kHalf: half layout, else interleaved.  kWhole: the half layout's halves are whole
// 16-byte chunks.
template <class QT, bool FP8, int D, bool kHalf, bool kWhole>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotParams p) {
  using T = typename QT::T;
  constexpr int kLanes = D / 8;         // lanes per row
  constexpr int kRows = 32 / kLanes;    // rows at once
  constexpr int kElem = FP8 ? 1 : 2;    // bytes per cache element
  const int lane = threadIdx.x & 31, sub = lane / kLanes, c = lane % kLanes;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tok = (int)(unit / p.parts), part = (int)(unit - (long long)tok * p.parts);
  if (tok >= p.num_tokens) return;
  const int pos = __ldg(p.positions + tok);
  if (pos < 0) return;  // padding: nothing is written
  const int64_t slot = __ldg(p.slots + tok);
  const bool cached = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && part == 0 && lane == 0) flag_error(p.errors, PKV_DEVERR_SLOT);
  const int H = p.num_heads, hk = p.num_kv_heads;
  const int r_end = min((part + 1) * p.rows_per_part, cached ? H + 2 * hk : H);

  // this lane's eight elements in every row; those below rot turn
  const int e0 = 8 * c, half = p.pairs, rot = 2 * half;
  const uint8_t* qs = p.q + 2 * (tok * p.q_stride + e0);
  const uint8_t* ks = p.k + 2 * (tok * p.k_stride + e0);
  const uint8_t* vs = p.v + 2 * (tok * p.v_stride + e0);
  uint8_t* qd = p.q_out + 2 * ((long long)tok * H * D + e0);
  const long long at = cached ? ((slot / kBlockSize) * hk * kBlockSize + slot % kBlockSize) * D + e0 : 0;
  uint8_t* kd = p.k_cache + at * kElem;
  uint8_t* vd = p.v_cache + at * kElem;
  auto load = [&](int r) -> uint4 {
    const uint8_t* s = r < H ? qs + (long long)r * (2 * D)
                             : (r < H + hk ? ks + (long long)(r - H) * (2 * D)
                                           : vs + (long long)(r - H - hk) * (2 * D));
    return *reinterpret_cast<const uint4*>(s);
  };
  const int r0 = part * p.rows_per_part;
  uint4 w[kDeep];
#pragma unroll
  for (int i = 0; i < kDeep; ++i) {
    const int r = r0 + i * kRows + sub;
    w[i] = r < r_end ? load(r) : make_uint4(0, 0, 0, 0);
  }

  // cosines and sines (with the factor) while the first rows are on their way
  constexpr int kAngles = kHalf ? 8 : 4;
  float cs[kAngles], sn[kAngles];
#pragma unroll
  for (int i = 0; i < kAngles; ++i) {
    const int e = kHalf ? e0 + i : e0 + 2 * i;
    const int j = kHalf ? (e < half ? e : e - half) : e >> 1;
    const unsigned long long turn =
        (unsigned long long)(long long)pos * p.phase[e < rot ? j : 0];
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn[i], &cs[i]);
    cs[i] *= p.factor;
    // the second element of a pair adds the first one's sine, the first subtracts the other's
    sn[i] *= kHalf && e < half ? -p.factor : p.factor;
  }
  // the lane that holds the other halves of this lane's pairs
  const int other = kHalf && kWhole && e0 < rot
                        ? sub * kLanes + (e0 < half ? c + half / 8 : c - half / 8)
                        : lane;

  for (int base = r0; base < r_end; base += kDeep * kRows) {
    uint4 nx[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int r = base + (kDeep + i) * kRows + sub;
      nx[i] = r < r_end ? load(r) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int r = base + i * kRows + sub;
      const bool turns = r < H + hk;
      float x[8], y[8];
      to_float(w[i], x, QT());
      if constexpr (kHalf) {
        if constexpr (kWhole) {
          uint4 o;
          o.x = __shfl_sync(kFull, w[i].x, other);
          o.y = __shfl_sync(kFull, w[i].y, other);
          o.z = __shfl_sync(kFull, w[i].z, other);
          o.w = __shfl_sync(kFull, w[i].w, other);
          to_float(o, y, QT());
        } else {
          const T* row = reinterpret_cast<const T*>(
              (r < H ? qs + (long long)r * (2 * D) : ks + (long long)(r - H) * (2 * D)) - 2 * e0);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = r < r_end && turns && e0 + e < rot
                       ? (float)row[e0 + e < half ? e0 + e + half : e0 + e - half]
                       : 0.0f;
          __syncwarp();  // (q_out may be q: every lane has read the row)
        }
        if (turns) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (kWhole ? e0 < rot : e0 + e < rot) x[e] = x[e] * cs[e] + y[e] * sn[e];
        }
      } else if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e0 + 2 * e < rot) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * cs[e] - b * sn[e];
            x[2 * e + 1] = b * cs[e] + a * sn[e];
          }
        }
      }
      if (r < r_end) {
        // elements that only pass keep their bits
        const bool pass = !turns || e0 >= rot;
        if (r < H) {
          *reinterpret_cast<uint4*>(qd + (long long)r * (2 * D)) = pass ? w[i] : pack8(x, QT());
        } else {
          const bool is_v = r >= H + hk;
          uint8_t* d = (is_v ? vd : kd) + (long long)(r - H - (is_v ? hk : 0)) * (kBlockSize * D * kElem);
          if constexpr (FP8) {
            const float sc = is_v ? p.v_scale : p.k_scale;
            *reinterpret_cast<uint2*>(d) = make_uint2(e4m3x4(x, sc), e4m3x4(x + 4, sc));
          } else {
            *reinterpret_cast<uint4*>(d) = pass ? w[i] : pack8(x, QT());
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) w[i] = nx[i];
  }
}

template <class QT, bool FP8, int D>
int launch_typed(RotParams& p, bool half, cudaStream_t stream) {
  auto kern = !half ? rotary_kernel<QT, FP8, D, false, true>
              : p.pairs % 8 == 0 ? rotary_kernel<QT, FP8, D, true, true>
                                 : rotary_kernel<QT, FP8, D, true, false>;
  // Warps per token: one where the tokens alone fill the GPU (eight warps on every
  // SM), else enough to, in steps of the rows that a warp has in flight at once.
  const int rows = p.num_heads + 2 * p.num_kv_heads, step = kDeep * (32 / (D / 8));
  const long long want = (8LL * sm_count() + p.num_tokens - 1) / p.num_tokens;
  long long per = (rows + want - 1) / want;
  per = (per + step - 1) / step * step;
  p.rows_per_part = (int)per;
  p.parts = (int)((rows + per - 1) / per);
  const long long ctas = ((long long)p.num_tokens * p.parts + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  kern<<<(unsigned)ctas, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <class QT, bool FP8>
int launch_dim(RotParams& p, int head_dim, bool half, cudaStream_t stream) {
  return head_dim == 64 ? launch_typed<QT, FP8, 64>(p, half, stream)
                        : launch_typed<QT, FP8, 128>(p, half, stream);
}

// frac(inv / 2 pi) * 2^64 for |inv| <= 1e3, to within 1.5: inv / 2 pi as the sum of two
// doubles (1 / 2 pi is one, kHi + kLo; the product's rounding comes by fma), of which the
// first one's fraction and the second are whole numbers of 2^-64 turns or nearly.  (The
// product is volatile so that no compiler takes it unrounded into the difference below,
// which would count its rounding twice.)
unsigned long long phase_of(double inv) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const volatile double product = inv * kHi;
  const double turns = product, rest = std::fma(inv, kHi, -turns) + inv * kLo;
  const unsigned long long whole =
      (unsigned long long)(std::fabs(turns - std::trunc(turns)) * 0x1p64);
  return (turns < 0.0 ? 0ull - whole : whole) +
         (unsigned long long)std::llrint(rest * 0x1p64);
}

}  // namespace

int launch_rotary_and_cache(const RotaryArgs& a, const double* inv_freq, cudaStream_t stream) {
  RotParams p{};
  p.q_out = static_cast<uint8_t*>(a.q_out);
  p.q = static_cast<const uint8_t*>(a.q);
  p.k = static_cast<const uint8_t*>(a.k);
  p.v = static_cast<const uint8_t*>(a.v);
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.slots = a.slot_mapping;
  p.positions = a.positions;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.num_tokens = a.num_tokens;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.pairs = a.rotary_dim / 2;
  p.num_slots = (long long)a.num_blocks * kBlockSize;
  p.factor = a.attn_factor;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.errors = a.errors;
  for (int i = 0; i < p.pairs; ++i) p.phase[i] = phase_of(inv_freq[i]);
  const bool fp8 = a.cache_dtype == PKV_FP8_E4M3, half = a.layout == PKV_ROTARY_HALF;
  if (a.src_dtype == PKV_BF16)
    return fp8 ? launch_dim<BF16, true>(p, a.head_dim, half, stream)
               : launch_dim<BF16, false>(p, a.head_dim, half, stream);
  return fp8 ? launch_dim<F16, true>(p, a.head_dim, half, stream)
             : launch_dim<F16, false>(p, a.head_dim, half, stream);
}

}  // namespace pkv

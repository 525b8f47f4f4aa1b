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
// rounding (below 2^-24 turns for every t < 2^30).  Its top 32 bits as a signed
// fraction go through sincospif.  No table is read, so there is none to size for
// the longest context.
//
// A CTA takes a tile of tokens and a share of their rows: it first turns the
// tile's angles into cosines and sines in shared memory (one thread per token
// and pair), then streams rows, a thread per 16-byte chunk (the half layout: the
// two chunks of eight pairs).  Rotation in fp32, one rounding on the way out (to
// 16 bits, or straight to E4M3 after the division by the scale).  HBM bound.

#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;  // head_dim 128

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
  int num_tokens, num_heads, num_kv_heads, head_dim, pairs;
  long long num_slots;
  float factor, k_scale, v_scale;
  uint32_t* errors;
  int tile;  // tokens per CTA
  unsigned long long phase[kMaxPairs];
};

template <class T>
__device__ __forceinline__ uint32_t e4m3x4(const T* f, float scale) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(f[i], scale), __NV_SATFINITE, __NV_E4M3)
         << (8 * i);
  return w;
}

// Where a row of Q, K or V goes: 16-bit elements, or E4M3 codes of x / scale.
struct Dst {
  uint8_t* p;
  bool fp8;
  float scale;
};

template <class QT, int N>
__device__ __forceinline__ void load_n(const uint8_t* src, float* f) {
  if constexpr (N == 8) {
    to_float(__ldg(reinterpret_cast<const uint4*>(src)), f, QT());
  } else {
    f[0] = static_cast<float>(*reinterpret_cast<const typename QT::T*>(src));
  }
}

template <class QT, bool FP8, int N>
__device__ __forceinline__ void store_n(const Dst& d, int elem, const float* f) {
  if (FP8 && d.fp8) {
    if constexpr (N == 8) {
      *reinterpret_cast<uint2*>(d.p + elem) = make_uint2(e4m3x4(f, d.scale), e4m3x4(f + 4, d.scale));
    } else {
      d.p[elem] = __nv_cvt_float_to_fp8(__fdiv_rn(f[0], d.scale), __NV_SATFINITE, __NV_E4M3);
    }
  } else if constexpr (N == 8) {
    *reinterpret_cast<uint4*>(d.p + 2 * (size_t)elem) = pack8(f, QT());
  } else {
    store_out(reinterpret_cast<typename QT::T*>(d.p) + elem, f[0]);
  }
}

// kHalf: half layout, else interleaved.  N: elements per access, 8, or 1 for a
// half layout whose halves are not whole 16-byte chunks.
template <class QT, bool FP8, bool kHalf, int N>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotParams p) {
  extern __shared__ float trig[];  // [tile][2][pairs]: cosines, then sines
  const int t0 = blockIdx.x * p.tile, nt = min(p.tile, p.num_tokens - t0);
  for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
    const int t = i / p.pairs, j = i - t * p.pairs;
    const int pos = __ldg(p.positions + t0 + t);
    const unsigned long long turn = (unsigned long long)(long long)pos * p.phase[j];
    float s, c;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
    trig[(2 * t) * p.pairs + j] = c * p.factor;
    trig[(2 * t + 1) * p.pairs + j] = s * p.factor;
  }
  __syncthreads();

  const int D = p.head_dim, rot = 2 * p.pairs;
  // units of a rotated row: the half layout's pairs of chunks, then single chunks
  const int paired = kHalf ? p.pairs / N : 0;
  const int per_row = kHalf ? paired + (D - rot) / N : D / N;
  const int per_v = D / N;
  const int rot_units = (p.num_heads + p.num_kv_heads) * per_row;
  const int units = rot_units + p.num_kv_heads * per_v;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < nt * units; i += gridDim.y * kThreads) {
    const int t = i / units;
    int u = i - t * units;
    const int tok = t0 + t;
    if (__ldg(p.positions + tok) < 0) continue;  // padding: nothing is written
    const bool is_v = u >= rot_units;
    if (is_v) u -= rot_units;
    const int per = is_v ? per_v : per_row;
    int h = u / per;
    u -= h * per;
    const uint8_t* src;
    Dst d;
    if (!is_v && h < p.num_heads) {
      src = p.q + 2 * (tok * p.q_stride + (long long)h * D);
      d = {p.q_out + 2 * ((long long)tok * p.num_heads + h) * D, false, 1.0f};
    } else {
      if (!is_v) h -= p.num_heads;
      const int64_t slot = __ldg(p.slots + tok);
      if (slot < 0) continue;  // not cached
      if (slot >= p.num_slots) {
        if (!is_v && h == 0 && u == 0) flag_error(p.errors, PKV_DEVERR_SLOT);
        continue;
      }
      src = is_v ? p.v + 2 * (tok * p.v_stride + (long long)h * D)
                 : p.k + 2 * (tok * p.k_stride + (long long)h * D);
      const long long row = ((slot / kBlockSize) * p.num_kv_heads + h) * kBlockSize + slot % kBlockSize;
      d = {(is_v ? p.v_cache : p.k_cache) + row * D * (FP8 ? 1 : 2), FP8,
           is_v ? p.v_scale : p.k_scale};
    }
    const float* cs = trig + 2 * t * p.pairs;
    const float* sn = cs + p.pairs;
    if (kHalf && !is_v && u < paired) {
      float a[N], b[N], x[N], y[N];
      load_n<QT, N>(src + 2 * u * N, a);
      load_n<QT, N>(src + 2 * (u * N + p.pairs), b);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float c = cs[u * N + e], s = sn[u * N + e];
        x[e] = a[e] * c - b[e] * s;
        y[e] = b[e] * c + a[e] * s;
      }
      store_n<QT, FP8, N>(d, u * N, x);
      store_n<QT, FP8, N>(d, u * N + p.pairs, y);
    } else {
      const int e0 = is_v ? u * N : (kHalf ? rot + (u - paired) * N : u * N);
      float a[N];
      load_n<QT, N>(src + 2 * e0, a);
      if constexpr (!kHalf) {
        if (!is_v) {
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const int j = (e0 + e) / 2;
            if (j < p.pairs) {
              const float x = a[e], y = a[e + 1];
              a[e] = x * cs[j] - y * sn[j];
              a[e + 1] = y * cs[j] + x * sn[j];
            }
          }
        }
      }
      store_n<QT, FP8, N>(d, e0, a);
    }
  }
}

template <class QT, bool FP8>
int launch_typed(RotParams& p, bool half, cudaStream_t stream) {
  const bool whole = !half || p.pairs % 8 == 0;
  auto kern = !half ? rotary_kernel<QT, FP8, false, 8>
                    : (whole ? rotary_kernel<QT, FP8, true, 8> : rotary_kernel<QT, FP8, true, 1>);
  // enough CTAs for every SM: tiles of four tokens, or single tokens whose rows
  // are shared by several CTAs
  const int sms = sm_count();
  p.tile = p.num_tokens >= 8 * sms ? 4 : 1;
  const int tiles = (p.num_tokens + p.tile - 1) / p.tile;
  const int n = whole ? 8 : 1;
  const long long units = (long long)p.tile * (p.num_heads + 2 * p.num_kv_heads) * (p.head_dim / n);
  long long split = (4LL * sms + tiles - 1) / tiles;
  const long long most = (units + kThreads - 1) / kThreads;
  if (split > most) split = most;
  if (split < 1) split = 1;
  const dim3 grid((unsigned)tiles, (unsigned)split);
  kern<<<grid, kThreads, (size_t)p.tile * 2 * p.pairs * sizeof(float), stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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
  p.head_dim = a.head_dim;
  p.pairs = a.rotary_dim / 2;
  p.num_slots = (long long)a.num_blocks * kBlockSize;
  p.factor = a.attn_factor;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.errors = a.errors;
  for (int i = 0; i < p.pairs; ++i) {
    const double turns = inv_freq[i] / 6.283185307179586476925286766559;
    const double frac = turns - std::floor(turns);  // [0, 1)
    p.phase[i] = frac < 1.0 ? (unsigned long long)(frac * 0x1p64) : 0ull;
  }
  const bool fp8 = a.cache_dtype == PKV_FP8_E4M3, half = a.layout == PKV_ROTARY_HALF;
  if (a.src_dtype == PKV_BF16)
    return fp8 ? launch_typed<BF16, true>(p, half, stream)
               : launch_typed<BF16, false>(p, half, stream);
  return fp8 ? launch_typed<F16, true>(p, half, stream)
             : launch_typed<F16, false>(p, half, stream);
}

}  // namespace pkv

// AdamW over many tensors in one launch (include/salr.h, salr_adamw_step).
//
// Per element, in fp32:  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
// p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
// 8-bit states hold m and s = sqrt(v) of 256 elements as e4m3 codes times
// largest / 448 (v spans twice the exponents of its root, which the format's
// 2^-9 .. 448 would not hold), the nearest code or one of the two around the
// value by chance.
//
// One workgroup per chunk of a tensor (2048 or 4096 elements), found in the
// plan's chunk list; 8 consecutive elements a thread, so a float array moves
// 32 bytes and the codes 8 bytes a thread, and an 8-bit run is 32 lanes of one
// wave.  Bound by HBM: 24 bytes an element with float states, 12 with 8-bit
// ones (bf16 parameters, float gradients, no master), 6 more with a master.
// 201 M with float states and masters: 1047 to 1101 us, 5.5 to 5.8 TB/s by
// where the arrays lie, without masters 800, 6.0 TB/s; 53 M with 8-bit states:
// 110 us, 5.8 TB/s; rounded by chance 128, then bound by the issue of
// instructions (201 M: 410 and 474 us; with masters 660 and 620, HBM in both).
#include <hip/hip_runtime.h>

#include "salr_device.hpp"
#include "salr_kernels.hpp"

namespace salr {
namespace {

constexpr int kPer = 8;  // elements a thread
constexpr int kRunLanes = 256 / kPer;
constexpr float kTiny = 0x1p-100f;

// Stores past the caches: nothing written is read again before the next step
// (201 M parameters with masters, mean over eight placements: 1072 us, cached
// 1097; without masters 803 either way).
template <class V>
__device__ __forceinline__ void stream_store(V* p, V v) {
  __builtin_nontemporal_store(v, p);
}

// 8 elements from i on; unless WHOLE those at or past n read as 0 (from the
// last one's address: no branch keeps the loads apart) and are not written.
// Pointers are 16-byte aligned and i is a multiple of 8, so whole groups move
// as 16-byte vectors.
template <bool WHOLE>
__device__ __forceinline__ void load8(const float* p, int64_t i, int64_t n, float* x) {
  if (WHOLE || i + kPer <= n) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p + i), b = *reinterpret_cast<const f32x4_t*>(p + i + 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] = a[c];
      x[c + 4] = b[c];
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) x[c] = p[min(i + c, n - 1)];
#pragma unroll
    for (int c = 0; c < kPer; ++c) x[c] = i + c < n ? x[c] : 0.f;
  }
}
template <bool WHOLE>
__device__ __forceinline__ void load8(const uint16_t* p, int64_t i, int64_t n, float* x) {
  if (WHOLE || i + kPer <= n) {
    const u32x4_t a = load16(p + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[2 * c] = bf16_to_f32((uint16_t)a[c]);
      x[2 * c + 1] = bf16_to_f32((uint16_t)(a[c] >> 16));
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) x[c] = bf16_to_f32(p[min(i + c, n - 1)]);
#pragma unroll
    for (int c = 0; c < kPer; ++c) x[c] = i + c < n ? x[c] : 0.f;
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store8(float* p, int64_t i, int64_t n, const float* x) {
  if (WHOLE || i + kPer <= n) {
    stream_store(reinterpret_cast<f32x4_t*>(p + i), f32x4_t{x[0], x[1], x[2], x[3]});
    stream_store(reinterpret_cast<f32x4_t*>(p + i + 4), f32x4_t{x[4], x[5], x[6], x[7]});
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) p[i + c] = x[c];
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store8(uint16_t* p, int64_t i, int64_t n, const float* x) {
  if (WHOLE || i + kPer <= n) {
    u32x4_t w;
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = (uint32_t)f32_to_bf16(x[2 * c]) | ((uint32_t)f32_to_bf16(x[2 * c + 1]) << 16);
    stream_store(reinterpret_cast<u32x4_t*>(p + i), w);
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) p[i + c] = f32_to_bf16(x[c]);
  }
}

// 8 codes as two words (the codes past n as 0).
template <bool WHOLE>
__device__ __forceinline__ u32x2_t load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if (WHOLE || i + kPer <= n) return *reinterpret_cast<const u32x2_t*>(p + i);
  uint32_t b[kPer], w[2] = {0u, 0u};
#pragma unroll
  for (int c = 0; c < kPer; ++c) b[c] = p[min(i + c, n - 1)];
#pragma unroll
  for (int c = 0; c < kPer; ++c) w[c / 4] |= i + c < n ? b[c] << (8 * (c % 4)) : 0u;
  return u32x2_t{w[0], w[1]};
}
template <bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, u32x2_t w) {
  if (WHOLE || i + kPer <= n) {
    stream_store(reinterpret_cast<u32x2_t*>(p + i), w);
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) p[i + c] = (uint8_t)((c < 4 ? w.x : w.y) >> (8 * (c % 4)));
  }
}
__device__ __forceinline__ void decode8(u32x2_t w, float scale, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int word = (int)(h ? w.y : w.x);
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
    x[4 * h] = lo[0] * scale;
    x[4 * h + 1] = lo[1] * scale;
    x[4 * h + 2] = hi[0] * scale;
    x[4 * h + 3] = hi[1] * scale;
  }
}
__device__ __forceinline__ u32x2_t encode8(const float* x) {
  int w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], 0, false);
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], w[h], true);
  }
  return u32x2_t{(uint32_t)w[0], (uint32_t)w[1]};
}

// The largest |x| of a run (32 lanes; NaN left aside), the run's scale and
// its inverse (0 and 0 for a run of zeros).
template <int N>
__device__ __forceinline__ float row_max(float v) {  // with the lane N before in its row of 16, cyclically
  const int i = __float_as_int(v);
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x120 + N, 0xF, 0xF, false)));
}
__device__ __forceinline__ void run_scale(const float* x, float* scale, float* inv) {
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) top = fmaxf(top, fabsf(x[c]));
  top = row_max<1>(row_max<2>(row_max<4>(row_max<8>(top))));
  top = fmaxf(top, __shfl_xor(top, 16, kRunLanes));
  const bool live = top >= kTiny;
  *scale = live ? top / 448.f : 0.f;
  *inv = live ? 448.f / top : 0.f;
}

// ---- random rounding of the codes ----
//
// A value x between two codes lo <= x < hi takes hi with a chance that makes
// what is expected of the stored value x itself: (x - lo) / (hi - lo) for m,
// and for s = sqrt(v) the chance of the squares, (x^2 - lo^2) / (hi^2 - lo^2),
// so that v is.  Only then do m and v follow their recurrences: a step changes
// s by (1 - b2) / 2 at most downwards, far below half a code, and rounding to
// the nearest would undo it every time.

// x's bits mixed, one to one (two multiplications by odd constants, the first
// bits of the roots of 2 and 3, between shifts).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B9u;

// Elements at or past 2^-6 (in scales) lie in steps of 1/8 of their power of
// two, so that the code below is a float's bits cut off after three; smaller
// ones in steps of 2^-9, as the floats in [2^-6, 2^-5) do.
constexpr uint32_t kCodeBits = 0xFFF00000u;
__device__ __forceinline__ float code_shift(float x) { return x < 0x1p-6f ? 0x1p-6f : 0.f; }

__device__ __forceinline__ float random_m(float x, uint32_t r) {
  const float mag = fminf(fabsf(x), 448.f);  // (the scale's rounding can leave 448 and an ulp)
  const float shift = code_shift(mag);
  const uint32_t b = (__float_as_uint(mag + shift) + (r & ~kCodeBits)) & kCodeBits;
  return x == x ? copysignf(__uint_as_float(b) - shift, x) : x;
}

__device__ __forceinline__ float random_s(float x, uint32_t r) {
  const float mag = fminf(x, 448.f);
  const float shift = code_shift(mag);
  const uint32_t b = __float_as_uint(mag + shift) & kCodeBits;
  const float lo = __uint_as_float(b) - shift, hi = __uint_as_float(b + ~kCodeBits + 1) - shift;
  const bool up = (float)r * 0x1p-32f * ((hi - lo) * (hi + lo)) < (mag - lo) * (mag + lo);
  return x == x ? (up ? hi : lo) : x;
}

// Square roots to 1 ulp (the instruction alone takes no subnormal: values
// below 2^-96, zeros among them, go scaled).
__device__ __forceinline__ void roots(const float* v, float* s) {
  float low = v[0];
#pragma unroll
  for (int c = 1; c < kPer; ++c) low = fminf(low, v[c]);
  if (low < 0x1p-96f) {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const bool tiny = v[c] < 0x1p-96f;
      s[c] = __builtin_amdgcn_sqrtf(tiny ? v[c] * 0x1p32f : v[c]) * (tiny ? 0x1p-16f : 1.f);
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) s[c] = __builtin_amdgcn_sqrtf(v[c]);
  }
}

// What a thread holds of its 8 elements.
template <class P, class G, bool S8, bool MASTER>
struct Eight {
  float g[kPer], m[kPer], v[kPer], p[kPer];
  float s[kPer];  // root of v (8-bit states)
  u32x2_t mc, vc;

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int c = 0; c < kPer; ++c) g[c] = m[c] = v[c] = p[c] = 0.f;
    mc = vc = u32x2_t{0u, 0u};
  }

  template <bool WHOLE>
  __device__ __forceinline__ void load(const AdamwTensor& t, int64_t i) {
    load8<WHOLE>(static_cast<const G*>(t.g), i, t.n, g);
    if constexpr (S8) {
      mc = load_codes<WHOLE>(static_cast<const uint8_t*>(t.m), i, t.n);
      vc = load_codes<WHOLE>(static_cast<const uint8_t*>(t.v), i, t.n);
    } else {
      load8<WHOLE>(static_cast<const float*>(t.m), i, t.n, m);
      load8<WHOLE>(static_cast<const float*>(t.v), i, t.n, v);
    }
    if constexpr (MASTER) load8<WHOLE>(t.master, i, t.n, p);
    else load8<WHOLE>(static_cast<const P*>(t.p), i, t.n, p);
  }

  template <bool WHOLE>
  __device__ __forceinline__ void store(const AdamwTensor& t, int64_t i) const {
    if constexpr (MASTER) store8<WHOLE>(t.master, i, t.n, p);
    store8<WHOLE>(static_cast<P*>(t.p), i, t.n, p);
    if constexpr (S8) {
      store_codes<WHOLE>(static_cast<uint8_t*>(t.m), i, t.n, mc);
      store_codes<WHOLE>(static_cast<uint8_t*>(t.v), i, t.n, vc);
    } else {
      store8<WHOLE>(static_cast<float*>(t.m), i, t.n, m);
      store8<WHOLE>(static_cast<float*>(t.v), i, t.n, v);
    }
  }
};

// FULL: the chunk has all its elements.  RANDOM: 8-bit codes by chance, from
// the bits of `key` (the chunk's) and the element's place.
template <class P, class G, bool S8, bool MASTER, bool RANDOM, bool FULL>
__device__ __forceinline__ void adamw_elements(const AdamwArgs& a, const AdamwTensor& t, int64_t i, uint32_t key) {
#pragma clang fp contract(off)
  const int64_t run = i / 256;
  float decay = a.decay, rate = a.rate, gs = a.grad_scale, isb2 = a.inv_sqrt_bias2;
  if (a.dyn) {
    const float lr = a.dyn[0];
    gs = a.dyn[1];
    decay = 1.f - lr * a.weight_decay;
    rate = lr * a.dyn[2];
    isb2 = a.dyn[3];
  }
  Eight<P, G, S8, MASTER> x;
  // (one branch around all the loads: around each, they wait for one another)
  const bool whole = FULL || i + kPer <= t.n, some = FULL || i < t.n;
  float scale_m = 0.f, scale_s = 0.f;
  if (S8 && some) {
    scale_m = t.ms[run];
    scale_s = t.vs[run];
  }
  if (whole) x.template load<true>(t, i);
  else if (some) x.template load<false>(t, i);
  else x.zero();
  if constexpr (S8) {
    decode8(x.mc, scale_m, x.m);
    decode8(x.vc, scale_s, x.s);
#pragma unroll
    for (int c = 0; c < kPer; ++c) x.v[c] = x.s[c] * x.s[c];
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    x.g[c] *= gs;
    x.m[c] = x.m[c] * a.beta1 + x.g[c] * a.rest1;
    x.v[c] = x.v[c] * a.beta2 + (x.g[c] * x.g[c]) * a.rest2;
  }
  roots(x.v, x.s);
#pragma unroll
  for (int c = 0; c < kPer; ++c)  // (the reciprocal to 1 ulp: the quotient's error stays far below m's)
    x.p[c] = x.p[c] * decay - (x.m[c] * __builtin_amdgcn_rcpf(x.s[c] * isb2 + a.eps)) * rate;
  if constexpr (S8) {
    float inv_m, inv_s;
    run_scale(x.m, &scale_m, &inv_m);
    run_scale(x.s, &scale_s, &inv_s);
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      x.m[c] *= inv_m;
      x.s[c] *= inv_s;
      x.s[c] = x.s[c] > 0.f ? fmaxf(x.s[c], 0x1p-9f) : x.s[c];  // (the smallest code)
      if constexpr (RANDOM) {
        const uint32_t r = mix(key + (uint32_t)(i + c) * kGolden);
        x.m[c] = random_m(x.m[c], r);  // (by its low 20 bits, s by all from the top)
        x.s[c] = random_s(x.s[c], r);
      }
    }
    x.mc = encode8(x.m);
    x.vc = encode8(x.s);
    if (some && (threadIdx.x & (kRunLanes - 1)) == 0) {
      t.ms[run] = scale_m;
      t.vs[run] = scale_s;
    }
  }
  if (whole) x.template store<true>(t, i);
  else if (some) x.template store<false>(t, i);
}

template <class P, class G, bool S8, bool MASTER, bool RANDOM>
__global__ __launch_bounds__(adamw_chunk(S8, MASTER) / kPer) void adamw_kernel(AdamwArgs a) {
  constexpr int kChunk = adamw_chunk(S8, MASTER);
  const AdamwChunk ch = a.chunks[blockIdx.x];
  const AdamwTensor t = a.tensors[ch.tensor];
  const int64_t base = (int64_t)ch.chunk * kChunk, i = base + threadIdx.x * kPer;
  uint32_t key = 0;
  if constexpr (RANDOM) {
    key = mix(a.seed + kGolden);
    key = mix(key ^ __float_as_uint(a.dyn ? a.dyn[4] : a.step));
    key = mix(key ^ (uint32_t)ch.tensor);
    key = mix(key ^ (uint32_t)(base >> 32));
  }
  if (base + kChunk <= t.n) adamw_elements<P, G, S8, MASTER, RANDOM, true>(a, t, i, key);
  else adamw_elements<P, G, S8, MASTER, RANDOM, false>(a, t, i, key);
}

// Loads in flight a CU: more of them than about 80 KB open more DRAM pages
// than it serves well, so the waves a CU holds are bounded, by asking for a
// share of its LDS (201 M bf16 parameters, float gradients and states, 28 KB
// of loads in 4 waves: 32 waves a CU 937 us, 16 933, 12 901, 8 818, 4 1012;
// 53 M with 8-bit states, 16 KB: 32 waves 128, 24 122, 16 117, 12 130, 8
// 164).  Eight, sixteen or twenty-four waves then load 48 to 80 KB.
constexpr int kLdsUnits = 128, kLdsUnit = 1280;  // a CU's LDS, as it is given out
constexpr int kFlightBytes = 80 * 1024;

template <class P, class G, bool S8, bool MASTER, bool RANDOM>
void launch(const AdamwArgs& a, hipStream_t s) {
  constexpr int kThreads = adamw_chunk(S8, MASTER) / kPer;
  constexpr int kFourWaves = 256 * kPer * (int)(sizeof(G) + (S8 ? 2 : 8) + (MASTER ? 4 : sizeof(P)));  // bytes
  constexpr int kGroups = (kFlightBytes / kFourWaves & ~1) * 256 / kThreads;
  static_assert(kGroups >= 1 && kGroups * kThreads <= 2048, "workgroups a CU");
  hipLaunchKernelGGL((adamw_kernel<P, G, S8, MASTER, RANDOM>), dim3((unsigned)a.n_chunks), dim3(kThreads),
                     kLdsUnits / kGroups * kLdsUnit, s, a);
}

template <class P, class G, bool MASTER>
void launch_g(const AdamwArgs& a, bool state8, bool random, hipStream_t s) {
  if (!state8) launch<P, G, false, MASTER, false>(a, s);
  else if (random) launch<P, G, true, MASTER, true>(a, s);
  else launch<P, G, true, MASTER, false>(a, s);
}
template <class P, bool MASTER>
void launch_p(const AdamwArgs& a, bool g_f32, bool state8, bool random, hipStream_t s) {
  if (g_f32) launch_g<P, float, MASTER>(a, state8, random, s);
  else launch_g<P, uint16_t, MASTER>(a, state8, random, s);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, bool p_f32, bool g_f32, bool state8, bool master, bool random,
                        hipStream_t s) {
  if (a.n_chunks == 0) return hipSuccess;
  if (p_f32) launch_p<float, false>(a, g_f32, state8, random, s);
  else if (master) launch_p<uint16_t, true>(a, g_f32, state8, random, s);
  else launch_p<uint16_t, false>(a, g_f32, state8, random, s);
  return hipGetLastError();
}

}  // namespace salr

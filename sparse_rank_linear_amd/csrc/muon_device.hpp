// Device code that the kernels of the orthogonalised step share.
#pragma once

#include "salr_device.hpp"
#include "salr_muon.hpp"

namespace salr {

typedef double f64x4_t __attribute__((ext_vector_type(4)));
typedef double f64x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// D of the double form: lane (i, g) holds rows 4e + g of column i.
__device__ __forceinline__ f64x4_t mfma_f64(double a, double b, f64x4_t c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ void lower_tile(int t, int* ti, int* tj) {
  int i = 0;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  *ti = i;
  *tj = t - i * (i + 1) / 2;
}

// Pointers that a kernel reads from memory, as pointers to global memory: the
// compiler would take them for pointers to anything, and such (flat) accesses
// count as LDS accesses too, so every wait for LDS would wait for them.
template <class T>
using global = __attribute__((address_space(1))) T*;
template <class T, class V>
__device__ __forceinline__ global<T> to_global(V* p) {
  return (global<T>)p;
}

// Four consecutive values of a float or bf16 array as they are loaded
// (converted only where they are used: a load stays in flight until then).
// Rows may start anywhere.
template <bool F32>
struct Four;
template <>
struct Four<true> {
  typedef f32x4_t raw;
  typedef float elem;
  typedef float any __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ f32x4_t value(raw x) { return x; }
  static __device__ __forceinline__ raw part(global<const elem> p, int n) {
    f32x4_t x = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) x[e] = p[e];
    return x;
  }
  static __device__ __forceinline__ any pack(f32x4_t x) { return x; }
  static __device__ __forceinline__ elem one(float x) { return x; }
};
template <>
struct Four<false> {
  typedef u32x2_t raw;
  typedef uint16_t elem;
  typedef uint32_t any __attribute__((ext_vector_type(2), aligned(2)));
  static __device__ __forceinline__ f32x4_t value(raw w) {
    return f32x4_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                   __uint_as_float(w.y & 0xFFFF0000u)};
  }
  static __device__ __forceinline__ raw part(global<const elem> p, int n) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) w[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    return raw{w[0], w[1]};
  }
  static __device__ __forceinline__ any pack(f32x4_t x) {
    return any{f32_to_bf16(x[0]) | (uint32_t)f32_to_bf16(x[1]) << 16,
               f32_to_bf16(x[2]) | (uint32_t)f32_to_bf16(x[3]) << 16};
  }
  static __device__ __forceinline__ elem one(float x) { return f32_to_bf16(x); }
};
template <bool F32>
__device__ __forceinline__ typename Four<F32>::raw load4(global<const typename Four<F32>::elem> p) {
  return *(global<const typename Four<F32>::any>)p;
}
// Waits for every load and store of the wave.  (Registers that are loaded once
// before a loop are waited for here: the compiler would wait for them in the
// loop, and so for the loads in flight there.)
__device__ __forceinline__ void wait_memory() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// A stage: KB columns of the long side from k on (`left` of them before the
// chunk's end), in groups of four elements that lie together in memory: of a
// wide matrix along its rows (the long side), of a tall one along the flat
// array.  In LDS a wide matrix's stage is [short][PITCH], a tall one's
// [long][PITCH]: whole groups either way (but where a tall matrix's rows are no
// multiple of four, whose groups run over their ends).  Thread t takes groups
// t, t + THREADS, ...
template <bool WIDE, int KB, int THREADS, int NQ>
struct Stage {
  int s, tid;
  int64_t L;
  uint32_t base[NQ];  // the group's first element, from the stage's on (a matrix has less than 2^29)
  __device__ __forceinline__ Stage(int s_, int64_t L_, int tid_) : s(s_), tid(tid_), L(L_) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      // (a thread without a group loads the last one's too)
      const int x = min(group(q), s * (KB / 4) - 1);
      base[q] = WIDE ? (uint32_t)(x / (KB / 4)) * (uint32_t)L + x % (KB / 4) * 4 : (uint32_t)(4 * x);
    }
  }
  __device__ __forceinline__ int group(int q) const { return tid + q * THREADS; }
  __device__ __forceinline__ bool has(int q) const { return group(q) < s * (KB / 4); }
  // (one address for all lanes, and a lane's 32 bits from there)
  template <class T>
  __device__ __forceinline__ global<T> element(global<T> p, int q, int64_t k) const {
    typedef std::conditional_t<std::is_const<T>::value, const char, char> byte;
    return (global<T>)((global<byte>)(p + (WIDE ? k : k * s)) + (uint32_t)(base[q] * (uint32_t)sizeof(T)));
  }
  // elements of group q (0 without one)
  __device__ __forceinline__ int count(int q, int left) const {
    const int x = group(q);
    if (!has(q)) return 0;
    return left >= KB ? 4 : max(0, min(4, WIDE ? left - x % (KB / 4) * 4 : left * s - 4 * x));
  }
  // A stage's groups: whole stages in one batch without branches, the rest of
  // the long side piece by piece.
  template <bool FULL, bool F32>
  __device__ __forceinline__ void load(global<const typename Four<F32>::elem> p, int64_t k, int left,
                                       typename Four<F32>::raw (&v)[NQ]) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      v[q] = FULL ? load4<F32>(element(p, q, k)) : Four<F32>::part(element(p, q, k), count(q, left));
  }
  template <bool FULL, bool F32>
  __device__ __forceinline__ void store(global<typename Four<F32>::elem> p, int q, int64_t k, int left,
                                        f32x4_t x) const {
    if (FULL) {
      if (has(q)) *(global<typename Four<F32>::any>)element(p, q, k) = Four<F32>::pack(x);
    } else {
      const int n = count(q, left);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) element(p, q, k)[e] = Four<F32>::one(x[e]);
    }
  }
  template <int PITCH>
  __device__ __forceinline__ int place(int q) const {
    const int x = WIDE ? group(q) : min(group(q), s * (KB / 4) - 1);
    return WIDE ? x / (KB / 4) * PITCH + x % (KB / 4) * 4 : 4 * x / s * PITCH + 4 * x % s;
  }
  template <int PITCH>
  __device__ __forceinline__ void put(float* lds, int at, f32x4_t x) const {
    if (WIDE || (s & 3) == 0) {
      *reinterpret_cast<f32x4_t*>(lds + at) = x;
    } else {
      int i = at % PITCH;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lds[at] = x[e];
        ++at;
        if (++i == s) {
          i = 0;
          at += PITCH - s;
        }
      }
    }
  }
  template <int PITCH>
  __device__ __forceinline__ f32x4_t get(const float* lds, int at) const {
    if (WIDE || (s & 3) == 0) return *reinterpret_cast<const f32x4_t*>(lds + at);
    f32x4_t x;
    int i = at % PITCH;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = lds[at];
      ++at;
      if (++i == s) {
        i = 0;
        at += PITCH - s;
      }
    }
    return x;
  }
};

}  // namespace salr

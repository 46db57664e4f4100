// The orthogonalised step over many matrices (include/salr.h,
// salr_muon_step).
//
// With u the update (momentum), X_0 = u / (|u|_F + eps) and A_k = X_k X_k^T
// (X with its short side first), a Newton-Schulz step is
//   X_{k+1} = P_k X_k,   P_k = a I + b A_k + c A_k^2.
// Every P_k is a polynomial of A_0, so they commute and
//   A_{k+1} = P_k A_k P_k,   X_n = Q X_0,   Q = P_{n-1} ... P_0:
// the long side is read for the product A_0 (whose trace is |u|_F^2) and once
// more for Q X_0; all that lies between is on s x s matrices.  Three kernels:
//   gram     m and u from the gradient, u u^T in pieces of the long side
//   iterate  the pieces' sum, the steps, Q
//   apply    u again, Q u, the parameters
#include <hip/hip_runtime.h>

#include <type_traits>

#include "salr_device.hpp"
#include "salr_muon.hpp"

namespace salr {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));
typedef double f64x2_t __attribute__((ext_vector_type(2)));
// (rows may start anywhere)
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));

__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// D of the double form: lane (i, g) holds rows 4e + g of column i.
__device__ __forceinline__ f64x4_t mfma_f64(double a, double b, f64x4_t c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// n of four values from element i of a float or bf16 array; the others are 0.
__device__ __forceinline__ f32x4_t load4(const void* p, bool f32, int64_t i, int n) {
  f32x4_t x = zero4();
  if (f32) {
    const float* q = static_cast<const float*>(p) + i;
    if (n == 4) return *reinterpret_cast<const f32x4_any_t*>(q);
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) x[e] = q[e];
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (n == 4) {
      const u32x2_t w = *reinterpret_cast<const u32x2_any_t*>(q);
      return f32x4_t{bf16_to_f32((uint16_t)w.x), bf16_to_f32((uint16_t)(w.x >> 16)), bf16_to_f32((uint16_t)w.y),
                     bf16_to_f32((uint16_t)(w.y >> 16))};
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) x[e] = bf16_to_f32(q[e]);
  }
  return x;
}
__device__ __forceinline__ void store4(void* p, bool f32, int64_t i, int n, f32x4_t x) {
  if (f32) {
    float* q = static_cast<float*>(p) + i;
    if (n == 4) *reinterpret_cast<f32x4_any_t*>(q) = x;
    else
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) q[e] = x[e];
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if (n == 4) {
      *reinterpret_cast<u32x2_any_t*>(q) = u32x2_t{f32_to_bf16(x[0]) | (uint32_t)f32_to_bf16(x[1]) << 16,
                                                   f32_to_bf16(x[2]) | (uint32_t)f32_to_bf16(x[3]) << 16};
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) q[e] = f32_to_bf16(x[e]);
    }
  }
}

// A stage: KB columns of the long side from k0 on (those before k1), held in
// LDS as [short][KP].  Its elements in groups of four that lie together in
// memory: of a wide matrix along the long side, of a tall one along the flat
// array (a group may run over a row's end).
template <int KB>
struct Stage {
  static constexpr int KP = KB + 4;
  int s;
  int64_t L;
  bool wide;
  __device__ __forceinline__ int groups() const { return wide ? s * (KB / 4) : (s * KB + 3) / 4; }
  // group q: element index in the matrix, elements of it that exist
  __device__ __forceinline__ void locate(int q, int64_t k0, int64_t k1, int64_t* at, int* n) const {
    if (wide) {
      const int i = q / (KB / 4), c = q % (KB / 4) * 4;
      *at = (int64_t)i * L + k0 + c;
      *n = (int)max((int64_t)0, min((int64_t)4, k1 - k0 - c));
    } else {
      *at = k0 * s + 4 * q;
      *n = (int)max((int64_t)0, min((int64_t)4, min(k1 * s, (k0 + KB) * s) - *at));
    }
  }
  __device__ __forceinline__ void put(float* lds, int q, f32x4_t x) const {
    if (wide) {
      *reinterpret_cast<f32x4_t*>(lds + q / (KB / 4) * KP + q % (KB / 4) * 4) = x;
    } else {
      int k = 4 * q / s, i = 4 * q - k * s;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k < KB) lds[i * KP + k] = x[e];
        if (++i == s) {
          i = 0;
          ++k;
        }
      }
    }
  }
  __device__ __forceinline__ f32x4_t get(const float* lds, int q) const {
    if (wide) return *reinterpret_cast<const f32x4_t*>(lds + q / (KB / 4) * KP + q % (KB / 4) * 4);
    f32x4_t x = zero4();
    int k = 4 * q / s, i = 4 * q - k * s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (k < KB) x[e] = lds[i * KP + k];
      if (++i == s) {
        i = 0;
        ++k;
      }
    }
    return x;
  }
};

// ---- gram ----
//
// 8 waves; GROUPS of them share the lower tiles of u u^T, and 8 / GROUPS take
// every such part of the columns.  A stage's sum (KB columns at most) is float,
// then joins a double: the smallest eigenvalues decide how fast their
// directions grow, and a float sum over thousands of columns would drown them.
template <int NT>
struct GramShape {
  static constexpr int kTiles = muon_lower(NT);
  static constexpr int kGroups = NT <= 3 ? 1 : NT <= 8 ? 4 : 8;
  static constexpr int kParts = 8 / kGroups;
  static constexpr int kPer = (kTiles + kGroups - 1) / kGroups;  // tiles of a wave
};
constexpr int kGramThreads = 512;

__device__ __forceinline__ void lower_tile(int t, int* ti, int* tj) {
  int i = 0;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  *ti = i;
  *tj = t - i * (i + 1) / 2;
}

template <int NT>
__global__ __launch_bounds__(kGramThreads) void muon_gram_kernel(MuonArgs a, int64_t c0) {
  constexpr int KB = muon_stage(NT), KP = Stage<KB>::KP, S = 16 * NT;
  using Shape = GramShape<NT>;
  constexpr int kNq = (S * KB / 4 + kGramThreads - 1) / kGramThreads;
  extern __shared__ __attribute__((aligned(16))) float lds[];  // [S][KP]
  const MuonChunk ch = a.chunks[c0 + blockIdx.x];
  const MuonMatrix& M = a.matrices[ch.matrix];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const Stage<KB> st{M.s, M.L, M.wide != 0};
  const int64_t k0 = (int64_t)ch.part * M.chunk, k1 = min(M.L, k0 + M.chunk);
  const float gs = a.dyn ? a.dyn[1] : a.grad_scale;
  const void* grad = M.g;
  float* mom = M.m;
  const int n_groups = st.groups();
  for (int q = tid; q < S * KP; q += kGramThreads) lds[q] = 0.f;  // (rows from s on stay so)
  const int group = wave % Shape::kGroups, part = wave / Shape::kGroups;
  f64x4_t sum[Shape::kPer];
  int row_i[Shape::kPer], row_j[Shape::kPer];
#pragma unroll
  for (int t = 0; t < Shape::kPer; ++t) {
    sum[t] = f64x4_t{0, 0, 0, 0};
    int ti, tj;
    lower_tile(min(group + t * Shape::kGroups, Shape::kTiles - 1), &ti, &tj);
    row_i[t] = (16 * ti + i) * KP + 4 * g;
    row_j[t] = (16 * tj + i) * KP + 4 * g;
  }
  f32x4_t vg[kNq], vm[kNq];
  const auto load = [&](int64_t k) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int x = tid + q * kGramThreads;
      int64_t at = 0;
      int n = 0;
      if (x < n_groups) st.locate(x, k, k1, &at, &n);
      vg[q] = load4(grad, a.g_f32, at, n);
      vm[q] = load4(mom, true, at, n);
    }
  };
  load(k0);
  for (int64_t k = k0; k < k1; k += KB) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int x = tid + q * kGramThreads;
      if (x >= n_groups) continue;
      int64_t at;
      int n;
      st.locate(x, k, k1, &at, &n);
      const f32x4_t gg = vg[q] * gs, mm = a.momentum * vm[q] + gg;
      if (n > 0) store4(mom, true, at, n, mm);
      st.put(lds, x, a.nesterov ? gg + a.momentum * mm : mm);
    }
    __syncthreads();
    if (k + KB < k1) load(k + KB);
    f32x4_t acc[Shape::kPer];
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) acc[t] = zero4();
#pragma unroll
    for (int c = 0; c < KB / 16 / Shape::kParts; ++c) {
      const int col = 16 * (part + c * Shape::kParts);
#pragma unroll
      for (int t = 0; t < Shape::kPer; ++t) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(lds + row_i[t] + col);
        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(lds + row_j[t] + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t] = mfma_f32(x[e], y[e], acc[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[t][e] += (double)acc[t][e];
  }
  // the column parts meet in LDS, in order
  f32x4_t* out = reinterpret_cast<f32x4_t*>(M.parts + (int64_t)ch.part * Shape::kTiles * 256);
  double* mine = reinterpret_cast<double*>(lds);
  for (int q = Shape::kParts - 1; q > 0; --q) {
    // (one tile of a group at a time: its LDS is as large as the stage's at least)
    for (int t = 0; t < Shape::kPer; ++t) {
      __syncthreads();
      double* at = mine + (group * 64 + lane) * 4;
      if (part == q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          double v = 0;
#pragma unroll
          for (int z = 0; z < Shape::kPer; ++z) v = z == t ? sum[z][e] : v;
          at[e] = v;
        }
      __syncthreads();
      if (part == q - 1)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int z = 0; z < Shape::kPer; ++z) sum[z][e] += z == t ? at[e] : 0.0;
    }
  }
  if (part == 0)
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) {
      const int tile = group + t * Shape::kGroups;
      if (tile < Shape::kTiles)
        out[tile * 64 + lane] = f32x4_t{(float)sum[t][0], (float)sum[t][1], (float)sum[t][2], (float)sum[t][3]};
    }
}

// ---- iterate, in one CU ----
//
// Symmetric matrices as their lower tiles of 16 x 16 in LDS (G and P double, Q
// float), a tile or two a wave.  In double: see gram; products of float
// matrices would put noise of 2^-24 of the largest eigenvalue on the smallest,
// which grow by a^2 = 12 a step.
constexpr int kIterThreads = 1024;
constexpr int kTileD = 16 * 17;  // (rows padded: columns lie on distinct banks)

// Lane (i, g)'s A operand (row i, column 4 kk + g) of tile (ti, tk); B's is
// the same of the transposed matrix, which is the matrix.
template <class T>
__device__ __forceinline__ double sym_at(const T* m, int ti, int tk, int i, int k) {
  return ti >= tk ? (double)m[(ti * (ti + 1) / 2 + tk) * kTileD + i * 17 + k]
                  : (double)m[(tk * (tk + 1) / 2 + ti) * kTileD + k * 17 + i];
}

// The lower tile (ti, tj) of A B.
template <int NT, class TA, class TB>
__device__ __forceinline__ f64x4_t sym_product(const TA* A, const TB* B, int ti, int tj, int i, int g) {
  f64x4_t acc{0, 0, 0, 0};
#pragma unroll
  for (int tk = 0; tk < NT; ++tk)
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      acc = mfma_f64(sym_at(A, ti, tk, i, 4 * kk + g), sym_at(B, tj, tk, i, 4 * kk + g), acc);
  return acc;
}

template <int NT>
__global__ __launch_bounds__(kIterThreads) void muon_iterate_kernel(MuonArgs a, int32_t m0) {
  constexpr int kTiles = muon_lower(NT), kWaves = kIterThreads / 64, kPer = (kTiles + kWaves - 1) / kWaves;
  extern __shared__ __attribute__((aligned(16))) double lds_d[];
  double* G = lds_d;                                         // [kTiles][kTileD]
  double* P = G + kTiles * kTileD;
  float* Q = reinterpret_cast<float*>(P + kTiles * kTileD);  // [kTiles][kTileD]
  __shared__ double trace;
  const MuonMatrix& M = a.matrices[m0 + blockIdx.x];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int chunks = M.chunks;
  // sums of the pieces; a piece's tile holds rows 4g + e of column i by lane
  for (int q = tid; q < kTiles * 64; q += kIterThreads) {
    const f32x4_t* at = reinterpret_cast<const f32x4_t*>(M.parts) + q;
    double v[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
      const f32x4_t x = at[(int64_t)c * kTiles * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += (double)x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) G[(q >> 6) * kTileD + (4 * ((q & 63) >> 4) + e) * 17 + (q & 15)] = v[e];
  }
  __syncthreads();
  if (wave == 0) {
    double v = 0;
    for (int r = lane; r < 16 * NT; r += 64) v += G[((r >> 4) * ((r >> 4) + 1) / 2 + (r >> 4)) * kTileD + (r & 15) * 18];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    if (lane == 0) trace = v;
  }
  __syncthreads();
  const double inv = 1.0 / (sqrt(trace) + a.eps);
  for (int q = tid; q < kTiles * 256; q += kIterThreads) {
    double* t = G + (q >> 8) * kTileD;
    t[((q >> 4) & 15) * 17 + (q & 15)] *= inv * inv;
  }
  int ti[kPer], tj[kPer];
  bool live[kPer];
#pragma unroll
  for (int t = 0; t < kPer; ++t) {
    live[t] = wave + t * kWaves < kTiles;
    lower_tile(min(wave + t * kWaves, kTiles - 1), &ti[t], &tj[t]);
  }
  __syncthreads();
  const auto at = [&](int t, int e) { return (wave + t * kWaves) * kTileD + (4 * e + g) * 17 + i; };
  for (int step = 0; step < a.steps; ++step) {
    const bool last = step == a.steps - 1;
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      if (!live[t]) continue;
      const f64x4_t h = sym_product<NT>(G, G, ti[t], tj[t], i, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double p = a.b * G[at(t, e)] + a.c * h[e] + (ti[t] == tj[t] && 4 * e + g == i ? a.a : 0.0);
        P[at(t, e)] = p;
        if (step == 0) Q[at(t, e)] = (float)p;
      }
    }
    __syncthreads();
    f64x4_t w[kPer], q[kPer];
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      if (!live[t]) continue;
      if (step > 0) q[t] = sym_product<NT>(P, Q, ti[t], tj[t], i, g);
      if (!last) w[t] = sym_product<NT>(P, G, ti[t], tj[t], i, g);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      if (!live[t]) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (step > 0) Q[at(t, e)] = (float)q[t][e];
        if (!last) G[at(t, e)] = w[t][e];
      }
    }
    __syncthreads();
    if (last) break;
#pragma unroll
    for (int t = 0; t < kPer; ++t)
      if (live[t]) w[t] = sym_product<NT>(P, G, ti[t], tj[t], i, g);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kPer; ++t)
      if (live[t])
#pragma unroll
        for (int e = 0; e < 4; ++e) G[at(t, e)] = w[t][e];
    __syncthreads();
  }
  constexpr int S = 16 * NT;
  for (int q = tid; q < S * S; q += kIterThreads) {
    const int r = q / S, c = q % S, hi = max(r, c), lo = min(r, c);
    M.q[q] = (float)((double)Q[((hi >> 4) * ((hi >> 4) + 1) / 2 + (lo >> 4)) * kTileD + (hi & 15) * 17 + (lo & 15)] * inv);
  }
}

// ---- iterate, larger matrices: one launch a product ----
//
// [S][S] doubles in memory, 32 x 32 of a product a workgroup (the lower
// blocks, mirrored), both operands read along their rows.
struct MuonProduct {
  // out = scale^x left right (+ ...) : which of the matrix's five
  int left, right, out;
  bool poly;      // out = a I + b left + c left right
  int first;      // left and right are not scaled yet: poly: both; else: right
  bool final;     // to M.q, times 1 / (|u| + eps)
};

template <int NT>
__global__ __launch_bounds__(256) void muon_sum_kernel(MuonArgs a, int32_t m0) {
  constexpr int kTiles = muon_lower(NT), S = 16 * NT;
  const MuonMatrix& M = a.matrices[m0 + blockIdx.y];
  const int q = blockIdx.x * 256 + threadIdx.x, tile = q >> 6;
  if (tile >= kTiles) return;
  const f32x4_t* at = reinterpret_cast<const f32x4_t*>(M.parts) + q;
  double v[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int c = 0; c < M.chunks; ++c) {
    const f32x4_t x = at[(int64_t)c * kTiles * 64];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += (double)x[e];
  }
  int ti, tj;
  lower_tile(tile, &ti, &tj);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 16 * ti + 4 * ((q & 63) >> 4) + e, c = 16 * tj + (q & 15);
    if (r < c) continue;  // (above the diagonal of a diagonal tile)
    M.work[r * S + c] = M.work[c * S + r] = v[e];
  }
}

template <int NT>
__global__ __launch_bounds__(256) void muon_product_kernel(MuonArgs a, int32_t m0, MuonProduct x, MuonProduct y) {
  constexpr int S = 16 * NT, kSide = S / 32;
  const MuonMatrix& M = a.matrices[m0 + blockIdx.y];
  const MuonProduct j = blockIdx.z ? y : x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  double inv = 1.0;
  if (j.first || j.final) {
    // (the trace of the first matrix of the five, which stays)
    double v = 0;
    for (int r = lane; r < S; r += 64) v += M.work[r * (S + 1)];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    inv = 1.0 / (sqrt(v) + a.eps);
  }
  int bi, bj;
  lower_tile(blockIdx.x, &bi, &bj);
  static_assert(kSide * 32 == S, "whole blocks");
  const int r0 = 32 * bi + 16 * (wave >> 1), c0 = 32 * bj + 16 * (wave & 1);
  const double* A = M.work + (size_t)j.left * S * S + (r0 + i) * S + 2 * g;
  const double* B = M.work + (size_t)j.right * S * S + (c0 + i) * S + 2 * g;
  f64x4_t acc{0, 0, 0, 0};
#pragma unroll 8
  for (int k = 0; k < S; k += 8) {
    const f64x2_t u = *reinterpret_cast<const f64x2_t*>(A + k), v = *reinterpret_cast<const f64x2_t*>(B + k);
    acc = mfma_f64(u.x, v.x, acc);
    acc = mfma_f64(u.y, v.y, acc);
  }
  const double i2 = inv * inv;
  double* out = M.work + (size_t)j.out * S * S;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = r0 + 4 * e + g, c = c0 + i;
    double v = acc[e];
    if (j.poly) {
      const double l = M.work[(size_t)j.left * S * S + r * S + c];
      v = j.first ? a.b * l * i2 + a.c * v * i2 * i2 : a.b * l + a.c * v;
      v += r == c ? a.a : 0.0;
    } else if (j.first) {
      v *= i2;
    }
    if (bi == bj && r < c) continue;
    if (j.final) {
      M.q[r * S + c] = M.q[c * S + r] = (float)(v * inv);
    } else {
      out[r * S + c] = out[c * S + r] = v;
    }
  }
}

// Q of a single step: P itself, scaled.
template <int NT>
__global__ __launch_bounds__(256) void muon_single_kernel(MuonArgs a, int32_t m0) {
  constexpr int S = 16 * NT;
  const MuonMatrix& M = a.matrices[m0 + blockIdx.y];
  double v = 0;
  for (int r = threadIdx.x & 63; r < S; r += 64) v += M.work[r * (S + 1)];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  const double inv = 1.0 / (sqrt(v) + a.eps);
  const int q = blockIdx.x * 256 + threadIdx.x;
  M.q[q] = (float)(M.work[(size_t)S * S + q] * inv);
}

// ---- apply ----
//
// Wave w holds row tile w % NT of Q in registers and takes its share of the
// stage's 16-column tiles; Q u goes through LDS to the threads that hold the
// parameters.
template <int NT>
struct ApplyShape {
  static constexpr int kWaves = NT <= 2 || NT == 4 ? 8 : NT == 3 ? 6 : NT == 5 ? 10 : NT;
  static constexpr int kCols = kWaves / NT;  // waves of a row tile
};

template <int NT>
__global__ __launch_bounds__(ApplyShape<NT>::kWaves * 64) void muon_apply_kernel(MuonArgs a, int64_t c0) {
  constexpr int KB = muon_stage(NT), KP = Stage<KB>::KP, S = 16 * NT;
  using Shape = ApplyShape<NT>;
  constexpr int kThreads = Shape::kWaves * 64, kNq = (S * KB / 4 + kThreads - 1) / kThreads;
  extern __shared__ __attribute__((aligned(16))) float lds[];  // u, then Q u: [S][KP] each
  float* res = lds + S * KP;
  const MuonChunk ch = a.chunks[c0 + blockIdx.x];
  const MuonMatrix& M = a.matrices[ch.matrix];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4, tile = wave % NT;
  const Stage<KB> st{M.s, M.L, M.wide != 0};
  const int64_t k0 = (int64_t)ch.part * M.chunk, k1 = min(M.L, k0 + M.chunk);
  const float gs = a.dyn ? a.dyn[1] : a.grad_scale, lr = a.dyn ? a.dyn[0] : a.lr;
  const float decay = 1.f - lr * a.weight_decay, rate = lr * M.lr_scale;
  const void* grad = M.g;
  const float* mom = M.m;
  void* param = M.p;
  float* master = M.master;
  const int n_groups = st.groups();
  for (int q = tid; q < S * KP; q += kThreads) lds[q] = 0.f;
  float qa[S / 4];  // Q[16 tile + i][4 kk + g]
#pragma unroll
  for (int kk = 0; kk < S / 4; ++kk) qa[kk] = M.q[(16 * tile + i) * S + 4 * kk + g];
  f32x4_t vg[kNq], vm[kNq], vp[kNq];
  const auto load = [&](int64_t k) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int x = tid + q * kThreads;
      int64_t at = 0;
      int n = 0;
      if (x < n_groups) st.locate(x, k, k1, &at, &n);
      if (a.nesterov) vg[q] = load4(grad, a.g_f32, at, n);
      vm[q] = load4(mom, true, at, n);
    }
  };
  load(k0);
  for (int64_t k = k0; k < k1; k += KB) {
    if (k == k0) __syncthreads();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int x = tid + q * kThreads;
      if (x < n_groups) st.put(lds, x, a.nesterov ? vg[q] * gs + a.momentum * vm[q] : vm[q]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int x = tid + q * kThreads;
      int64_t at = 0;
      int n = 0;
      if (x < n_groups) st.locate(x, k, k1, &at, &n);
      vp[q] = a.master ? load4(master, true, at, n) : load4(param, a.p_f32, at, n);
    }
    if (k + KB < k1) load(k + KB);
    for (int c = wave / NT; c < KB / 16; c += Shape::kCols) {
      f32x4_t acc = zero4();
#pragma unroll
      for (int kk = 0; kk < S / 4; ++kk) acc = mfma_f32(qa[kk], lds[(4 * kk + g) * KP + 16 * c + i], acc);
#pragma unroll
      for (int e = 0; e < 4; ++e) res[(16 * tile + 4 * g + e) * KP + 16 * c + i] = acc[e];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int x = tid + q * kThreads;
      if (x >= n_groups) continue;
      int64_t at;
      int n;
      st.locate(x, k, k1, &at, &n);
      if (n == 0) continue;
      const f32x4_t p = vp[q] * decay - rate * st.get(res, x);
      if (a.master) store4(master, true, at, n, p);
      store4(param, a.p_f32, at, n, p);
    }
  }
}

template <int NT>
hipError_t launch_class(const MuonArgs& a, int32_t m0, int32_t n, int64_t c0, int64_t chunks, hipStream_t s) {
  constexpr int KB = muon_stage(NT), S = 16 * NT;
  constexpr size_t kStage = (size_t)S * Stage<KB>::KP * 4;
  using Shape = GramShape<NT>;
  static_assert(Shape::kParts == 1 || kStage >= (size_t)Shape::kGroups * 64 * 4 * 8, "the parts' sums fit the stage");
  hipLaunchKernelGGL(muon_gram_kernel<NT>, dim3((unsigned)chunks), dim3(kGramThreads), kStage, s, a, c0);
  if constexpr (NT <= kMuonTiles[kMuonLdsClasses - 1]) {
    constexpr size_t kLds = (size_t)muon_lower(NT) * kTileD * (8 + 8 + 4);
    hipLaunchKernelGGL(muon_iterate_kernel<NT>, dim3((unsigned)n), dim3(kIterThreads), kLds, s, a, m0);
  } else {
    const dim3 tiles((unsigned)((muon_lower(NT) + 3) / 4), (unsigned)n);
    hipLaunchKernelGGL(muon_sum_kernel<NT>, tiles, dim3(256), 0, s, a, m0);
    // of the five: 0 the first product (which stays), 1 and 2 Q in turn, 3 P, 4 W; A_1 and on: in 5
    const unsigned blocks = (unsigned)muon_lower(S / 32);
    const auto product = [&](MuonProduct x, MuonProduct y, int jobs) {
      hipLaunchKernelGGL(muon_product_kernel<NT>, dim3(blocks, (unsigned)n, (unsigned)jobs), dim3(256), 0, s, a, m0, x,
                         y);
    };
    int q = 1, A = 0;
    for (int step = 0; step < a.steps; ++step) {
      const bool first = step == 0, last = step == a.steps - 1;
      const int P = first ? 1 : 3;
      product({A, A, P, true, first, false}, {}, 1);
      const MuonProduct w{P, A, 4, false, first, false}, qn{P, q, 3 - q, false, 0, last};
      if (first && last) {
        hipLaunchKernelGGL(muon_single_kernel<NT>, dim3(S * S / 256, (unsigned)n), dim3(256), 0, s, a, m0);
      } else if (first) {
        product(w, {}, 1);
      } else if (last) {
        product(qn, {}, 1);
      } else {
        product(w, qn, 2);
        q = 3 - q;
      }
      if (!last) {
        product({P, 4, 5, false, 0, false}, {}, 1);
        A = 5;
      }
    }
  }
  hipLaunchKernelGGL(muon_apply_kernel<NT>, dim3((unsigned)chunks), dim3(ApplyShape<NT>::kWaves * 64), 2 * kStage, s, a,
                     c0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon(const MuonArgs& a, int cls, int32_t m0, int32_t n_matrices, int64_t c0, int64_t n_chunks,
                       hipStream_t s) {
  switch (kMuonTiles[cls]) {
#define SALR_MUON_CASE(nt) \
  case nt: return launch_class<nt>(a, m0, n_matrices, c0, n_chunks, s);
    SALR_MUON_CASE(1)
    SALR_MUON_CASE(2)
    SALR_MUON_CASE(3)
    SALR_MUON_CASE(4)
    SALR_MUON_CASE(5)
    SALR_MUON_CASE(6)
    SALR_MUON_CASE(7)
    SALR_MUON_CASE(8)
    SALR_MUON_CASE(10)
    SALR_MUON_CASE(12)
    default: return launch_class<16>(a, m0, n_matrices, c0, n_chunks, s);
#undef SALR_MUON_CASE
  }
}

}  // namespace salr

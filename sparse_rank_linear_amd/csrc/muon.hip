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

// A stage: KB columns of the long side from k on (those before k1), in groups
// of four elements that lie together in memory: of a wide matrix along its rows
// (the long side), of a tall one along the flat array.  In LDS a wide matrix's
// stage is [short][PW], a tall one's [long][PT]: whole groups either way (but
// where a tall matrix's rows are no multiple of four, whose groups run over
// their ends).  Thread t takes groups t, t + THREADS, ...
template <bool WIDE, int KB, int THREADS, int NQ, int PITCH>
struct Stage {
  int s, tid;
  int64_t L;
  __device__ __forceinline__ int group(int q) const { return tid + q * THREADS; }
  __device__ __forceinline__ bool has(int q) const { return group(q) < s * (KB / 4); }
  // group q of the stage from k on: its first element in the matrix, and how many of it there are
  __device__ __forceinline__ int64_t element(int q, int64_t k) const {
    const int x = group(q);
    return WIDE ? (int64_t)(x / (KB / 4)) * L + k + x % (KB / 4) * 4 : k * s + 4 * x;
  }
  __device__ __forceinline__ int count(int q, int left) const {  // left: columns from k to k1
    const int x = group(q);
    if (!has(q)) return 0;
    if (left >= KB) return 4;
    return max(0, min(4, WIDE ? left - x % (KB / 4) * 4 : left * s - 4 * x));
  }
  __device__ __forceinline__ int place(int q) const {
    const int x = group(q);
    return WIDE ? x / (KB / 4) * PITCH + x % (KB / 4) * 4 : 4 * x / s * PITCH + 4 * x % s;
  }
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

// ---- gram ----
//
// 8 or 16 waves; kGroups of them share the lower tiles of u u^T, and kParts
// such groups take every kParts-th 16 columns of a stage.  A stage's sum (KB columns at most) is float,
// then joins a double: the smallest eigenvalues decide how fast their
// directions grow, and a float sum over thousands of columns would drown them.
template <int NT>
struct GramShape {
  static constexpr int KB = muon_stage(NT), S = 16 * NT;
  static constexpr int kTiles = muon_lower(NT);
  static constexpr int kWaves = NT <= 8 ? 8 : 16;
  static constexpr int kGroups = NT <= 3 ? 1 : NT == 4 ? 4 : kWaves;
  static constexpr int kParts = kWaves / kGroups;
  static constexpr int kPer = (kTiles + kGroups - 1) / kGroups;  // tiles of a wave
  // (wide: 16 rows' 16-byte reads on all banks; tall: 4 rows of 16 values on all banks)
  static constexpr int PW = KB + 4, PT = S % 32 == 16 ? S : S + 16;
  static constexpr int kFloats = S * PW > KB * PT ? S * PW : KB * PT;
};

__device__ __forceinline__ void lower_tile(int t, int* ti, int* tj) {
  int i = 0;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  *ti = i;
  *tj = t - i * (i + 1) / 2;
}

template <int NT, bool WIDE>
__device__ __forceinline__ void gram(const MuonArgs& a, const MuonMatrix& M, int piece, float* lds) {
  using Shape = GramShape<NT>;
  constexpr int KB = Shape::KB, S = Shape::S, P = WIDE ? Shape::PW : Shape::PT, kThreads = 64 * Shape::kWaves;
  constexpr int kNq = (S * KB / 4 + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const Stage<WIDE, KB, kThreads, kNq, P> st{M.s, tid, M.L};
  const int64_t k0 = (int64_t)piece * M.chunk, k1 = min(M.L, k0 + M.chunk);
  const float gs = a.dyn ? a.dyn[1] : a.grad_scale;
  const void* grad = M.g;
  float* mom = M.m;
  float* parts = M.parts;
  for (int q = tid; q < Shape::kFloats; q += kThreads) lds[q] = 0.f;  // (past the short side it stays so)
  const int group = wave % Shape::kGroups, part = wave / Shape::kGroups;
  f64x4_t sum[Shape::kPer];
  int row_i[Shape::kPer], row_j[Shape::kPer], place[kNq];
#pragma unroll
  for (int t = 0; t < Shape::kPer; ++t) {
    sum[t] = f64x4_t{0, 0, 0, 0};
    int ti, tj;
    lower_tile(min(group + t * Shape::kGroups, Shape::kTiles - 1), &ti, &tj);
    row_i[t] = WIDE ? (16 * ti + i) * P + 4 * g : g * P + 16 * ti + i;
    row_j[t] = WIDE ? (16 * tj + i) * P + 4 * g : g * P + 16 * tj + i;
  }
#pragma unroll
  for (int q = 0; q < kNq; ++q) place[q] = st.place(q);
  f32x4_t vg[kNq], vm[kNq];
  const auto load = [&](int64_t k) __attribute__((always_inline)) {
    const int left = (int)(k1 - k);
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int n = st.count(q, left);
      const int64_t at = n > 0 ? st.element(q, k) : 0;
      vg[q] = load4(grad, a.g_f32, at, n);
      vm[q] = load4(mom, true, at, n);
    }
  };
  load(k0);
  for (int64_t k = k0; k < k1; k += KB) {
    const int left = (int)(k1 - k);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      if (!st.has(q)) continue;
      const int n = st.count(q, left);
      const f32x4_t gg = vg[q] * gs, mm = a.momentum * vm[q] + gg;
      if (n > 0) store4(mom, true, st.element(q, k), n, mm);
      st.put(lds, place[q], a.nesterov ? gg + a.momentum * mm : mm);
    }
    __syncthreads();
    if (k + KB < k1) load(k + KB);
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) {
      f32x4_t acc = zero4();
#pragma unroll
      for (int c = 0; c < KB / 16 / Shape::kParts; ++c) {
        const int col = 16 * (part + c * Shape::kParts);
        // (which column of the sixteen is whose does not matter)
        f32x4_t x, y;
        if constexpr (WIDE) {
          x = *reinterpret_cast<const f32x4_t*>(lds + row_i[t] + col);
          y = *reinterpret_cast<const f32x4_t*>(lds + row_j[t] + col);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = lds[row_i[t] + (col + 4 * e) * P];
            y[e] = lds[row_j[t] + (col + 4 * e) * P];
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma_f32(x[e], y[e], acc);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[t][e] += (double)acc[e];
    }
  }
  // the column parts meet in LDS, in order
  f32x4_t* out = reinterpret_cast<f32x4_t*>(parts + (int64_t)piece * Shape::kTiles * 256);
  double* at = reinterpret_cast<double*>(lds) + (group * 64 + lane) * 4;
  for (int q = Shape::kParts - 1; q > 0; --q) {
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) {
      __syncthreads();
      if (part == q)
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e] = sum[t][e];
      __syncthreads();
      if (part == q - 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[t][e] += at[e];
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

template <int NT>
__global__ __launch_bounds__(GramShape<NT>::kWaves * 64) void muon_gram_kernel(MuonArgs a, int64_t c0) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const MuonChunk ch = a.chunks[c0 + blockIdx.x];
  const MuonMatrix& M = a.matrices[ch.matrix];
  if (M.wide) gram<NT, true>(a, M, ch.part, lds);
  else gram<NT, false>(a, M, ch.part, lds);
}

// ---- iterate, in one CU ----
//
// Symmetric matrices as their lower tiles of 16 x 16 in LDS, a tile or two a
// wave.  The first kMuonDouble steps in double (see gram): products of float
// matrices put noise of 2^-24 of the largest eigenvalue on the smallest ones,
// which grow by a^2 = 12 a step, so what the later steps add counts for 144
// times less.  Q is float throughout.
constexpr int kTileP = 17, kTileD = 16 * kTileP;  // (rows padded: columns lie on distinct banks)
constexpr int kMuonDouble = 2;

template <class T>
struct Acc;
template <>
struct Acc<double> {
  typedef f64x4_t type;
  static __device__ __forceinline__ type mul(double x, double y, type c) { return mfma_f64(x, y, c); }
  static __device__ __forceinline__ int row(int e, int g) { return 4 * e + g; }
};
template <>
struct Acc<float> {
  typedef f32x4_t type;
  static __device__ __forceinline__ type mul(float x, float y, type c) { return mfma_f32(x, y, c); }
  static __device__ __forceinline__ int row(int e, int g) { return 4 * g + e; }
};

// Where lane (i, g) finds its operands (row i, columns 4 kk + g) of tile (t,
// tk): first + kk * step.  Both operands of a product are read like this (B's
// is a row of the transposed matrix, which is the matrix), from the stored
// tile (tk, t) by columns where t < tk.
struct Operand {
  int first, step;
};
__device__ __forceinline__ Operand operand(int t, int tk, int i, int g) {
  const bool low = t >= tk;
  const int hi = low ? t : tk, lo = low ? tk : t;
  return {(hi * (hi + 1) / 2 + lo) * kTileD + (low ? i * kTileP + g : g * kTileP + i), low ? 4 : 4 * kTileP};
}

template <int NT>
struct IterShape {
  static constexpr int kTiles = muon_lower(NT), kWaves = NT <= 5 ? 16 : 8, kThreads = 64 * kWaves;
  static constexpr int kPer = (kTiles + kWaves - 1) / kWaves;
};

// A wave's lower tiles (ti, tj) of A B, the products of type T.  (A wave with
// fewer tiles computes its last one again: nothing reads it.)
template <int NT, class T, class TA, class TB>
__device__ __forceinline__ void sym_products(const TA* A, const TB* B, const int (&ti)[IterShape<NT>::kPer],
                                             const int (&tj)[IterShape<NT>::kPer], int i, int g,
                                             typename Acc<T>::type (&acc)[IterShape<NT>::kPer]) {
  constexpr int kPer = IterShape<NT>::kPer;
#pragma unroll
  for (int t = 0; t < kPer; ++t) acc[t] = typename Acc<T>::type{0, 0, 0, 0};
  constexpr int kUnroll = kPer == 1 ? NT : 1;  // (several tiles are enough to overlap; more does not fit the registers)
#pragma unroll kUnroll
  for (int tk = 0; tk < NT; ++tk) {
    T u[kPer][4], v[kPer][4];
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      const Operand x = operand(ti[t], tk, i, g), y = operand(tj[t], tk, i, g);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        u[t][kk] = (T)A[x.first + kk * x.step];
        v[t][kk] = (T)B[y.first + kk * y.step];
      }
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int t = 0; t < kPer; ++t) acc[t] = Acc<T>::mul(u[t][kk], v[t][kk], acc[t]);
  }
}

// One step on G (of type T, TN after it), P and Q.
template <int NT, class T, class TN>
__device__ __forceinline__ void iterate_step(const MuonArgs& a, double* Gd, double* Pd, float* Q, bool first, bool last,
                                             const int (&ti)[IterShape<NT>::kPer], const int (&tj)[IterShape<NT>::kPer],
                                             const bool (&live)[IterShape<NT>::kPer], int wave, int i, int g) {
  constexpr int kPer = IterShape<NT>::kPer, kWaves = IterShape<NT>::kWaves;
  T* G = reinterpret_cast<T*>(Gd);
  T* P = reinterpret_cast<T*>(Pd);
  const auto at = [&](int t, int row) { return (wave + t * kWaves) * kTileD + row * kTileP + i; };
  const T ca = (T)a.a, cb = (T)a.b, cc = (T)a.c;
  typename Acc<T>::type w[kPer];
  f32x4_t q[kPer];
  sym_products<NT, T>(G, G, ti, tj, i, g, w);
#pragma unroll
  for (int t = 0; t < kPer; ++t) {
    if (!live[t]) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = Acc<T>::row(e, g);
      const T p = cb * G[at(t, row)] + cc * w[t][e] + (ti[t] == tj[t] && row == i ? ca : (T)0);
      P[at(t, row)] = p;
      if (first) Q[at(t, row)] = (float)p;
    }
  }
  __syncthreads();
  if (!first) sym_products<NT, float>(P, Q, ti, tj, i, g, q);
  if (!last) sym_products<NT, T>(P, G, ti, tj, i, g, w);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kPer; ++t) {
    if (!live[t]) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!first) Q[at(t, Acc<float>::row(e, g))] = q[t][e];
      if (!last) G[at(t, Acc<T>::row(e, g))] = w[t][e];
    }
  }
  __syncthreads();
  if (last) return;
  sym_products<NT, T>(P, G, ti, tj, i, g, w);
  __syncthreads();
  TN* next = reinterpret_cast<TN*>(Gd);
#pragma unroll
  for (int t = 0; t < kPer; ++t)
    if (live[t])
#pragma unroll
      for (int e = 0; e < 4; ++e) next[at(t, Acc<T>::row(e, g))] = (TN)w[t][e];
  __syncthreads();
}

template <int NT>
__global__ __launch_bounds__(IterShape<NT>::kThreads) void muon_iterate_kernel(MuonArgs a, int32_t m0) {
  using Shape = IterShape<NT>;
  constexpr int kTiles = Shape::kTiles, kPer = Shape::kPer, kIterThreads = Shape::kThreads;
  extern __shared__ __attribute__((aligned(16))) double lds_d[];
  double* G = lds_d;                                         // [kTiles][kTileD]
  double* P = G + kTiles * kTileD;
  float* Q = reinterpret_cast<float*>(P + kTiles * kTileD);  // [kTiles][kTileD]
  __shared__ double trace;
  const MuonMatrix& M = a.matrices[m0 + blockIdx.x];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int chunks = M.chunks;
  float* out = M.q;
  // sums of the pieces; a piece's tile holds rows 4g + e of column i by lane
  for (int q = tid; q < kTiles * 64; q += kIterThreads) {
    const f32x4_t* at = reinterpret_cast<const f32x4_t*>(M.parts) + q;
    double v[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
      const f32x4_t x = at[(int64_t)c * kTiles * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += (double)x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) G[(q >> 6) * kTileD + (4 * ((q & 63) >> 4) + e) * kTileP + (q & 15)] = v[e];
  }
  __syncthreads();
  if (wave == 0) {
    double v = 0;
    for (int r = lane; r < 16 * NT; r += 64)
      v += G[((r >> 4) * ((r >> 4) + 1) / 2 + (r >> 4)) * kTileD + (r & 15) * (kTileP + 1)];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    if (lane == 0) trace = v;
  }
  __syncthreads();
  const double inv = 1.0 / (sqrt(trace) + a.eps);
  for (int q = tid; q < kTiles * 256; q += kIterThreads)
    G[(q >> 8) * kTileD + ((q >> 4) & 15) * kTileP + (q & 15)] *= inv * inv;
  int ti[kPer], tj[kPer];
  bool live[kPer];
#pragma unroll
  for (int t = 0; t < kPer; ++t) {
    live[t] = wave + t * Shape::kWaves < kTiles;
    lower_tile(min(wave + t * Shape::kWaves, kTiles - 1), &ti[t], &tj[t]);
  }
  __syncthreads();
  static_assert(kMuonDouble == 2, "the steps below");
  iterate_step<NT, double, double>(a, G, P, Q, true, a.steps == 1, ti, tj, live, wave, i, g);
  if (a.steps > 1) iterate_step<NT, double, float>(a, G, P, Q, false, a.steps == 2, ti, tj, live, wave, i, g);
  for (int step = 2; step < a.steps; ++step)
    iterate_step<NT, float, float>(a, G, P, Q, false, step == a.steps - 1, ti, tj, live, wave, i, g);
  constexpr int S = 16 * NT;
  for (int q = tid; q < S * S; q += kIterThreads) {
    const int r = q / S, c = q % S, hi = max(r, c), lo = min(r, c);
    out[q] =
        (float)((double)Q[((hi >> 4) * ((hi >> 4) + 1) / 2 + (lo >> 4)) * kTileD + (hi & 15) * kTileP + (lo & 15)] * inv);
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

constexpr int kProductThreads = 1024;
template <int NT>
__global__ __launch_bounds__(kProductThreads) void muon_product_kernel(MuonArgs a, int32_t m0, MuonProduct x,
                                                                       MuonProduct y) {
  constexpr int S = 16 * NT, kSplit = 4, kEach = S / kSplit;  // columns of a wave
  static_assert(S % 32 == 0, "whole blocks and operands");
  __shared__ f64x4_t part[kSplit - 1][4][64];
  const MuonMatrix& M = a.matrices[m0 + blockIdx.y];
  const MuonProduct j = blockIdx.z ? y : x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int tile = wave & 3, split = wave >> 2;
  double* work = M.work;
  int bi, bj;
  lower_tile(blockIdx.x, &bi, &bj);
  const int r0 = 32 * bi + 16 * (tile >> 1), c0 = 32 * bj + 16 * (tile & 1);
  const double* A = work + (size_t)j.left * S * S + (r0 + i) * S + 2 * g + split * kEach;
  const double* B = work + (size_t)j.right * S * S + (c0 + i) * S + 2 * g + split * kEach;
  f64x2_t u[kEach / 8], v[kEach / 8];
#pragma unroll
  for (int k = 0; k < kEach / 8; ++k) {
    u[k] = *reinterpret_cast<const f64x2_t*>(A + 8 * k);
    v[k] = *reinterpret_cast<const f64x2_t*>(B + 8 * k);
  }
  double inv = 1.0;
  if (j.first || j.final) {
    // (the trace of the first matrix of the six, which stays)
    double t = 0;
    for (int r = lane; r < S; r += 64) t += work[r * (S + 1)];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) t += __shfl_xor(t, d, 64);
    inv = 1.0 / (sqrt(t) + a.eps);
  }
  f64x4_t acc{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kEach / 8; ++k) {
    acc = mfma_f64(u[k].x, v[k].x, acc);
    acc = mfma_f64(u[k].y, v[k].y, acc);
  }
  if (split > 0) part[split - 1][tile][lane] = acc;
  __syncthreads();
  if (split > 0) return;
#pragma unroll
  for (int q = 0; q < kSplit - 1; ++q) acc += part[q][tile][lane];
  const double i2 = inv * inv;
  double* out = work + (size_t)j.out * S * S;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = r0 + 4 * e + g, c = c0 + i;
    double t = acc[e];
    if (j.poly) {
      const double l = work[(size_t)j.left * S * S + r * S + c];
      t = j.first ? a.b * l * i2 + a.c * t * i2 * i2 : a.b * l + a.c * t;
      t += r == c ? a.a : 0.0;
    } else if (j.first) {
      t *= i2;
    }
    if (bi == bj && r < c) continue;
    if (j.final) {
      M.q[r * S + c] = M.q[c * S + r] = (float)(t * inv);
    } else {
      out[r * S + c] = out[c * S + r] = t;
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
  static constexpr int KB = muon_stage(NT), S = 16 * NT;
  static constexpr int kWaves = NT <= 2 || NT == 4 ? 8 : NT == 3 ? 6 : NT == 5 ? 10 : NT;
  static constexpr int kCols = kWaves / NT;  // waves of a row tile
  // u's pitch and the result's: reads and writes that touch all banks
  static constexpr int PW = KB + 16, RW = KB + 4, PT = S + 4, RT = S + 4;
  static constexpr int kU = S * PW > KB * PT ? S * PW : KB * PT, kR = S * RW > KB * RT ? S * RW : KB * RT;
};

template <int NT, bool WIDE>
__device__ __forceinline__ void apply(const MuonArgs& a, const MuonMatrix& M, int piece, float* lds) {
  using Shape = ApplyShape<NT>;
  constexpr int KB = Shape::KB, S = Shape::S, P = WIDE ? Shape::PW : Shape::PT, R = WIDE ? Shape::RW : Shape::RT;
  constexpr int kThreads = Shape::kWaves * 64, kNq = (S * KB / 4 + kThreads - 1) / kThreads;
  float* res = lds + Shape::kU;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4, tile = wave % NT;
  const Stage<WIDE, KB, kThreads, kNq, P> st{M.s, tid, M.L};
  const Stage<WIDE, KB, kThreads, kNq, R> st_r{M.s, tid, M.L};
  const int64_t k0 = (int64_t)piece * M.chunk, k1 = min(M.L, k0 + M.chunk);
  const float gs = a.dyn ? a.dyn[1] : a.grad_scale, lr = a.dyn ? a.dyn[0] : a.lr;
  const float decay = 1.f - lr * a.weight_decay, rate = lr * M.lr_scale;
  const void* grad = M.g;
  const float* mom = M.m;
  void* param = M.p;
  float* master = M.master;
  // (parameters a stage ahead as well, where the registers hold them)
  constexpr bool kEarly = NT < 16;
  f32x4_t vg[kNq], vm[kNq], vp[kNq], next_p[kNq];
  const auto load = [&](int64_t k) __attribute__((always_inline)) {
    const int left = (int)(k1 - k);
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int n = st.count(q, left);
      const int64_t at = n > 0 ? st.element(q, k) : 0;
      if (a.nesterov) vg[q] = load4(grad, a.g_f32, at, n);
      vm[q] = load4(mom, true, at, n);
      if (kEarly) next_p[q] = a.master ? load4(master, true, at, n) : load4(param, a.p_f32, at, n);
    }
  };
  load(k0);
  // Q's rows, columns in the order that the operands of u come in
  float qa[S / 4];
#pragma unroll
  for (int kk = 0; kk < S / 4; ++kk)
    qa[kk] = M.q[(16 * tile + i) * S + (WIDE ? 4 * kk + g : 16 * (kk / 4) + 4 * g + kk % 4)];
  for (int q = tid; q < Shape::kU; q += kThreads) lds[q] = 0.f;
  int place[kNq], place_r[kNq];
#pragma unroll
  for (int q = 0; q < kNq; ++q) {
    place[q] = st.place(q);
    place_r[q] = st_r.place(q);
  }
  __syncthreads();
  for (int64_t k = k0; k < k1; k += KB) {
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      if (kEarly) vp[q] = next_p[q];
      if (st.has(q)) st.put(lds, place[q], a.nesterov ? vg[q] * gs + a.momentum * vm[q] : vm[q]);
    }
    __syncthreads();
    if (k + KB < k1) load(k + KB);
    for (int c = wave / NT; c < KB / 16; c += Shape::kCols) {
      f32x4_t acc = zero4();
      if constexpr (WIDE) {
        // (Q u)^T, four columns of the long side a lane
#pragma unroll
        for (int kk = 0; kk < S / 4; ++kk) acc = mfma_f32(lds[(4 * kk + g) * P + 16 * c + i], qa[kk], acc);
        *reinterpret_cast<f32x4_t*>(res + (16 * tile + i) * R + 16 * c + 4 * g) = acc;
      } else {
#pragma unroll
        for (int kk = 0; kk < S / 16; ++kk) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(lds + (16 * c + i) * P + 16 * kk + 4 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc = mfma_f32(qa[4 * kk + e], x[e], acc);
        }
        *reinterpret_cast<f32x4_t*>(res + (16 * c + i) * R + 16 * tile + 4 * g) = acc;
      }
    }
    const int left = (int)(k1 - k);
    if (!kEarly) {
#pragma unroll
      for (int q = 0; q < kNq; ++q) {
        const int n = st.count(q, left);
        const int64_t at = n > 0 ? st.element(q, k) : 0;
        vp[q] = a.master ? load4(master, true, at, n) : load4(param, a.p_f32, at, n);
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const int n = st.count(q, left);
      if (n == 0) continue;
      const int64_t at = st.element(q, k);
      const f32x4_t p = vp[q] * decay - rate * st_r.get(res, place_r[q]);
      if (a.master) store4(master, true, at, n, p);
      store4(param, a.p_f32, at, n, p);
    }
  }
}

template <int NT>
__global__ __launch_bounds__(ApplyShape<NT>::kWaves * 64, 4) void muon_apply_kernel(MuonArgs a, int64_t c0) {
  extern __shared__ __attribute__((aligned(16))) float lds[];  // u, then Q u
  const MuonChunk ch = a.chunks[c0 + blockIdx.x];
  const MuonMatrix& M = a.matrices[ch.matrix];
  if (M.wide) apply<NT, true>(a, M, ch.part, lds);
  else apply<NT, false>(a, M, ch.part, lds);
}

template <int NT>
hipError_t launch_class(const MuonArgs& a, int32_t m0, int32_t n, int64_t c0, int64_t chunks, hipStream_t s) {
  constexpr int S = 16 * NT;
  using Shape = GramShape<NT>;
  constexpr size_t kGram = (size_t)Shape::kFloats * 4, kApply = (size_t)(ApplyShape<NT>::kU + ApplyShape<NT>::kR) * 4;
  static_assert(Shape::kParts == 1 || kGram >= (size_t)Shape::kGroups * 64 * 4 * 8, "the parts' sums fit the stage");
  hipLaunchKernelGGL(muon_gram_kernel<NT>, dim3((unsigned)chunks), dim3(Shape::kWaves * 64), kGram, s, a, c0);
  if constexpr (NT <= kMuonTiles[kMuonLdsClasses - 1]) {
    constexpr size_t kLds = (size_t)muon_lower(NT) * kTileD * (8 + 8 + 4);
    hipLaunchKernelGGL(muon_iterate_kernel<NT>, dim3((unsigned)n), dim3(IterShape<NT>::kThreads), kLds, s, a, m0);
  } else {
    const dim3 tiles((unsigned)((muon_lower(NT) + 3) / 4), (unsigned)n);
    hipLaunchKernelGGL(muon_sum_kernel<NT>, tiles, dim3(256), 0, s, a, m0);
    // of the six: 0 the first product (which stays), 1 and 2 Q in turn, 3 P, 4 W; A_1 and on: in 5
    const unsigned blocks = (unsigned)muon_lower(S / 32);
    const auto product = [&](MuonProduct x, MuonProduct y, int jobs) {
      hipLaunchKernelGGL(muon_product_kernel<NT>, dim3(blocks, (unsigned)n, (unsigned)jobs), dim3(kProductThreads), 0, s, a, m0, x,
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
  hipLaunchKernelGGL(muon_apply_kernel<NT>, dim3((unsigned)chunks), dim3(ApplyShape<NT>::kWaves * 64), kApply, s, a,
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

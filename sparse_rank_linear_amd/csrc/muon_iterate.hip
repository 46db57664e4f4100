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
//   gram     (muon_gram.hip) m and u from the gradient, u u^T in pieces of
//            the long side
//   iterate  (here) the pieces' sum, the steps, Q
//   apply    (muon_apply.hpp) u again, Q u, the parameters
#include "muon_device.hpp"

namespace salr {
namespace {

// ---- iterate, in one CU ----
//
// Symmetric matrices as their lower tiles of 16 x 16 in LDS, a tile or two a
// wave.  The first kMuonDouble steps in double (see gram): products of float
// matrices put noise of 2^-24 of the largest eigenvalue on the smallest ones,
// which grow by a^2 = 12 a step, so what the later steps add counts for 1700
// times less (an 80 x 2048 update whose singular values differ 250-fold: X is
// 1.5e-5 off, after two such steps 5e-5, by float steps on X itself 4e-6; a step
// in float takes 6 us, in double 9.5).  Q is float throughout.  Bound by the
// chain of products of one matrix, each waiting for LDS: 53 us for rank 80,
// alone or one matrix a CU, of which nine products in double are 19 on the matrix
// cores and eight in float some 8; 159 for 128 matrices of rank 112.
constexpr int kTileP = 17, kTileD = 16 * kTileP;  // (rows padded: columns lie on distinct banks)
constexpr int kMuonDouble = 3;

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
  static constexpr int kWaves = NT == 1 ? 1 : NT == 2 ? 4 : NT == 3 ? 8 : NT == 7 ? 14 : 16;
  static constexpr int kTiles = muon_lower(NT), kThreads = 64 * kWaves;
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
  T u[2][kPer][4], v[2][kPer][4];
  const auto load = [&](int tk, T (&x)[kPer][4], T (&y)[kPer][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      const Operand p = operand(ti[t], tk, i, g), q = operand(tj[t], tk, i, g);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        x[t][kk] = (T)A[p.first + kk * p.step];
        y[t][kk] = (T)B[q.first + kk * q.step];
      }
    }
  };
  const auto multiply = [&](const T (&x)[kPer][4], const T (&y)[kPer][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int t = 0; t < kPer; ++t) acc[t] = Acc<T>::mul(x[t][kk], y[t][kk], acc[t]);
  };
  // The next tiles' operands are read while these are multiplied.
  load(0, u[0], v[0]);
  if constexpr (kPer == 1) {
#pragma unroll
    for (int tk = 0; tk < NT; ++tk) {
      if (tk + 1 < NT) load(tk + 1, u[(tk + 1) & 1], v[(tk + 1) & 1]);
      multiply(u[tk & 1], v[tk & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    // (unrolled, all addresses would be computed first, which the registers do not hold)
#pragma unroll 1
    for (int tk = 0; tk + 1 < NT; tk += 2) {
      load(tk + 1, u[1], v[1]);
      multiply(u[0], v[0]);
      __builtin_amdgcn_sched_barrier(0);
      load(min(tk + 2, NT - 1), u[0], v[0]);
      multiply(u[1], v[1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (NT % 2 == 1) multiply(u[0], v[0]);
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
  lds_barrier();
  if (!first) sym_products<NT, float>(P, Q, ti, tj, i, g, q);
  if (!last) sym_products<NT, T>(P, G, ti, tj, i, g, w);
  lds_barrier();
#pragma unroll
  for (int t = 0; t < kPer; ++t) {
    if (!live[t]) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!first) Q[at(t, Acc<float>::row(e, g))] = q[t][e];
      if (!last) G[at(t, Acc<T>::row(e, g))] = w[t][e];
    }
  }
  lds_barrier();
  if (last) return;
  sym_products<NT, T>(P, G, ti, tj, i, g, w);
  lds_barrier();
  TN* next = reinterpret_cast<TN*>(Gd);
#pragma unroll
  for (int t = 0; t < kPer; ++t)
    if (live[t])
#pragma unroll
      for (int e = 0; e < 4; ++e) next[at(t, Acc<T>::row(e, g))] = (TN)w[t][e];
  lds_barrier();
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
  const auto out = to_global<float>(M.q);
  const auto parts = to_global<const double>(M.parts);
  // sums of the pieces; a piece's tile holds rows 4g + e of column i by lane
  for (int q = tid; q < kTiles * 64; q += kIterThreads) {
    const auto at = (global<const f64x4_t>)parts + q;
    double v[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
      const f64x4_t x = at[(int64_t)c * kTiles * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) G[(q >> 6) * kTileD + (4 * ((q & 63) >> 4) + e) * kTileP + (q & 15)] = v[e];
  }
  lds_barrier();
  if (wave == 0) {
    double v = 0;
    for (int r = lane; r < 16 * NT; r += 64)
      v += G[((r >> 4) * ((r >> 4) + 1) / 2 + (r >> 4)) * kTileD + (r & 15) * (kTileP + 1)];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    if (lane == 0) trace = v;
  }
  lds_barrier();
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
  lds_barrier();
  for (int step = 0; step < min(kMuonDouble - 1, a.steps); ++step)
    iterate_step<NT, double, double>(a, G, P, Q, step == 0, step == a.steps - 1, ti, tj, live, wave, i, g);
  if (a.steps >= kMuonDouble)
    iterate_step<NT, double, float>(a, G, P, Q, false, a.steps == kMuonDouble, ti, tj, live, wave, i, g);
  for (int step = kMuonDouble; step < a.steps; ++step)
    iterate_step<NT, float, float>(a, G, P, Q, false, step == a.steps - 1, ti, tj, live, wave, i, g);
  constexpr int S = 16 * NT;
  for (int q = tid; q < S * S; q += kIterThreads) {
    const int r = q / S, c = q % S, hi = max(r, c), lo = min(r, c);
    const int tile = (hi >> 4) * ((hi >> 4) + 1) / 2 + (lo >> 4);
    out[q] = (float)((double)Q[tile * kTileD + (hi & 15) * kTileP + (lo & 15)] * inv);
  }
}

// ---- iterate, larger matrices: one launch a product ----
//
// [S][S] doubles in memory, 32 x 32 of a product a workgroup (the lower
// blocks, mirrored), both operands read along their rows.  (Eight tiles' lower
// halves in double take more than a CU's LDS.)  14 products for five steps, 12.4
// us each for six matrices of 256 x 256: a launch, a trip through the caches for
// operands that other dies wrote, 16 double products a wave one after another.
// Hundreds of matrices are bound by those trips: 380 of 256 x 256, 8.7 ms a step
// (256 x 411, bf16), of which a plain step in float takes 6.3.
struct MuonProduct {
  // out = left right: which of the matrix's six
  int left, right, out;
  bool poly;      // out = a I + b left + c left right
  int first;      // left and right are not scaled yet: poly: both; else: right
  bool final;     // to M.q, times 1 / (|u| + eps)
};

// The pieces' sum, both halves.  (Six matrices in 237 pieces of 278 KB: 66 MB in
// 12 us, most of them from the caches.)
template <int NT>
__global__ __launch_bounds__(256) void muon_sum_kernel(MuonArgs a, int32_t m0) {
  constexpr int kTiles = muon_lower(NT), S = 16 * NT;
  const MuonMatrix& M = a.matrices[m0 + blockIdx.y];
  const int q = blockIdx.x * 256 + threadIdx.x, tile = q >> 6;
  if (tile >= kTiles) return;
  const auto at = to_global<const f64x4_t>(M.parts) + q;
  const auto work = to_global<double>(M.work);
  double v[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int c = 0; c < M.chunks; ++c) {
    const f64x4_t x = at[(int64_t)c * kTiles * 64];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e];
  }
  int ti, tj;
  lower_tile(tile, &ti, &tj);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 16 * ti + 4 * ((q & 63) >> 4) + e, c = 16 * tj + (q & 15);
    if (r < c) continue;  // (above the diagonal of a diagonal tile)
    work[r * S + c] = work[c * S + r] = v[e];
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
  const auto work = to_global<double>(M.work);
  int bi, bj;
  lower_tile(blockIdx.x, &bi, &bj);
  const int r0 = 32 * bi + 16 * (tile >> 1), c0 = 32 * bj + 16 * (tile & 1);
  const auto A = work + (size_t)j.left * S * S + (r0 + i) * S + 2 * g + split * kEach;
  const auto B = work + (size_t)j.right * S * S + (c0 + i) * S + 2 * g + split * kEach;
  f64x2_t u[kEach / 8], v[kEach / 8];
#pragma unroll
  for (int k = 0; k < kEach / 8; ++k) {
    u[k] = *(global<const f64x2_t>)(A + 8 * k);
    v[k] = *(global<const f64x2_t>)(B + 8 * k);
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
  lds_barrier();
  if (split > 0) return;
#pragma unroll
  for (int q = 0; q < kSplit - 1; ++q) acc += part[q][tile][lane];
  const double i2 = inv * inv;
  const auto out = work + (size_t)j.out * S * S;
  const auto q_out = to_global<float>(M.q);
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
      q_out[r * S + c] = q_out[c * S + r] = (float)(t * inv);
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

template <int NT>
hipError_t launch_class(const MuonArgs& a, int32_t m0, int32_t n, hipStream_t s) {
  constexpr int S = 16 * NT;
  if constexpr (NT <= kMuonTiles[kMuonLdsClasses - 1]) {
    constexpr size_t kLds = (size_t)muon_lower(NT) * kTileD * (8 + 8 + 4);
    hipLaunchKernelGGL(muon_iterate_kernel<NT>, dim3((unsigned)n), dim3(IterShape<NT>::kThreads), kLds, s, a, m0);
  } else {
    const dim3 tiles((unsigned)((muon_lower(NT) + 3) / 4), (unsigned)n);
    hipLaunchKernelGGL(muon_sum_kernel<NT>, tiles, dim3(256), 0, s, a, m0);
    // of the six: 0 the first product (which stays), 1 and 2 Q in turn, 3 P, 4 W; A_1 and on: in 5
    const unsigned blocks = (unsigned)muon_lower(S / 32);
    const auto product = [&](MuonProduct x, MuonProduct y, int jobs) {
      hipLaunchKernelGGL(muon_product_kernel<NT>, dim3(blocks, (unsigned)n, (unsigned)jobs), dim3(kProductThreads), 0, s,
                         a, m0, x, y);
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
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon_iterate(const MuonArgs& a, int cls, int32_t m0, int32_t n_matrices, hipStream_t s) {
  return with_muon_tiles(cls, [&](auto nt) { return launch_class<decltype(nt)::value>(a, m0, n_matrices, s); });
}

}  // namespace salr

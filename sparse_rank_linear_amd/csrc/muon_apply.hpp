// The parameters' step with the orthogonalised update (see muon_iterate.hip for
// the method): one file for each kind of parameter includes this.
#pragma once

#include "muon_device.hpp"

namespace salr {
namespace {

// ---- apply ----
//
// Wave w holds row tile w % NT of Q in registers and takes its share of the
// stage's 16-column tiles; Q u goes through LDS to the threads that hold the
// parameters.  Bound by memory and the fp32 products one after the other, as
// the waves of a workgroup do the same at a time: 192 pairs of 80 x 2048 and 80
// x 1408, bf16 parameters and float gradients, 179 us (3.6 TB/s; the
// products are a quarter of it), 64 of 112 x 4096 and 112 x 14336 with masters
// 592 us (4.0 TB/s), three of 253 x 8191 and 253 x 14337 149 us (273 MB, 56 us,
// and 8.9 GFLOP, 58).  The forms of 3, 6, 7 and 16 tiles, and of 5 and 12 with
// masters (5 also floats with bf16 gradients), spill up to 27 registers under the
// bounds below.
// Stores past the caches, loads ahead by two stages and stores spread over the
// next stage's products were all slower.
template <int NT>
struct ApplyShape {
  static constexpr int KB = muon_stage(NT), S = 16 * NT;
  static constexpr int kWaves = NT <= 2 || NT == 4 ? 8 : NT == 3 ? 6 : NT == 5 ? 10 : NT;
  static constexpr int kCols = kWaves / NT;  // waves of a row tile
  // u's pitch and the result's: reads and writes that touch all banks
  static constexpr int PW = KB + 16, RW = KB + 4, PT = S + 4, RT = S + 4;
  static constexpr int kU = S * PW > KB * PT ? S * PW : KB * PT, kR = S * RW > KB * RT ? S * RW : KB * RT;
};

template <int NT, bool GF, bool PF, bool MASTER, bool WIDE>
__device__ __forceinline__ void apply(const MuonArgs& a, const MuonMatrix& M, int64_t k0, int64_t k1, float* lds) {
  using Shape = ApplyShape<NT>;
  constexpr int KB = Shape::KB, S = Shape::S, P = WIDE ? Shape::PW : Shape::PT, R = WIDE ? Shape::RW : Shape::RT;
  constexpr int kThreads = Shape::kWaves * 64, kNq = (S * KB / 4 + kThreads - 1) / kThreads;
  constexpr bool kSrc = PF || MASTER;  // what the step updates is float
  float* res = lds + Shape::kU;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4, tile = wave % NT;
  const Stage<WIDE, KB, kThreads, kNq> st(M.s, M.L, tid);
  const float gs = a.dyn ? a.dyn[1] : a.grad_scale, lr = a.dyn ? a.dyn[0] : a.lr;
  const float decay = 1.f - lr * a.weight_decay, rate = lr * M.lr_scale;
  const auto grad = to_global<const typename Four<GF>::elem>(M.g);
  const auto mom = to_global<const float>(M.m);
  const auto param = to_global<typename Four<PF>::elem>(M.p);
  const auto src = to_global<typename Four<kSrc>::elem>(MASTER ? (void*)M.master : M.p);
  const auto qm = to_global<const float>(M.q);
  // (parameters a stage ahead as well, where the registers hold them)
  constexpr bool kEarly = NT < 6;
  typename Four<GF>::raw vg[kNq];
  f32x4_t vm[kNq];
  typename Four<kSrc>::raw vp[kNq], next_p[kNq];
  const auto load = [&](int64_t k, auto full) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full)::value;
    const int left = (int)(k1 - k);
    if (a.nesterov) st.template load<FULL, GF>(grad, k, left, vg);
    st.template load<FULL, true>(mom, k, left, vm);
    if (kEarly) st.template load<FULL, kSrc>(src, k, left, next_p);
  };
  if (k0 + KB <= k1) load(k0, std::true_type{});
  // Q's rows, columns in the order that the operands of u come in
  float qa[S / 4];
#pragma unroll
  for (int kk = 0; kk < S / 4; ++kk)
    qa[kk] = qm[(16 * tile + i) * S + (WIDE ? 4 * kk + g : 16 * (kk / 4) + 4 * g + kk % 4)];
  for (int q = tid; q < Shape::kU; q += kThreads) lds[q] = 0.f;
  // (tall: both pitches are one, and the places take a division; wide: a shift)
  static_assert(WIDE || P == R, "one place");
  int tall_place[kNq];
#pragma unroll
  for (int q = 0; q < kNq; ++q) tall_place[q] = WIDE ? 0 : st.template place<P>(q);
  const auto place = [&](int q) { return WIDE ? st.template place<P>(q) : tall_place[q]; };
  const auto place_r = [&](int q) { return WIDE ? st.template place<R>(q) : tall_place[q]; };
  wait_memory();
  lds_barrier();
  const auto stage = [&](int64_t k, auto full) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full)::value;
    const int left = (int)(k1 - k);
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      if (kEarly) vp[q] = next_p[q];
      if (st.has(q))
        st.template put<P>(lds, place(q), a.nesterov ? Four<GF>::value(vg[q]) * gs + a.momentum * vm[q] : vm[q]);
    }
    lds_barrier();
    if (!kEarly) st.template load<FULL, kSrc>(src, k, left, vp);
    if (FULL && k + 2 * KB <= k1) load(k + KB, full);
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
    lds_barrier();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const f32x4_t p = Four<kSrc>::value(vp[q]) * decay - rate * st.template get<R>(res, place_r(q));
      if (MASTER) st.template store<FULL, true>(to_global<float>(M.master), q, k, left, p);
      st.template store<FULL, PF>(param, q, k, left, p);
    }
  };
  int64_t k = k0;
  for (; k + KB <= k1; k += KB) stage(k, std::true_type{});
  if (k < k1) {
    load(k, std::false_type{});
    stage(k, std::false_type{});
  }
}

template <int NT, bool GF, bool PF, bool MASTER>
__global__ __launch_bounds__(ApplyShape<NT>::kWaves * 64, NT == 3 || NT > 5 ? 4 : 5) void muon_apply_kernel(
    MuonArgs a, int64_t c0, int sub) {
  extern __shared__ __attribute__((aligned(16))) float lds[];  // u, then Q u
  const MuonChunk ch = a.chunks[c0 + blockIdx.x / sub];
  const MuonMatrix& M = a.matrices[ch.matrix];
  // (one of the chunk's `sub` parts, whole stages each)
  constexpr int KB = ApplyShape<NT>::KB;
  const int part = blockIdx.x % sub, each = (M.chunk / KB + sub - 1) / sub * KB;
  const int64_t k0 = (int64_t)ch.part * M.chunk + part * each;
  const int64_t k1 = min(min(M.L, (int64_t)(ch.part + 1) * M.chunk), k0 + each);
  if (k0 >= k1) return;
  if (M.wide) apply<NT, GF, PF, MASTER, true>(a, M, k0, k1, lds);
  else apply<NT, GF, PF, MASTER, false>(a, M, k0, k1, lds);
}

template <bool PF, bool MASTER>
hipError_t launch_apply(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s) {
  return with_muon_tiles(cls, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    using Shape = ApplyShape<NT>;
    constexpr size_t kLds = (size_t)(Shape::kU + Shape::kR) * 4;
    // (few chunks: their parts on workgroups of their own; 80 x 4096 and its
    // transpose: 13.7 us in 64 workgroups, 11 in 128)
    const int sub = chunks < 256 ? 2 : 1;
    const dim3 grid((unsigned)(chunks * sub)), threads(Shape::kWaves * 64);
    if (a.g_f32)
      hipLaunchKernelGGL((muon_apply_kernel<NT, true, PF, MASTER>), grid, threads, kLds, s, a, c0, sub);
    else
      hipLaunchKernelGGL((muon_apply_kernel<NT, false, PF, MASTER>), grid, threads, kLds, s, a, c0, sub);
    return hipGetLastError();
  });
}

}  // namespace
}  // namespace salr

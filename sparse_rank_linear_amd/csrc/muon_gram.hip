// The product of the update with itself, over the long side (see
// muon_iterate.hip for the method).
#include "muon_device.hpp"

namespace salr {
namespace {

// ---- gram ----
//
// 8 or 16 waves; kGroups of them share the lower tiles of u u^T, and kParts
// such groups take every kParts-th 16 columns of a stage.  Sixteen columns'
// sums are float, then join a double: the smallest eigenvalues decide how fast
// their directions grow, and longer float sums drown them (an 80 x 2048 update
// whose singular values differ 250-fold: X is 1.5e-5 off; summed in float over
// 64 columns 6e-5, and over all of them some 1e-3).  The next stage's loads are
// under way while one is multiplied.  Bound by memory (g and m read, m written)
// up to the ranks of ordinary adapters: 192 pairs of 80 x 2048 and 80 x 1408 in
// 120 us, 5.3 TB/s; 64 of 112 x 4096 and 112 x 14336 381 us, 4.2; above those by
// a CU's one workgroup, whose loads, LDS reads and products follow each other:
// three of 253 x 8191 and 253 x 14337 in 114 us (205 MB, 42 us, and 4.7 GFLOP, 31;
// 16 waves leave 128 registers a lane, and the 16 tiles' form spills 88: a wait
// for one of those waits for the loads that are to stay in flight too).
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

template <int NT, bool GF, bool WIDE>
__device__ __forceinline__ void gram(const MuonArgs& a, const MuonMatrix& M, int piece, float* lds) {
  using Shape = GramShape<NT>;
  constexpr int KB = Shape::KB, S = Shape::S, P = WIDE ? Shape::PW : Shape::PT, kThreads = 64 * Shape::kWaves;
  constexpr int kNq = (S * KB / 4 + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const Stage<WIDE, KB, kThreads, kNq> st(M.s, M.L, tid);
  const int64_t k0 = (int64_t)piece * M.chunk, k1 = min(M.L, k0 + M.chunk);
  const float gs = a.dyn ? a.dyn[1] : a.grad_scale;
  const auto grad = to_global<const typename Four<GF>::elem>(M.g);
  const auto mom = to_global<float>(M.m);
  const auto parts = to_global<double>(M.parts);
  typename Four<GF>::raw vg[kNq];
  f32x4_t vm[kNq];
  const auto load = [&](int64_t k, auto full) __attribute__((always_inline)) {
    const int left = (int)(k1 - k);
    st.template load<decltype(full)::value, GF>(grad, k, left, vg);
    st.template load<decltype(full)::value, true>((global<const float>)mom, k, left, vm);
  };
  if (k0 + KB <= k1) load(k0, std::true_type{});
  for (int q = tid; q < Shape::kFloats; q += kThreads) lds[q] = 0.f;  // (past the short side it stays so)
  const int group = wave % Shape::kGroups, part = wave / Shape::kGroups;
  f64x4_t sum[Shape::kPer];
  int row_i[Shape::kPer], row_j[Shape::kPer], tall_place[kNq];
#pragma unroll
  for (int t = 0; t < Shape::kPer; ++t) {
    sum[t] = f64x4_t{0, 0, 0, 0};
    int ti, tj;
    lower_tile(min(group + t * Shape::kGroups, Shape::kTiles - 1), &ti, &tj);
    row_i[t] = WIDE ? (16 * ti + i) * P + 4 * g : g * P + 16 * ti + i;
    row_j[t] = WIDE ? (16 * tj + i) * P + 4 * g : g * P + 16 * tj + i;
  }
#pragma unroll
  for (int q = 0; q < kNq; ++q) tall_place[q] = WIDE ? 0 : st.template place<P>(q);
  const auto place = [&](int q) { return WIDE ? st.template place<P>(q) : tall_place[q]; };
  const auto stage = [&](int64_t k, auto full) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full)::value;
    const int left = (int)(k1 - k);
    lds_barrier();
#pragma unroll
    for (int q = 0; q < kNq; ++q) {
      const f32x4_t gg = Four<GF>::value(vg[q]) * gs, mm = a.momentum * vm[q] + gg;
      st.template store<FULL, true>(mom, q, k, left, mm);
      if (st.has(q)) st.template put<P>(lds, place(q), a.nesterov ? gg + a.momentum * mm : mm);
    }
    lds_barrier();
    if (FULL && k + 2 * KB <= k1) load(k + KB, full);
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) {
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
        f32x4_t acc = zero4();
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma_f32(x[e], y[e], acc);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[t][e] += (double)acc[e];
      }
    }
  };
  int64_t k = k0;
  for (; k + KB <= k1; k += KB) stage(k, std::true_type{});
  if (k < k1) {
    load(k, std::false_type{});
    stage(k, std::false_type{});
  }
  // the column parts meet in LDS, in order
  const auto out = (global<f64x4_t>)(parts + (int64_t)piece * Shape::kTiles * 256);
  double* at = reinterpret_cast<double*>(lds) + (group * 64 + lane) * 4;
  for (int q = Shape::kParts - 1; q > 0; --q) {
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) {
      lds_barrier();
      if (part == q)
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e] = sum[t][e];
      lds_barrier();
      if (part == q - 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[t][e] += at[e];
    }
  }
  if (part == 0)
#pragma unroll
    for (int t = 0; t < Shape::kPer; ++t) {
      const int tile = group + t * Shape::kGroups;
      if (tile < Shape::kTiles) out[tile * 64 + lane] = sum[t];
    }
}

template <int NT, bool GF>
__global__ __launch_bounds__(GramShape<NT>::kWaves * 64) void muon_gram_kernel(MuonArgs a, int64_t c0) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const MuonChunk ch = a.chunks[c0 + blockIdx.x];
  const MuonMatrix& M = a.matrices[ch.matrix];
  if (M.wide) gram<NT, GF, true>(a, M, ch.part, lds);
  else gram<NT, GF, false>(a, M, ch.part, lds);
}

template <int NT, bool GF>
hipError_t launch_class(const MuonArgs& a, int64_t c0, int64_t chunks, hipStream_t s) {
  using Shape = GramShape<NT>;
  constexpr size_t kLds = (size_t)Shape::kFloats * 4;
  static_assert(Shape::kParts == 1 || kLds >= (size_t)Shape::kGroups * 64 * 4 * 8, "the parts' sums fit the stage");
  hipLaunchKernelGGL((muon_gram_kernel<NT, GF>), dim3((unsigned)chunks), dim3(Shape::kWaves * 64), kLds, s, a, c0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon_gram(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s) {
  return with_muon_tiles(cls, [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    return a.g_f32 ? launch_class<NT, true>(a, c0, chunks, s) : launch_class<NT, false>(a, c0, chunks, s);
  });
}

}  // namespace salr

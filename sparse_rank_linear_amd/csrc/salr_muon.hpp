// The orthogonalised step: what the C ABI (salr_muon_api.cpp) and the kernels
// (muon_*.hip) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

namespace salr {

// A matrix's short side in tiles of 16, rounded up to one of these (a class).
constexpr int kMuonClasses = 11;
constexpr int kMuonTiles[kMuonClasses] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16};
constexpr int kMuonLdsClasses = 7;  // the first ones iterate within one CU's LDS
constexpr int kMuonMaxSteps = 6;

// Columns of the long side that a workgroup holds in LDS at a time.
constexpr int muon_stage(int tiles) {
  return tiles == 1 ? 256 : tiles <= 3 ? 128 : tiles <= 7 ? 64 : 32;
}
constexpr int muon_lower(int tiles) { return tiles * (tiles + 1) / 2; }

struct MuonMatrix {
  void* p;
  const void* g;
  float* m;
  float* master;
  double* parts;  // partial products with itself: [chunks][lower tiles][256]
  float* q;       // [S][S]: what the update is multiplied with, S = 16 tiles
  double* work;   // large classes: six [S][S] matrices
  int64_t L;      // long side
  int32_t s;      // short side
  int32_t wide;   // the long side is the contiguous one
  int32_t chunks, chunk;  // pieces of the long side, and their columns
  float lr_scale;
  int32_t pad;
};

struct MuonChunk {
  int32_t matrix, part;
};

struct MuonArgs {
  const MuonMatrix* matrices;
  const MuonChunk* chunks;
  const float* dyn;     // nullptr, or {lr, grad_scale}
  float lr, grad_scale, momentum, weight_decay;
  double eps, a, b, c;
  int32_t steps;
  bool nesterov, p_f32, g_f32, master;
};

// f with a class's tiles as a constant.
template <class F>
hipError_t with_muon_tiles(int cls, F f) {
  switch (cls) {
    case 0: return f(std::integral_constant<int, kMuonTiles[0]>{});
    case 1: return f(std::integral_constant<int, kMuonTiles[1]>{});
    case 2: return f(std::integral_constant<int, kMuonTiles[2]>{});
    case 3: return f(std::integral_constant<int, kMuonTiles[3]>{});
    case 4: return f(std::integral_constant<int, kMuonTiles[4]>{});
    case 5: return f(std::integral_constant<int, kMuonTiles[5]>{});
    case 6: return f(std::integral_constant<int, kMuonTiles[6]>{});
    case 7: return f(std::integral_constant<int, kMuonTiles[7]>{});
    case 8: return f(std::integral_constant<int, kMuonTiles[8]>{});
    case 9: return f(std::integral_constant<int, kMuonTiles[9]>{});
    default: return f(std::integral_constant<int, kMuonTiles[10]>{});
  }
}
static_assert(kMuonClasses == 11, "the cases above");

// One class: its matrices [m0, m0 + n_matrices) or its chunks [c0, c0 + chunks).
hipError_t launch_muon_gram(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s);
hipError_t launch_muon_iterate(const MuonArgs& a, int cls, int32_t m0, int32_t n_matrices, hipStream_t s);
hipError_t launch_muon_apply_f32(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s);
hipError_t launch_muon_apply_bf16(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s);
hipError_t launch_muon_apply_master(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s);

}  // namespace salr

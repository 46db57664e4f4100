// Adapters of many requests: what the C ABI (salr_adapters_api.cpp) and the
// kernels (adapters.hip) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace salr {

// Tokens of a tile, all of one adapter.  Few tokens take small tiles: more
// workgroups, leaner kernels, and the pieces of T few enough to be summed where
// they are used (256 tokens of 32 adapters, rank 16, 4096 x 14336: 13 us, with
// large tiles 20; 64 tokens of 64 adapters, rank 64, 4096 x 4096: 20 and 28).
// Many take large ones: the adapter is read once for four times the tokens
// (8191 tokens, ranks 8 to 64, 4096 x 11008: 133 us, with small tiles 228).
constexpr int kAdapterSmallTile = 16, kAdapterLargeTile = 64;
constexpr int64_t kAdapterSmallTokens = 1024;  // the most with small tiles
// Tokens that one workgroup sums a gradient over, at least (more from 16384
// tokens on, a 32nd of them), and so not more than 64 partial sums in all:
// products and sums take 56 us for 4099 tokens of 6 adapters, rank 80, 4096 x
// 11008, in chunks of 1024 tokens 64, of 256 63.
constexpr int kAdapterMinChunk = 512;
constexpr int kAdapterMaxSplits = 32;  // pieces of a contraction over K (or N)
constexpr int kAdapterThreads = 256;   // of a workgroup, all kernels but the plan's

// The rank tiles of 16 go in groups of up to five, as even as they go.
inline int adapter_rank_groups(int r) { return ((r + 15) / 16 + 4) / 5; }

// One tile or chunk: tokens order[begin, end) of one adapter (`count`: tokens
// without any).  part: a chunk's place among the partial sums, -1 where its
// adapter has no other chunk.
struct alignas(16) AdapterTile {
  int32_t adapter, begin, end, part;
};

// The device arrays of a plan and the bounds that launches go by.
struct AdapterPlan {
  int32_t* head;        // {tiles, chunks}
  int32_t* offsets;     // [count + 2]: where each adapter's tokens begin in `order`
  int32_t* parts;       // [count + 2]: partial sums before each adapter's
  int32_t* order;       // [M]: the tokens, sorted by adapter (stable)
  AdapterTile* tiles;
  AdapterTile* chunks;
  int64_t M;
  int32_t count, tile, chunk;
  int32_t max_tiles, max_chunks;
};

// One contraction T[t][j] = sum_k X[t][k] W[a][j][k], in `splits` pieces of
// `cols` columns: T[piece][sorted token][j].
struct AdapterDown {
  const uint16_t* X;
  const uint16_t* W;
  float* T;
  int64_t K;
  int32_t splits, cols;
};

// The sums of T's pieces, times the adapter's scale, as three bf16 planes
// whose sum is the value: planes[3][M][r].
struct AdapterFinish {
  const float* T;
  uint16_t* planes;
  int32_t splits;
};

// out[t][n] = base[t][n] + sum_j V[t][j] W[a][n][j], V from T's pieces (times
// the scale) or from planes.
struct AdapterUp {
  const float* T;
  const uint16_t* planes;
  const uint16_t* W;
  const uint16_t* base;
  uint16_t* out;
  int64_t N;
  int32_t splits, slices;
};

// The sum over an adapter's tokens of cols[t][c] planes[t][j], stored [r][C] (dA)
// or [C][r] (dB).  other: the planes of what cols gave (dA: T, dB: G).
struct AdapterGrad {
  const uint16_t* cols;
  const uint16_t* planes;
  const uint16_t* other;
  float* out;
  float* parts;
  int64_t C;
};

struct AdapterCommon {
  AdapterPlan plan;
  const int32_t* ranks;
  const float* scales;
  int32_t r;
};

hipError_t launch_adapter_plan(const int32_t* ids, const AdapterPlan& p, hipStream_t s);
hipError_t launch_adapter_down(const AdapterCommon& c, const AdapterDown* jobs, int n_jobs, hipStream_t s);
hipError_t launch_adapter_finish(const AdapterCommon& c, const AdapterFinish* jobs, int n_jobs, hipStream_t s);
hipError_t launch_adapter_up(const AdapterCommon& c, const AdapterUp& u, hipStream_t s);
hipError_t launch_adapter_transpose(const AdapterCommon& c, const uint16_t* a, uint16_t* at, int64_t K,
                                    const uint16_t* b, uint16_t* bt, int64_t N, hipStream_t s);
// d_a: rank-major [r][K], d_b: [N][r].
hipError_t launch_adapter_grads(const AdapterCommon& c, const AdapterGrad& d_a, const AdapterGrad& d_b, hipStream_t s);

}  // namespace salr

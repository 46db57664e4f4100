// Adapters of many requests beside a shared projection, and their gradients
// (include/salr.h, salr_adapters_forward and salr_adapters_backward).
//
// With a = ids[t] and s_a its scale:
//   T[t][j] = sum_k X[t][k] A_a[j][k],   Y[t][n] = base[t][n] + s_a sum_j T[t][j] B_a[n][j]
//   G[t][j] = s_a sum_n dY[t][n] B_a[n][j],   dX[t][k] = base[t][k] + sum_j G[t][j] A_a[j][k]
//   dA_a[j][k] = sum_t G[t][j] X[t][k],   dB_a[n][j] = s_a sum_t dY[t][n] T[t][j]
// A plan sorts the tokens by adapter once for all the projections of a batch
// and cuts them into tiles of up to 64 tokens of one adapter, so every product
// is a matrix product of one adapter with a tile's (gathered) rows on the
// matrix cores.  With r small beside N and K all of it is bound by memory; the
// forward's floor is one read of X and base and one write of Y.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "salr_adapters.hpp"
#include "salr_device.hpp"

namespace salr {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kThreads = kAdapterThreads;
constexpr int kWaves = kThreads / 64;

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// ---- the plan ----

__device__ __forceinline__ uint32_t wave_prefix(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

// The largest g in [0, n] with start[g] <= x, of those the last (start
// ascending, start[0] = 0): the group that item x belongs to.
__device__ __forceinline__ int group_of(const uint32_t* start, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One workgroup sorts: a stable counting sort over the groups 0..count (the
// last: no adapter), each wave on its own stretch of the tokens.  One pass
// counts, prefix sums place the groups and the waves within them, and a second
// pass places, 64 tokens at a time: those of one adapter find each other by a
// ballot for each bit of its number.  Then the lists of tiles and chunks.
// Bound by its chain of barriers and LDS and memory round trips (64 tokens 6.0
// us, 8192 tokens of 16 adapters 10.2; with the ids read and matched twice 6.6
// and 10.8): once for all projections of a batch.  From some 16384 tokens on one
// workgroup is too few (65536 tokens of 16 adapters in 64 runs 43 us, in any
// order 83; 2^20 tokens 592 and 1246).
__global__ __launch_bounds__(kPlanThreads) void adapter_plan_kernel(const int32_t* ids, AdapterPlan p, int waves,
                                                                    int bits) {
  extern __shared__ uint32_t sm[];
  const int G = p.count + 1;
  uint32_t* cnt = sm;                          // [waves][G]
  uint32_t* off = cnt + waves * G;             // [G + 1] tokens before each group
  uint32_t* tile = off + G + 1;                // [G + 1] tiles before each group
  uint32_t* chunk = tile + G + 1;              // [G + 1] chunks
  uint32_t* part = chunk + G + 1;              // [G + 1] partial sums
  __shared__ uint32_t wsum[4][kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < waves * G; i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t M = p.M;
  const int64_t each = ((M + waves - 1) / waves + 63) / 64 * 64;
  const int64_t t0 = min(M, wave * each), t1 = min(M, t0 + each);  // (no tokens from wave `waves` on)
  const uint64_t below = (1ull << lane) - 1ull;
  // f(token, its group, whether it exists, the lanes of the same group) for 64
  // tokens at a time, in order; kAhead such batches are read together, and kept
  // for the second pass where there are no more
  constexpr int kAhead = 8;
  int group[kAhead];
  uint64_t alike[kAhead];
  const auto walk = [&](bool second, auto f) __attribute__((always_inline)) {
    for (int64_t b = t0; b < t1; b += 64 * kAhead) {
      if (!second || each > 64 * kAhead) {
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          const int x = ids[min(b + 64 * q + lane, t1 - 1)];
          group[q] = (uint32_t)x < (uint32_t)p.count ? x : p.count;
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          if (b + 64 * q >= t1) break;
          const bool live = b + 64 * q + lane < t1;
          const int x = group[q];
          uint64_t same = __ballot(live);
          if (__ballot(live && x == __builtin_amdgcn_readfirstlane(x)) != same) {  // (a prompt's tokens are alike)
            for (int k = 0; k < bits; ++k) {
              const uint64_t set = __ballot((x >> k) & 1);
              same &= (x >> k) & 1 ? set : ~set;
            }
          }
          alike[q] = same;
        }
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (b + 64 * q >= t1) break;
        f(b + 64 * q + lane, group[q], b + 64 * q + lane < t1, alike[q]);
      }
    }
  };
  walk(false, [&](int64_t, int g, bool live, uint64_t same) {
    if (live && (same & below) == 0) cnt[wave * G + g] += (uint32_t)__popcll(same);
  });
  __syncthreads();
  // each thread a run of groups: their totals, then what lies before them
  const int per = (G + kPlanThreads - 1) / kPlanThreads;
  const int g0 = min(G, tid * per), g1 = min(G, g0 + per);
  uint32_t n[4] = {0, 0, 0, 0};
  const auto add = [&](int g, uint32_t c) {
    const uint32_t ch = g < p.count ? (c + p.chunk - 1) / p.chunk : 0;
    n[0] += c;
    n[1] += (c + p.tile - 1) / p.tile;
    n[2] += ch;
    n[3] += ch > 1 ? ch : 0;
  };
  for (int g = g0; g < g1; ++g) {
    uint32_t run = 0;
    for (int w = 0; w < waves; ++w) {
      const uint32_t c = cnt[w * G + g];
      cnt[w * G + g] = run;
      run += c;
    }
    off[g] = run;  // (the group's own count until it is placed below)
    add(g, run);
  }
  uint32_t before[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t incl = wave_prefix(n[q], lane);
    if (lane == 63) wsum[q][wave] = incl;
    before[q] = incl - n[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // (all read: a loop to `wave` would wait for one after another, 0.7 us)
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) before[q] += w < wave ? wsum[q][w] : 0u;
    n[q] = before[q];
  }
  for (int g = g0; g < g1; ++g) {
    const uint32_t c = off[g];
    off[g] = n[0];
    tile[g] = n[1];
    chunk[g] = n[2];
    part[g] = n[3];
    for (int w = 0; w < waves; ++w) cnt[w * G + g] += n[0];
    add(g, c);
    if (g == G - 1) {
      off[G] = n[0];
      tile[G] = n[1];
      chunk[G] = n[2];
      part[G] = n[3];
    }
  }
  __syncthreads();
  for (int g = tid; g <= G; g += kPlanThreads) {
    p.offsets[g] = (int32_t)off[g];
    p.parts[g] = (int32_t)part[g];
  }
  if (tid == 0) {
    p.head[0] = (int32_t)tile[G];
    p.head[1] = (int32_t)chunk[G];
  }
  // place the tokens
  walk(true, [&](int64_t t, int g, bool live, uint64_t same) {
    if (!live) return;
    uint32_t* at = &cnt[wave * G + g];
    const uint32_t first = *at;
    __builtin_amdgcn_wave_barrier();
    if ((same & below) == 0) *at = first + (uint32_t)__popcll(same);
    p.order[first + __popcll(same & below)] = (int32_t)t;
    __builtin_amdgcn_wave_barrier();
  });
  // the lists
  for (uint32_t i = tid; i < tile[G]; i += kPlanThreads) {
    const int g = group_of(tile, G, i);
    const uint32_t b = off[g] + (i - tile[g]) * p.tile;
    p.tiles[i] = AdapterTile{g, (int32_t)b, (int32_t)min(off[g + 1], b + (uint32_t)p.tile), -1};
  }
  for (uint32_t i = tid; i < chunk[G]; i += kPlanThreads) {
    const int g = group_of(chunk, G, i);
    const uint32_t b = off[g] + (i - chunk[g]) * p.chunk;
    const bool alone = chunk[g + 1] - chunk[g] == 1;
    p.chunks[i] = AdapterTile{g, (int32_t)b, (int32_t)min(off[g + 1], b + (uint32_t)p.chunk),
                              alone ? -1 : (int32_t)(part[g] + i - chunk[g])};
  }
}

__device__ __forceinline__ int live_ranks(const AdapterCommon& c, int adapter) {
  return c.ranks ? min(max(c.ranks[adapter], 0), c.r) : c.r;
}
__device__ __forceinline__ float scale_of(const AdapterCommon& c, int adapter) {
  return c.scales ? c.scales[adapter] : 1.f;
}

// x as a sum of bf16 values, the first the nearest to it (of those that are
// finite, where x is): two of them hold 16 of a float's 24 bits, three all of
// them.  An infinite first one is all.
__device__ __forceinline__ void limbs(float x, uint16_t* w, int n) {
  constexpr uint32_t kExp = 0x7F800000u;
  const bool finite = (__float_as_uint(x) & kExp) != kExp;
  w[0] = f32_to_bf16(x);
  if (finite && (w[0] & 0x7FFFu) == 0x7F80u) w[0] -= 1;
  float rest = finite ? x - bf16_to_f32(w[0]) : 0.f;
  for (int i = 1; i < n; ++i) {
    w[i] = f32_to_bf16(rest);
    rest -= bf16_to_f32(w[i]);
  }
}

// The sum of T's pieces at one place, eight loads at a time.
__device__ __forceinline__ f32x4_t sum_pieces(const float* at, int64_t plane, int splits) {
  f32x4_t v = zero4();
  for (int s = 0; s < splits; s += 8) {
    f32x4_t x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = *reinterpret_cast<const f32x4_t*>(at + min(s + q, splits - 1) * plane);
#pragma unroll
    for (int q = 0; q < 8; ++q) v += s + q < splits ? x[q] : zero4();
  }
  return v;
}

// ---- down: T = X W^T for one tile, RT x 16 ranks, one piece of the columns ----
//
// D[rank][token] tiles; both operands run along the columns and come straight
// from memory, 16 bytes a lane.  Each wave takes every kWaves-th 64 columns of
// the piece; the waves' sums meet in LDS, in wave order.  Neighbouring
// workgroups take a tile's pieces (they run on different dies: a die then sees
// the same pieces of the adapters again and again, in its own cache; empty
// workgroups between them would leave some dies less to do).  Bound by
// the reads of X and dY, and above 32 ranks by how few waves have them in flight:
// 8192 tokens x 4096, rank 16, both sides 37.5 us, 3.6 TB/s (and 8 MB of pieces
// written; 122 + 36 registers and accumulators a lane, three waves a SIMD); 8191
// prompt tokens 25, 2.7 TB/s (ranks 8 to 64: 132 + 88, two waves); rank 80, 4099
// tokens, 4096 + 11008 columns 51, 2.4 TB/s (150 + 116, ten more than two waves
// would leave each, so one, without loads ahead); ranks 128 and 256 run as two
// and four groups of 64, each of which reads the tokens again (8192 tokens x
// 4096, both sides: 105 and 162 us).  One token: a
// wait for memory, 3.3 us.  One launch with the outputs' kernel, each workgroup
// of a small tile contracting for itself, takes longer than the two: 64 tokens
// of 64 adapters 30 us for 20, one token 9.2 for 8.6.
template <int RT, int NS>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(AdapterCommon c, AdapterDown j0, AdapterDown j1,
                                                                int parts0, int parts, int groups) {
  __shared__ f32x4_t sums[kWaves][RT][64];
  const AdapterPlan& p = c.plan;
  const int ti = blockIdx.x / parts, any = blockIdx.x % parts;  // (parts: those of both contractions)
  const AdapterTile t = p.tiles[ti];                           // (past the last: whatever was there)
  if (ti >= p.head[0] || t.adapter >= p.count) return;
  const bool first = any < parts0;
  const AdapterDown j = first ? j0 : j1;
  const int part = first ? any : any - parts0, split = part / groups, rank0 = (part % groups) * RT * 16;
  const int live = live_ranks(c, t.adapter);
  if (split >= j.splits || rank0 >= live) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int n = t.end - t.begin, subs = (n + 15) / 16;
  // (tokens past the tile's last and ranks past the live ones repeat those:
  // what comes of them is not used)
  const uint16_t* xr[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) xr[s] = j.X + (int64_t)p.order[t.begin + min(16 * s + i, n - 1)] * j.K;
  const int64_t k0 = (int64_t)split * j.cols, k1 = min(j.K, k0 + j.cols);
  constexpr int64_t kStep = 64 * kWaves;
  f32x4_t acc[RT][NS];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[a][s] = zero4();
  // RL rank tiles: those with live ranks, as far as they are told apart
  const auto body = [&](auto ranks) __attribute__((always_inline)) {
    constexpr int RL = decltype(ranks)::value;
    const uint16_t* wr[RL];
#pragma unroll
    for (int a = 0; a < RL; ++a)
      wr[a] = j.W + ((int64_t)t.adapter * c.r + min(rank0 + 16 * a + i, live - 1)) * j.K;
    const auto load = [&](int64_t k, u32x4_t (&xs)[2][NS], u32x4_t (&ws)[2][RL]) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a lane past the piece reads its first columns instead, and takes zeros)
        const int64_t at = k + 32 * h + 8 * g < k1 ? k + 32 * h + 8 * g : k0;
#pragma unroll
        for (int a = 0; a < RL; ++a) ws[h][a] = load16(wr[a] + at);
#pragma unroll
        for (int s = 0; s < NS; ++s) xs[h][s] = load16(xr[s] + at);
      }
    };
    const auto multiply = [&](int64_t k, u32x4_t (&xs)[2][NS], u32x4_t (&ws)[2][RL]) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (k + 64 > k1) {
          const bool in = k + 32 * h + 8 * g < k1;
#pragma unroll
          for (int a = 0; a < RL; ++a) ws[h][a] = in ? ws[h][a] : zero_u4();
#pragma unroll
          for (int s = 0; s < NS; ++s) xs[h][s] = in ? xs[h][s] : zero_u4();
        }
#pragma unroll
        for (int a = 0; a < RL; ++a)
#pragma unroll
          for (int s = 0; s < NS; ++s) acc[a][s] = mfma_16x16x32(ws[h][a], xs[h][s], acc[a][s]);
      }
    };
    if constexpr (NS == 1 || RL == 1) {
      // (few registers a step: the next step's loads ahead)
      u32x4_t x[2][2][NS], w[2][2][RL];
      int64_t k = k0 + 64 * wave;
      if (k < k1) load(k, x[0], w[0]);
      for (; k < k1; k += 2 * kStep) {
        if (k + kStep < k1) load(k + kStep, x[1], w[1]);
        multiply(k, x[0], w[0]);
        if (k + kStep >= k1) break;
        if (k + 2 * kStep < k1) load(k + 2 * kStep, x[0], w[0]);
        multiply(k + kStep, x[1], w[1]);
      }
    } else {
      u32x4_t x[2][NS], w[2][RL];
      for (int64_t k = k0 + 64 * wave; k < k1; k += kStep) {
        load(k, x, w);
        multiply(k, x, w);
      }
    }
  };
  constexpr int kHalf = (RT + 1) / 2;
  if (RT > 1 && live - rank0 <= 16) body(std::integral_constant<int, 1>{});
  else if (kHalf > 1 && live - rank0 <= 16 * kHalf) body(std::integral_constant<int, kHalf>{});
  else body(std::integral_constant<int, RT>{});
  float* out = j.T + (int64_t)split * p.M * c.r;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if (s >= subs) break;
#pragma unroll
    for (int a = 0; a < RT; ++a) sums[wave][a][lane] = acc[a][s];
    lds_barrier();
    for (int q = tid; q < RT * 64; q += kThreads) {
      const int a = q >> 6, l = q & 63;
      f32x4_t v = sums[0][a][l];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += sums[w][a][l];
      const int row = 16 * s + (l & 15), rank = rank0 + 16 * a + 4 * (l >> 4);
      if (row < n && rank < c.r) *reinterpret_cast<f32x4_t*>(out + (int64_t)(t.begin + row) * c.r + rank) = v;
    }
    if (NS > 1) lds_barrier();
  }
}

// ---- finish: the pieces' sums as bf16 planes, for large tiles and gradients,
// whose many workgroups would each sum the pieces (8191 tokens, 4096 x 11008,
// ranks 8 to 64: up 109 us with that, 101 and 6 without) ----
__global__ __launch_bounds__(kThreads) void adapter_finish_kernel(AdapterCommon c, AdapterFinish x, AdapterFinish y) {
  const AdapterPlan& p = c.plan;
  const AdapterTile t = p.tiles[blockIdx.x];  // (past the last: whatever was there)
  if ((int)blockIdx.x >= p.head[0] || t.adapter >= p.count) return;
  const AdapterFinish f = blockIdx.y ? y : x;
  const int live = live_ranks(c, t.adapter), rq = c.r / 4;
  const float scale = scale_of(c, t.adapter);
  const int64_t plane = p.M * c.r;
  for (int q = threadIdx.x; q < (t.end - t.begin) * rq; q += kThreads) {
    const int rank = q % rq * 4;
    const int64_t at = (int64_t)(t.begin + q / rq) * c.r + rank;
    f32x4_t v = zero4();
    if (rank < live) v = sum_pieces(f.T + at, plane, f.splits);
    uint16_t w[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) limbs(rank + e < live ? v[e] * scale : 0.f, w[e], 3);
#pragma unroll
    for (int l = 0; l < 3; ++l)
      *reinterpret_cast<u32x2_t*>(f.planes + l * plane + at) =
          u32x2_t{w[0][l] | (uint32_t)w[1][l] << 16, w[2][l] | (uint32_t)w[3][l] << 16};
  }
}

// ---- up: out = base + V W^T for one tile and a slice of the outputs ----
//
// D[output][token] tiles.  V (two bf16 planes: its rounding stays below 2^-16
// of it) waits in LDS.  A wave takes 64 outputs at a time; row m of the four
// tiles q is output 32 (q / 2) + 8 (m / 4) + 4 (q % 2) + m % 4, so that a lane
// ends up with twice 8 consecutive outputs of one token, and four lanes with 64
// bytes that lie together.  Bound by memory, reads and writes in equal parts:
// 8191 tokens x 11008 outputs 101 us, 3.6 TB/s (a copy of that size: 74); 8192 x
// 4096 32 us, 4.2.  Stores past the caches are slower.  Above 96 ranks
// (large tiles: 128) the weights of 64 outputs leave room for one wave a SIMD (64
// tokens, 4096 outputs, rank 128 6.4 us, 256 10.8; 8192 tokens 67 and 142 to 157).
// An adapter of fewer ranks than are stored is read whole, as its ranks share
// their lines (64 adapters of 64 to 8 ranks: 34.6 MB for 16).
template <int RC, int NS, bool PLANES>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(AdapterCommon c, AdapterUp u) {
  constexpr int kPitch = RC * 32 + 8;
  __shared__ __attribute__((aligned(16))) uint16_t v[2][16 * NS][kPitch];
  const AdapterPlan& p = c.plan;
  const int ti = blockIdx.x / u.slices, slice = blockIdx.x % u.slices;
  const AdapterTile t = p.tiles[ti];  // (past the last: whatever was there)
  if (ti >= p.head[0]) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int n = t.end - t.begin;
  const bool bare = t.adapter >= p.count;
  const int live = bare ? 0 : live_ranks(c, t.adapter);
  if (live == 0 && u.base == u.out) return;
  const bool vec = (u.N & 7) == 0;
  const int64_t steps = (u.N + 64 * kWaves - 1) / (64 * kWaves);
  const int64_t n0 = steps * slice / u.slices * 64 * kWaves;
  const int64_t n1 = min(u.N, steps * (slice + 1) / u.slices * 64 * kWaves);
  const uint16_t* W = u.W + (int64_t)(bare ? 0 : t.adapter) * u.N * c.r;
  // past the live ranks the weights may hold anything: masked out
  u32x4_t mask[RC];
#pragma unroll
  for (int k = 0; k < RC; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int left = live - 32 * k - 8 * g - 2 * e;
      mask[k][e] = (left > 0 ? 0xFFFFu : 0u) | (left > 1 ? 0xFFFF0000u : 0u);
    }
  int64_t row[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) row[s] = (int64_t)p.order[t.begin + min(16 * s + i, n - 1)] * u.N;
  // 64 outputs' weights and base
  const auto load = [&](int64_t nb, u32x4_t (&w)[4][RC], u32x4_t (&b)[NS][2]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t o = min(nb + 32 * (q >> 1) + 8 * (i >> 2) + 4 * (q & 1) + (i & 3), u.N - 1);
#pragma unroll
      for (int k = 0; k < RC; ++k) {
        const int rank = 32 * k + 8 * g;
        w[q][k] = load16(W + o * c.r + (rank < live ? rank : 0));
      }
    }
    if (vec && u.base) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) b[s][h] = load16(u.base + row[s] + min(nb + 32 * h + 8 * g, u.N - 8));
    }
  };
  const auto finish = [&](int64_t nb, u32x4_t (&w)[4][RC], const u32x4_t (&b)[NS][2]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int k = 0; k < RC; ++k) w[q][k] &= mask[k];
    const int64_t o0 = nb + 8 * g;  // this lane's outputs: 8 from here, 8 from 32 on
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      f32x4_t acc[4] = {zero4(), zero4(), zero4(), zero4()};
      if (live > 0) {
#pragma unroll
        for (int k = 0; k < RC; ++k)
#pragma unroll
          for (int l = 0; l < 2; ++l) {
            const u32x4_t x = load16(&v[l][16 * s + i][32 * k + 8 * g]);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = mfma_16x16x32(w[q][k], x, acc[q]);
          }
      }
      if (16 * s + i >= n) continue;
      uint16_t* out = u.out + row[s];
      if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t o = o0 + 32 * h;
          const u32x4_t x = u.base ? b[s][h] : zero_u4();
          u32x4_t y;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = bf16_to_f32((uint16_t)x[e]) + acc[2 * h + e / 2][2 * (e & 1)];
            const float hi = bf16_to_f32((uint16_t)(x[e] >> 16)) + acc[2 * h + e / 2][2 * (e & 1) + 1];
            y[e] = f32_to_bf16(lo) | (uint32_t)f32_to_bf16(hi) << 16;
          }
          if (o < n1) *reinterpret_cast<u32x4_t*>(out + o) = live > 0 ? y : x;
        }
      } else {
        const uint16_t* base = u.base ? u.base + row[s] : nullptr;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t o = o0 + 32 * (q >> 1) + 4 * (q & 1) + e;
            if (o >= n1) continue;
            const uint16_t x = base ? base[o] : (uint16_t)0;
            out[o] = live > 0 ? f32_to_bf16(bf16_to_f32(x) + acc[q][e]) : x;
          }
      }
    }
  };
  // (the next outputs' loads ahead, where the registers hold them)
  constexpr bool kAhead = NS == 1;
  u32x4_t w[2][4][RC], b[2][NS][2];
  constexpr int64_t kStep = 64 * kWaves;
  int64_t nb = n0 + 64 * wave;
  if (nb < n1) load(nb, w[0], b[0]);
  // V into LDS while those are under way
  if (live > 0) {
    const float scale = scale_of(c, t.adapter);
    const int64_t plane = p.M * c.r;
    constexpr int kQuads = RC * 8;
    for (int q = tid; q < NS * 16 * kQuads; q += kThreads) {
      const int vr = q / kQuads, rank = q % kQuads * 4;
      const bool in = vr < n && rank < live;
      const int64_t at = (int64_t)(t.begin + vr) * c.r + rank;
      u32x2_t hi = {0u, 0u}, lo = {0u, 0u};
      if constexpr (PLANES) {
        if (in) {
          hi = *reinterpret_cast<const u32x2_t*>(u.planes + at);
          lo = *reinterpret_cast<const u32x2_t*>(u.planes + plane + at);
        }
      } else if (in) {
        const f32x4_t x = sum_pieces(u.T + at, plane, u.splits);
        uint16_t h[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) limbs(rank + e < live ? x[e] * scale : 0.f, h[e], 2);
        hi = u32x2_t{h[0][0] | (uint32_t)h[1][0] << 16, h[2][0] | (uint32_t)h[3][0] << 16};
        lo = u32x2_t{h[0][1] | (uint32_t)h[1][1] << 16, h[2][1] | (uint32_t)h[3][1] << 16};
      }
      *reinterpret_cast<u32x2_t*>(&v[0][vr][rank]) = hi;
      *reinterpret_cast<u32x2_t*>(&v[1][vr][rank]) = lo;
    }
    lds_barrier();
  }
  if constexpr (!kAhead) {
    for (; nb < n1; nb += kStep) {
      finish(nb, w[0], b[0]);
      if (nb + kStep < n1) load(nb + kStep, w[0], b[0]);
    }
    return;
  }
  for (; nb < n1; nb += 2 * kStep) {
    if (nb + kStep < n1) load(nb + kStep, w[1], b[1]);
    finish(nb, w[0], b[0]);
    if (nb + kStep >= n1) break;
    if (nb + 2 * kStep < n1) load(nb + 2 * kStep, w[0], b[0]);
    finish(nb + kStep, w[1], b[1]);
  }
}

// ---- the adapters transposed (for the gradients): [R][C] -> [C][R], those
// with tokens only, 64 x 64 at a time; their bytes twice, 3 to 9 us, and 25 for
// 16 adapters of rank 256 ----
__global__ __launch_bounds__(kThreads) void adapter_transpose_kernel(AdapterCommon c, const uint16_t* a, uint16_t* at,
                                                                     int64_t K, const uint16_t* b, uint16_t* bt,
                                                                     int64_t N) {
  __shared__ uint16_t tile[64][66];
  const int adapter = blockIdx.z >> 1;
  const bool second = blockIdx.z & 1;
  if (c.plan.offsets[adapter] == c.plan.offsets[adapter + 1]) return;
  const int64_t R = second ? N : c.r, C = second ? c.r : K;
  const uint16_t* src = (second ? b : a) + (int64_t)adapter * R * C;
  uint16_t* dst = (second ? bt : at) + (int64_t)adapter * R * C;
  // (blockIdx.x along the long side, blockIdx.y along the ranks)
  const int64_t r0 = (int64_t)(second ? blockIdx.x : blockIdx.y) * 64;
  const int64_t c0 = (int64_t)(second ? blockIdx.y : blockIdx.x) * 64;
  if (r0 >= R || c0 >= C) return;
  const int ch = threadIdx.x & 7;  // 8 values
  for (int y = threadIdx.x >> 3; y < 64; y += kThreads / 8) {
    const bool in = r0 + y < R && c0 + 8 * ch < C;
    const u32x4_t x = in ? load16(src + (r0 + y) * C + c0 + 8 * ch) : zero_u4();
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(&tile[y][8 * ch + 2 * e]) = x[e];
  }
  __syncthreads();
  for (int y = threadIdx.x >> 3; y < 64; y += kThreads / 8) {
    if (c0 + y >= C || r0 + 8 * ch >= R) continue;
    u32x4_t x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = tile[8 * ch + 2 * e][y] | (uint32_t)tile[8 * ch + 2 * e + 1][y] << 16;
    *reinterpret_cast<u32x4_t*>(dst + (c0 + y) * R + r0 + 8 * ch) = x;
  }
}

// ---- gradients of the adapters: sums over a chunk's tokens ----
//
// Both operands run along the tokens while memory runs along the columns, so
// 32 tokens at a time go to LDS as they are and come back transposed (4 x 16
// values a 16 lanes).  T and G are three bf16 planes each: the float sums see
// all their bits.  Bound by the reads of X and dY, once for each group of up to
// 80 ranks: 8192 tokens, rank 16, 4096 x 4096 33.5 us, 4.0 TB/s; rank 80, 4099
// tokens, 4096 x 11008 48 us, 2.6 TB/s, three products a pair and 40
// accumulators a lane.  A look at one value a token first, for what is not
// finite, takes 1 us of each; at the columns themselves, stage by stage, up to 13.

__device__ __forceinline__ u32x4_t read_transposed(const uint16_t* tile, int pitch, int lane) {
  // lane (i, g) gets column i of rows 4g..4g+3 and 16+4g..16+4g+3
  typedef __attribute__((address_space(3))) s16x4_t lds_t;
  const int q = lane & 15, g = lane >> 4;
  const uint16_t* at = tile + (4 * g + (q >> 2)) * pitch + 4 * (q & 3);
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)at);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(at + 16 * pitch));
  const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
  return u32x4_t{a.x, a.y, b.x, b.y};
}

constexpr int kGradCols = 128;

template <int RT>
__global__ __launch_bounds__(kThreads) void adapter_grad_kernel(AdapterCommon c, AdapterGrad ga, AdapterGrad gb,
                                                                int blocks_a, int groups) {
  // (a wave: CT x 16 columns; 256 columns a workgroup, which read T and G half
  // as often, are slower: 41 us for 36 at 8192 tokens, rank 16, 4096 x 4096, in
  // chunks of 1024 tokens)
  constexpr int kCols = kGradCols, CT = kCols / (16 * kWaves), kColPitch = kCols + 8, kRankPitch = RT * 16 + 8;
  __shared__ __attribute__((aligned(16))) uint16_t cols[32 * kColPitch];
  __shared__ __attribute__((aligned(16))) uint16_t rank[3][32 * kRankPitch];
  const AdapterPlan& p = c.plan;
  const AdapterTile t = p.chunks[blockIdx.y];
  if ((int)blockIdx.y >= p.head[1]) return;
  const int by = blockIdx.x / groups, rank0 = (blockIdx.x % groups) * RT * 16;
  const bool is_a = by < blocks_a;
  const AdapterGrad j = is_a ? ga : gb;
  const int64_t c0 = (int64_t)(is_a ? by : by - blocks_a) * kCols;
  const int live = live_ranks(c, t.adapter);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int64_t plane = p.M * c.r;
  f32x4_t acc[RT][CT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int h = 0; h < CT; ++h) acc[a][h] = zero4();
  // A token whose columns hold an infinity or a NaN has one in the other product
  // of its row too, at every rank.
  bool odd = false;
  for (int b = t.begin + tid; b < t.end; b += kThreads)
    odd |= (j.other[(int64_t)b * c.r] & 0x7F80u) == 0x7F80u;
  // Sums over the chunk.  With APART, what is not finite among the columns meets
  // the first plane alone, which is infinite or NaN where T or G is, and zero
  // where it is: the others would make inf - inf or 0 * inf of it.  Otherwise the
  // same sums, in the same order.
  const auto sums = [&](int tid, auto apart) __attribute__((always_inline)) {
    constexpr bool APART = decltype(apart)::value;
    const int lane = tid & 63, wave = tid >> 6;
    // staging: 16 bytes of CT rows' columns, and 8 ranks of a plane's row a pass
    constexpr int kRowThreads = kCols / 8, kRows = kThreads / kRowThreads, kPasses = 32 / kRows;
    const int row = tid / kRowThreads, col = 8 * (tid % kRowThreads);
    const bool col_in = c0 + col < j.C;
    constexpr int kRankPieces = 3 * 32 * RT * 2, kRankPasses = (kRankPieces + kThreads - 1) / kThreads;
    u32x4_t vc[kPasses], vr[kRankPasses];
    int tok[kPasses];  // the tokens of the next stage
    const auto next_tokens = [&](int b) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < kPasses; ++h) tok[h] = p.order[min(b + row + kRows * h, t.end - 1)];
    };
    const auto load = [&](int b) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < kPasses; ++h)
        vc[h] = b + row + kRows * h < t.end && col_in ? load16(j.cols + (int64_t)tok[h] * j.C + c0 + col) : zero_u4();
      if (b + 32 < t.end) next_tokens(b + 32);
#pragma unroll
      for (int q = 0; q < kRankPasses; ++q) {
        const int x = tid + q * kThreads, l = x / (32 * RT * 2), y = x / (RT * 2) % 32, z = rank0 + x % (RT * 2) * 8;
        vr[q] = x < kRankPieces && b + y < t.end && z < live
                    ? load16(j.planes + l * plane + (int64_t)(b + y) * c.r + z)
                    : zero_u4();
      }
    };
    next_tokens(t.begin);
    load(t.begin);
    for (int b = t.begin; b < t.end; b += 32) {
      lds_barrier();
#pragma unroll
      for (int h = 0; h < kPasses; ++h) *reinterpret_cast<u32x4_t*>(&cols[(row + kRows * h) * kColPitch + col]) = vc[h];
#pragma unroll
      for (int q = 0; q < kRankPasses; ++q) {
        const int x = tid + q * kThreads, l = x / (32 * RT * 2), y = x / (RT * 2) % 32, z = x % (RT * 2) * 8;
        if (x < kRankPieces) *reinterpret_cast<u32x4_t*>(&rank[l][y * kRankPitch + z]) = vr[q];
      }
      lds_barrier();
      if (b + 32 < t.end) load(b + 32);
      u32x4_t x[CT];
#pragma unroll
      for (int h = 0; h < CT; ++h) x[h] = read_transposed(cols + 16 * (CT * wave + h), kColPitch, lane);
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        if (rank0 + 16 * a >= live) break;  // (zeros from here on)
#pragma unroll
        for (int l = 0; l < 3; ++l) {
          const u32x4_t y = read_transposed(rank[l] + 16 * a, kRankPitch, lane);
#pragma unroll
          for (int h = 0; h < CT; ++h) {
            u32x4_t v = x[h];
            if (APART && l > 0)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] &= ~(((((v[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xFFFFu);
            acc[a][h] = is_a ? mfma_16x16x32(v, y, acc[a][h]) : mfma_16x16x32(y, v, acc[a][h]);
          }
        }
      }
    }
  };
  if (!__syncthreads_or(odd)) {
    sums(tid, std::false_type{});
  } else {
    int again = tid;  // (one that shares no addresses with the loop above: they would stay in registers)
    asm volatile("" : "+v"(again));
    sums(again, std::true_type{});
  }
  // dA: the lane holds four columns of rank i; dB: four ranks of column i.
  // (Ranks past the live ones take zeros, whatever their planes' zeros met: 0
  // times an infinity or a NaN is none.)
  float* out = t.part < 0 ? j.out + (int64_t)t.adapter * c.r * j.C : j.parts + (int64_t)t.part * c.r * j.C;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int h = 0; h < CT; ++h) {
      const int64_t cc = c0 + 16 * (CT * wave + h) + (is_a ? 4 * g : i);
      const int rr = rank0 + 16 * a + (is_a ? i : 4 * g);
      f32x4_t v = acc[a][h];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = rr + (is_a ? 0 : e) < live ? v[e] : 0.f;
      if (cc < j.C && rr < c.r)
        *reinterpret_cast<f32x4_t*>(is_a ? out + (int64_t)rr * j.C + cc : out + cc * c.r + rr) = v;
    }
}

// The chunks' sums in order, for adapters with several; zeros for those
// without tokens.  (A few rows of float sums: 5 to 8 us.)
__global__ __launch_bounds__(kThreads) void adapter_grad_sum_kernel(AdapterCommon c, AdapterGrad ga, AdapterGrad gb,
                                                                    int blocks_a) {
  const AdapterPlan& p = c.plan;
  const int adapter = blockIdx.y;
  const int n = p.offsets[adapter + 1] - p.offsets[adapter], chunks = (n + p.chunk - 1) / p.chunk;
  if (chunks == 1) return;
  const bool is_a = (int)blockIdx.x < blocks_a;
  const AdapterGrad j = is_a ? ga : gb;
  const int64_t size = (int64_t)c.r * j.C;
  const int64_t e = ((int64_t)(is_a ? blockIdx.x : blockIdx.x - blocks_a) * kThreads + threadIdx.x) * 4;
  if (e >= size) return;
  const float* part = j.parts + p.parts[adapter] * size + e;
  f32x4_t v = zero4();
  for (int q = 0; q < chunks; ++q) v += *reinterpret_cast<const f32x4_t*>(part + q * size);
  *reinterpret_cast<f32x4_t*>(j.out + (int64_t)adapter * size + e) = v;
}

template <class F>
void with_rank_tiles(int r, F f) {
  const int groups = adapter_rank_groups(r), rt = ((r + 15) / 16 + groups - 1) / groups;
  if (rt == 1) f(std::integral_constant<int, 1>{}, groups);
  else if (rt == 2) f(std::integral_constant<int, 2>{}, groups);
  else if (rt == 3) f(std::integral_constant<int, 3>{}, groups);
  else if (rt == 4) f(std::integral_constant<int, 4>{}, groups);
  else f(std::integral_constant<int, 5>{}, groups);
}
template <class F>
void with_rank_chunks(int r, F f) {
  if (r <= 32) f(std::integral_constant<int, 1>{});
  else if (r <= 64) f(std::integral_constant<int, 2>{});
  else if (r <= 96) f(std::integral_constant<int, 3>{});
  else if (r <= 128) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_adapter_plan(const int32_t* ids, const AdapterPlan& p, hipStream_t s) {
  // (each wave's counters: 4 waves keep 4096 adapters within 132 KB of LDS; no
  // more waves than have 128 tokens each, as their counters are added up)
  const int waves = (int)std::max<int64_t>(1, std::min<int64_t>((p.M + 127) / 128, p.count <= 1024 ? kPlanWaves : 4));
  const size_t lds = ((size_t)waves * (p.count + 1) + 4 * (size_t)(p.count + 2)) * 4;
  int bits = 0;
  while ((1 << bits) <= p.count) ++bits;
  hipLaunchKernelGGL(adapter_plan_kernel, dim3(1), dim3(kPlanThreads), lds, s, ids, p, waves, bits);
  return hipGetLastError();
}

hipError_t launch_adapter_down(const AdapterCommon& c, const AdapterDown* jobs, int n_jobs, hipStream_t s) {
  int splits = 0;
  for (int q = 0; q < n_jobs; ++q) splits += jobs[q].splits;
  with_rank_tiles(c.r, [&](auto rt, int groups) {
    constexpr int RT = decltype(rt)::value;
    const int parts0 = jobs[0].splits * groups, parts = splits * groups;
    const dim3 grid((unsigned)c.plan.max_tiles * parts);
    if (c.plan.tile == kAdapterSmallTile)
      hipLaunchKernelGGL((adapter_down_kernel<RT, 1>), grid, dim3(kThreads), 0, s, c, jobs[0], jobs[n_jobs - 1], parts0,
                         parts, groups);
    else
      hipLaunchKernelGGL((adapter_down_kernel<RT, 4>), grid, dim3(kThreads), 0, s, c, jobs[0], jobs[n_jobs - 1], parts0,
                         parts, groups);
  });
  return hipGetLastError();
}

hipError_t launch_adapter_finish(const AdapterCommon& c, const AdapterFinish* jobs, int n_jobs, hipStream_t s) {
  hipLaunchKernelGGL(adapter_finish_kernel, dim3((unsigned)c.plan.max_tiles, (unsigned)n_jobs), dim3(kThreads), 0, s, c,
                     jobs[0], jobs[n_jobs - 1]);
  return hipGetLastError();
}

hipError_t launch_adapter_up(const AdapterCommon& c, const AdapterUp& u, hipStream_t s) {
  const dim3 grid((unsigned)c.plan.max_tiles * u.slices);
  with_rank_chunks(c.r, [&](auto rc) {
    constexpr int RC = decltype(rc)::value;
    const auto go = [&](auto ns) {
      constexpr int NS = decltype(ns)::value;
      if (u.planes)
        hipLaunchKernelGGL((adapter_up_kernel<RC, NS, true>), grid, dim3(kThreads), 0, s, c, u);
      else
        hipLaunchKernelGGL((adapter_up_kernel<RC, NS, false>), grid, dim3(kThreads), 0, s, c, u);
    };
    if (c.plan.tile == kAdapterSmallTile) go(std::integral_constant<int, 1>{});
    else go(std::integral_constant<int, 4>{});
  });
  return hipGetLastError();
}

hipError_t launch_adapter_transpose(const AdapterCommon& c, const uint16_t* a, uint16_t* at, int64_t K,
                                    const uint16_t* b, uint16_t* bt, int64_t N, hipStream_t s) {
  hipLaunchKernelGGL(adapter_transpose_kernel,
                     dim3((unsigned)((std::max(K, N) + 63) / 64), (unsigned)((c.r + 63) / 64),
                          (unsigned)(2 * c.plan.count)),
                     dim3(kThreads), 0, s, c, a, at, K, b, bt, N);
  return hipGetLastError();
}

hipError_t launch_adapter_grads(const AdapterCommon& c, const AdapterGrad& d_a, const AdapterGrad& d_b,
                                hipStream_t s) {
  const auto blocks = [](int64_t n, int64_t per) { return (int)((n + per - 1) / per); };
  if (c.plan.M > 0) {
    const int ba = blocks(d_a.C, kGradCols), bb = blocks(d_b.C, kGradCols);
    with_rank_tiles(c.r, [&](auto rt, int groups) {
      hipLaunchKernelGGL((adapter_grad_kernel<decltype(rt)::value>),
                         dim3((unsigned)((ba + bb) * groups), (unsigned)c.plan.max_chunks), dim3(kThreads), 0, s, c, d_a,
                         d_b, ba, groups);
    });
  }
  const int sa = blocks(d_a.C * c.r, 4 * kThreads), sb = blocks(d_b.C * c.r, 4 * kThreads);
  hipLaunchKernelGGL(adapter_grad_sum_kernel, dim3((unsigned)(sa + sb), (unsigned)c.plan.count), dim3(kThreads), 0, s, c,
                     d_a, d_b, sa);
  return hipGetLastError();
}

}  // namespace salr

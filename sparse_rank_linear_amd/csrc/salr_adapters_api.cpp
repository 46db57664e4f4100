// C ABI of the adapters of many requests: argument validation, plan and
// workspace layout.  See include/salr.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "salr.h"
#include "salr_adapters.hpp"
#include "salr_api_checks.hpp"

namespace {

// The most tokens: 2^21 + 4097 tiles, whose contraction of up to four groups of
// ranks is one launch still (launch_down).
constexpr int64_t kMaxTokens = int64_t(1) << 27;
constexpr int64_t kLaunchThreads = int64_t(1) << 32;  // a launch has fewer
constexpr int64_t kMaxColumns = int64_t(1) << 20;
constexpr int32_t kMaxRank = 256;
using namespace salr;

bool plan_shape_ok(int64_t M, int32_t count) {
  return M >= 0 && M <= kMaxTokens && count >= 1 && count <= SALR_ADAPTERS_MAX;
}

bool shape_ok(const salr_adapters_t* A) {
  return A && A->count >= 1 && A->count <= SALR_ADAPTERS_MAX && A->N >= 1 && A->N <= kMaxColumns && A->K >= 8 &&
         A->K <= kMaxColumns && A->K % 8 == 0 && A->r >= 8 && A->r <= kMaxRank && A->r % 8 == 0;
}

// Most pieces of `each` that the non-empty ones of `groups` groups of M tokens
// come to.
int64_t most_pieces(int64_t M, int64_t groups, int64_t each) {
  const int64_t used = std::min(M, groups);
  return (M + (each - 1) * used) / each;
}

// The plan's arrays in its buffer.  `bytes` (may be null): how long that is.
salr::AdapterPlan lay_out_plan(void* buffer, int64_t M, int32_t count, size_t* bytes) {
  salr::AdapterPlan p{};
  p.M = M;
  p.count = count;
  p.chunk = (int32_t)std::max<int64_t>(salr::kAdapterMinChunk, cdiv(cdiv(M, 32), 64) * 64);
  p.tile = M <= salr::kAdapterSmallTokens ? salr::kAdapterSmallTile : salr::kAdapterLargeTile;
  p.max_tiles = (int32_t)most_pieces(M, count + 1, p.tile);
  p.max_chunks = (int32_t)most_pieces(M, count, p.chunk);
  size_t at = 0;
  const auto take = [&](size_t n) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(buffer) + at;  // (the buffer may be null: sizes alone)
    at += align_up(n, 16);
    return reinterpret_cast<void*>(q);
  };
  p.head = static_cast<int32_t*>(take(16));
  p.offsets = static_cast<int32_t*>(take(((size_t)count + 2) * 4));
  p.parts = static_cast<int32_t*>(take(((size_t)count + 2) * 4));
  p.order = static_cast<int32_t*>(take((size_t)M * 4));
  // (room for what shorter batches have more of, so that a buffer serves those
  // too: small tiles, and chunks, which are M / 32 tokens long or more)
  const int64_t chunk_room = std::min<int64_t>(32, M / salr::kAdapterMinChunk) + std::min<int64_t>(M, count);
  const int64_t room = std::max<int64_t>(p.max_tiles, most_pieces(std::min(M, salr::kAdapterSmallTokens), count + 1,
                                                                  salr::kAdapterSmallTile));
  p.tiles = static_cast<salr::AdapterTile*>(take((size_t)room * sizeof(salr::AdapterTile)));
  p.chunks = static_cast<salr::AdapterTile*>(take((size_t)chunk_room * sizeof(salr::AdapterTile)));
  if (bytes) *bytes = at;
  return p;
}

// Contractions over their columns in pieces: enough workgroups for the CUs, and
// fewer for small tiles, whose pieces are summed by every workgroup that uses
// them, and where a token's sums are long (each piece writes them).  Above
// kFewRanks, pieces as long for one contraction as for the other and kRound
// workgroups in all, in eights where there are eight (4099 tokens, rank 80, 4096
// and 11008 columns: 51 us in 8 pieces; in 10 or 11 56, in 16 55).  A CU holds
// one workgroup of large tiles at a time at rank 80 (266 registers a lane), two
// at 48 and 64; with 256, 512, 768 and 1024 workgroups that batch takes 67, 53,
// 51 and 50 us, and 8192 tokens with 4096 columns on both sides 79, 64, 60 and
// 56 at rank 64 and 73, 58, 55 and 51 at rank 48, their sums 0.2 more: there more
// pieces would be better.  Up to kFewRanks kGroups workgroups or
// more for each contraction (rank 16: 37.5 us, cut as above 43.5; 24: 41.5 and
// 47; 32: 44.5 and 48.5).  The two, their sums added, come together at rank 64
// (40: 58 and 60 us, 48: 60 and 62, 64: 68 and 68).
//   Each of `work` tiles has at most 64 tokens, so that one piece, or up to
// (kGroups + work) / work, or up to kRound / work, come to at most M + 64
// kGroups rows of T, and as many as kAdapterMaxSplits M.
constexpr int64_t kGroups = 1024, kRound = 768;
constexpr int32_t kFewRanks = 32;
int64_t t_rows(int64_t M) { return std::min<int64_t>(salr::kAdapterMaxSplits * M, M + 64 * kGroups); }
void cut(salr::AdapterDown* d, int n, const salr::AdapterPlan& p, int32_t r) {
  const int64_t work = std::max<int64_t>(1, (int64_t)p.max_tiles * adapter_rank_groups(r));
  const bool small = p.tile == salr::kAdapterSmallTile, few = r <= kFewRanks;
  int64_t all = 0, round = kRound / work;
  if (round >= 8) round -= round % 8;
  for (int q = 0; q < n; ++q) all += d[q].K;
  for (int q = 0; q < n; ++q) {
    const int64_t each = small || few ? cdiv(kGroups / (small ? 2 : 1) / (few ? 1 : 2), work)
                                      : std::max<int64_t>(1, (2 * d[q].K * round + all) / (2 * all));
    const int64_t want = std::min<int64_t>(salr::kAdapterMaxSplits, each);
    d[q].cols = (int32_t)(cdiv(cdiv(d[q].K, want), 256) * 256);
    d[q].splits = (int32_t)cdiv(d[q].K, d[q].cols);
  }
}
// The contractions in one launch, or where that would have too many threads (both
// of a backward call whose tiles times groups of ranks are 2^23 or more) in one
// each.
hipError_t launch_down(const salr::AdapterCommon& c, const salr::AdapterDown* d, int n, hipStream_t s) {
  int64_t pieces = 0;
  for (int q = 0; q < n; ++q) pieces += d[q].splits;
  if (c.plan.max_tiles * adapter_rank_groups(c.r) * pieces * salr::kAdapterThreads < kLaunchThreads)
    return salr::launch_adapter_down(c, d, n, s);
  for (int q = 0; q < n; ++q)
    if (const hipError_t e = salr::launch_adapter_down(c, d + q, 1, s)) return e;
  return hipSuccess;
}
// Slices of N outputs: as many as 512 (small tiles, whose workgroups sum T's
// pieces first) or 2048 workgroups take, in eights where there are eight (one
// for each die, see adapter_down_kernel).  With 1024 for both: 64 tokens of 64
// adapters 12.9 us for 9.8, 8191 tokens 110 for 101.
int32_t up_slices(int64_t N, const salr::AdapterPlan& p) {
  const int64_t groups = p.tile == salr::kAdapterSmallTile ? 512 : 2048;
  const int64_t steps = cdiv(N, 256), want = cdiv(groups, std::max<int64_t>(1, p.max_tiles));
  return (int32_t)std::min(steps, want < 8 ? want : cdiv(want, 8) * 8);
}

struct Workspace {
  size_t t, planes, a, b, parts_a, parts_b, total;  // byte offsets (t: two of t_bytes in the backward)
  size_t t_bytes, planes_bytes;
};
Workspace lay_out(int64_t count, int64_t N, int64_t K, int32_t r, int64_t M, bool backward) {
  Workspace w{};
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t q = at;
    at += align_up(n, 256);
    return q;
  };
  w.t_bytes = align_up((size_t)t_rows(M) * r * 4, 256);
  w.planes_bytes = align_up((size_t)M * r * 6, 256);
  w.t = take(w.t_bytes * (backward ? 2 : 1));
  w.planes = take(w.planes_bytes * (backward ? 2 : 1));
  if (backward) {
    const int64_t parts = std::min<int64_t>(64, 2 * M / salr::kAdapterMinChunk);
    w.a = take((size_t)count * r * K * 2);
    w.b = take((size_t)count * r * N * 2);
    w.parts_a = take((size_t)parts * r * K * 4);
    w.parts_b = take((size_t)parts * r * N * 4);
  }
  w.total = std::max<size_t>(at, 256);
  return w;
}

// What both directions ask of the adapters and the plan.
int check(const salr_adapters_t* A, const salr_adapters_plan_t* P) {
  if (!shape_ok(A) || !P || !plan_shape_ok(P->M, P->count) || P->count != A->count) return SALR_ERR_INVALID_ARG;
  if (!P->buffer || !aligned16(P->buffer) || !A->a || !A->b) return SALR_ERR_INVALID_ARG;
  if (!aligned16(A->a) || !aligned16(A->b) || !aligned16(A->ranks) || !aligned16(A->scales))
    return SALR_ERR_INVALID_ARG;
  return SALR_OK;
}

}  // namespace

extern "C" {

int salr_adapters_plan_bytes(int64_t M, int32_t count, size_t* out) {
  if (!out || !plan_shape_ok(M, count)) return SALR_ERR_INVALID_ARG;
  lay_out_plan(nullptr, M, count, out);
  return SALR_OK;
}

int salr_adapters_plan(const int32_t* ids, int64_t M, int32_t count, void* buffer, size_t buffer_bytes,
                       salr_adapters_plan_t* out, void* stream) {
  if (!out || !plan_shape_ok(M, count) || (M > 0 && !ids) || !aligned16(ids)) return SALR_ERR_INVALID_ARG;
  size_t bytes = 0;
  const salr::AdapterPlan p = lay_out_plan(buffer, M, count, &bytes);
  if (!apart({ids, (size_t)M * 4}, {buffer, bytes})) return SALR_ERR_INVALID_ARG;
  if (!buffer || !aligned16(buffer) || buffer_bytes < bytes) return SALR_ERR_WORKSPACE;
  const int rc = status(salr::launch_adapter_plan(ids, p, static_cast<hipStream_t>(stream)));
  if (rc != SALR_OK) return rc;
  out->buffer = buffer;
  out->M = M;
  out->count = count;
  return SALR_OK;
}

int salr_adapters_ws_bytes(int32_t count, int64_t N, int64_t K, int32_t r, int64_t M_max, int32_t backward,
                           size_t* out) {
  salr_adapters_t A{};
  A.count = count;
  A.N = N;
  A.K = K;
  A.r = r;
  if (!out || !shape_ok(&A) || M_max < 0 || M_max > kMaxTokens) return SALR_ERR_INVALID_ARG;
  if (backward && N % 8 != 0) return SALR_ERR_UNSUPPORTED;
  *out = lay_out(count, N, K, r, M_max, backward != 0).total;
  return SALR_OK;
}

int salr_adapters_forward(const salr_adapters_t* A, const salr_adapters_plan_t* P, const uint16_t* X,
                          const uint16_t* base, uint16_t* Y, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(A, P);
  if (rc != SALR_OK) return rc;
  if (P->M == 0) return SALR_OK;
  if (!X || !Y || !aligned16(X) || !aligned16(Y) || !aligned16(base)) return SALR_ERR_INVALID_ARG;
  size_t plan_bytes = 0;
  const salr::AdapterPlan p = lay_out_plan(P->buffer, P->M, P->count, &plan_bytes);
  const Workspace w = lay_out(A->count, A->N, A->K, A->r, P->M, false);
  const size_t out_bytes = (size_t)P->M * A->N * 2, each = (size_t)A->count * A->r * 2;
  if (!writes_apart({{Y, out_bytes}, {ws, w.total}},
                    {{X, (size_t)P->M * A->K * 2}, {base == Y ? nullptr : base, out_bytes}, {A->a, each * A->K},
                     {A->b, each * A->N}, {A->ranks, (size_t)A->count * 4}, {A->scales, (size_t)A->count * 4},
                     {P->buffer, plan_bytes}}))
    return SALR_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return SALR_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const salr::AdapterCommon c{p, A->ranks, A->scales, A->r};
  char* at = static_cast<char*>(ws);
  salr::AdapterDown d{X, A->a, reinterpret_cast<float*>(at + w.t), A->K, 0, 0};
  cut(&d, 1, p, A->r);
  if (const int e = status(launch_down(c, &d, 1, s))) return e;
  uint16_t* planes = nullptr;
  if (p.tile == salr::kAdapterLargeTile) {
    planes = reinterpret_cast<uint16_t*>(at + w.planes);
    const salr::AdapterFinish f{d.T, planes, d.splits};
    if (const int e = status(salr::launch_adapter_finish(c, &f, 1, s))) return e;
  }
  const salr::AdapterUp u{d.T, planes, A->b, base, Y, A->N, d.splits, up_slices(A->N, p)};
  return status(salr::launch_adapter_up(c, u, s));
}

int salr_adapters_backward(const salr_adapters_t* A, const salr_adapters_plan_t* P, const uint16_t* X,
                           const uint16_t* dY, const uint16_t* base, uint16_t* dX, float* dA, float* dB, void* ws,
                           size_t ws_bytes, void* stream) {
  const int rc = check(A, P);
  if (rc != SALR_OK) return rc;
  if (A->N % 8 != 0) return SALR_ERR_UNSUPPORTED;
  if (!dA || !dB || !aligned16(dA) || !aligned16(dB)) return SALR_ERR_INVALID_ARG;
  if (P->M > 0 && (!X || !dY)) return SALR_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(dY) || !aligned16(base) || !aligned16(dX)) return SALR_ERR_INVALID_ARG;
  size_t plan_bytes = 0;
  const salr::AdapterPlan p = lay_out_plan(P->buffer, P->M, P->count, &plan_bytes);
  const Workspace w = lay_out(A->count, A->N, A->K, A->r, P->M, true);
  const size_t x_bytes = (size_t)P->M * A->K * 2, each = (size_t)A->count * A->r * 2;
  if (!writes_apart({{dX, x_bytes}, {dA, each * A->K * 2}, {dB, each * A->N * 2}, {ws, w.total}},
                    {{X, x_bytes}, {dY, (size_t)P->M * A->N * 2}, {base == dX ? nullptr : base, x_bytes},
                     {A->a, each * A->K}, {A->b, each * A->N}, {A->ranks, (size_t)A->count * 4},
                     {A->scales, (size_t)A->count * 4}, {P->buffer, plan_bytes}}))
    return SALR_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return SALR_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* at = static_cast<char*>(ws);
  const auto floats = [&](size_t o) { return reinterpret_cast<float*>(at + o); };
  const auto halves = [&](size_t o) { return reinterpret_cast<uint16_t*>(at + o); };
  const salr::AdapterCommon c{p, A->ranks, A->scales, A->r};
  uint16_t *t_planes = halves(w.planes), *g_planes = halves(w.planes + w.planes_bytes);
  if (P->M > 0) {
    uint16_t *a_t = halves(w.a), *b_t = halves(w.b);
    if (const int e = status(salr::launch_adapter_transpose(c, A->a, a_t, A->K, A->b, b_t, A->N, s))) return e;
    salr::AdapterDown d[2] = {{X, A->a, floats(w.t), A->K, 0, 0}, {dY, b_t, floats(w.t + w.t_bytes), A->N, 0, 0}};
    cut(d, 2, p, A->r);
    if (const int e = status(launch_down(c, d, 2, s))) return e;
    const salr::AdapterFinish f[2] = {{d[0].T, t_planes, d[0].splits}, {d[1].T, g_planes, d[1].splits}};
    if (const int e = status(salr::launch_adapter_finish(c, f, 2, s))) return e;
    if (dX) {
      const salr::AdapterUp u{nullptr, g_planes, a_t, base, dX, A->K, 0, up_slices(A->K, p)};
      if (const int e = status(salr::launch_adapter_up(c, u, s))) return e;
    }
  }
  return status(salr::launch_adapter_grads(c, {X, g_planes, t_planes, dA, floats(w.parts_a), A->K},
                                           {dY, t_planes, g_planes, dB, floats(w.parts_b), A->N}, s));
}

}  // extern "C"

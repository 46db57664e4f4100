// C ABI around the grouped experts (router, dispatch, combine and their
// gradients) and of the AdamW step: argument validation, plan layout and
// kernel dispatch.  See include/salr.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "salr.h"
#include "salr_api_checks.hpp"
#include "salr_kernels.hpp"

namespace {

constexpr int32_t kMaxExperts = 4096;
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - 65536;  // (int32 rows, with room to round up)
constexpr int64_t kMaxColumns = int64_t(1) << 20;
constexpr int64_t kMaxTensorElements = int64_t(1) << 40;
constexpr int32_t kMaxTensors = 1 << 20;
// Workgroups of one launch: its threads, 8 elements each, stay below 2^32.
constexpr int64_t max_chunks(int64_t chunk) { return ((int64_t(1) << 32) - 1) / (chunk / 8); }

using namespace salr;

size_t type_bytes(int32_t t) { return t == SALR_TYPE_F32 ? 4 : 2; }

bool slots_ok(int64_t T, int32_t k) {
  return T >= 0 && k >= 1 && k <= SALR_MOE_MAX_TOPK && T <= kMaxSlots / k;
}

bool route_ok(int32_t type, int64_t T, int32_t E, int32_t k) {
  return type_ok(type) && E >= 1 && E <= kMaxExperts && slots_ok(T, k) && k <= E;
}

// Every pointer given and 16-byte aligned.
template <size_t n>
bool all_given(const void* const (&p)[n]) {
  for (const void* q : p)
    if (!q || !aligned16(q)) return false;
  return true;
}
template <size_t n>
bool all_aligned(const void* const (&p)[n]) {
  for (const void* q : p)
    if (q && !aligned16(q)) return false;
  return true;
}

size_t dispatch_ws(int64_t n, int32_t E) {
  return align_up((size_t)std::min<int64_t>(salr::kMoeSortChunks, std::max<int64_t>(1, cdiv(n, 1024))) * E * 4, 256);
}

}  // namespace

extern "C" {

int salr_moe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k, int32_t renorm,
                   int32_t* ids, float* weights, void* stream) {
  if (!route_ok(logits_type, T, E, k)) return SALR_ERR_INVALID_ARG;
  if (T == 0) return SALR_OK;
  if (!all_given({logits, ids, weights})) return SALR_ERR_INVALID_ARG;
  const size_t n = (size_t)T * k;
  if (!writes_apart({{ids, n * 4}, {weights, n * 4}}, {{logits, (size_t)T * E * type_bytes(logits_type)}}))
    return SALR_ERR_INVALID_ARG;
  return status(salr::launch_moe_route(logits, logits_type == SALR_TYPE_F32, T, E, k, renorm != 0, ids, weights,
                                       static_cast<hipStream_t>(stream)));
}

int salr_moe_route_backward(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k, int32_t renorm,
                            const int32_t* ids, const float* dweights, void* dlogits, void* stream) {
  if (!route_ok(logits_type, T, E, k)) return SALR_ERR_INVALID_ARG;
  if (T == 0) return SALR_OK;
  if (!all_given({logits, ids, dweights, dlogits})) return SALR_ERR_INVALID_ARG;
  const size_t n = (size_t)T * k, bytes = (size_t)T * E * type_bytes(logits_type);
  if (!writes_apart({{dlogits, bytes}}, {{ids, n * 4}, {dweights, n * 4}, {dlogits == logits ? nullptr : logits, bytes}}))
    return SALR_ERR_INVALID_ARG;
  return status(salr::launch_moe_route_backward(logits, logits_type == SALR_TYPE_F32, T, E, k, renorm != 0, ids,
                                                dweights, dlogits, static_cast<hipStream_t>(stream)));
}

int salr_moe_dispatch_ws_bytes(int64_t T_max, int32_t k, int32_t E, size_t* out) {
  if (!out || !slots_ok(T_max, k) || E < 1 || E > kMaxExperts) return SALR_ERR_INVALID_ARG;
  *out = dispatch_ws(T_max * k, E);
  return SALR_OK;
}

int salr_moe_dispatch(const int32_t* ids, int64_t T, int32_t k, int32_t E, const uint16_t* X, int64_t D,
                      int32_t* expert_offsets, int32_t* rows, int32_t* slots, uint16_t* Xs, void* ws, size_t ws_bytes,
                      void* stream) {
  if (!slots_ok(T, k) || E < 1 || E > kMaxExperts) return SALR_ERR_INVALID_ARG;
  if (!expert_offsets || (T > 0 && (!ids || !rows || !X != !Xs))) return SALR_ERR_INVALID_ARG;
  if (T > 0 && X && (D < 1 || D > kMaxColumns)) return SALR_ERR_INVALID_ARG;
  if (!all_aligned({ids, X, expert_offsets, rows, slots, Xs})) return SALR_ERR_INVALID_ARG;
  const size_t n = (size_t)T * k, row = X ? (size_t)D * 2 : 0;
  const Span w{ws, dispatch_ws(n, E)};
  if (!writes_apart({{expert_offsets, ((size_t)E + 1) * 4}, {rows, n * 4}, {slots, n * 4}, {Xs, n * row}, w},
                    {{ids, n * 4}, {X, T * row}}))
    return SALR_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < w.bytes) return SALR_ERR_WORKSPACE;
  salr::MoeDispatchArgs a{};
  a.ids = ids;
  a.X = T > 0 ? X : nullptr;
  a.Xs = Xs;
  a.off = expert_offsets;
  a.rows = rows;
  a.slots = slots;
  a.hist = static_cast<uint32_t*>(ws);
  a.D = D;
  a.n = (int32_t)(T * k);
  a.k = k;
  a.E = E;
  a.chunk = salr::moe_sort_chunk(a.n);
  a.chunks = (int32_t)std::max<int64_t>(1, cdiv(a.n, a.chunk));
  return status(salr::launch_moe_dispatch(a, static_cast<hipStream_t>(stream)));
}

int salr_moe_combine(const uint16_t* Ys, int64_t R, const int32_t* rows, const float* weights, const uint16_t* base,
                     int64_t T, int32_t k, int64_t D, uint16_t* Y, void* stream) {
  if (!slots_ok(T, k) || R < 0 || R > kMaxSlots || D < 1 || D > kMaxColumns) return SALR_ERR_INVALID_ARG;
  if (T == 0) return SALR_OK;
  if (!rows || !Y || (R > 0 && !Ys)) return SALR_ERR_INVALID_ARG;
  if (!all_aligned({Ys, rows, weights, base, Y})) return SALR_ERR_INVALID_ARG;
  const size_t n = (size_t)T * k, row = (size_t)D * 2;
  if (!writes_apart({{Y, T * row}},
                    {{Ys, R * row}, {rows, n * 4}, {weights, n * 4}, {base == Y ? nullptr : base, T * row}}))
    return SALR_ERR_INVALID_ARG;
  salr::MoeCombineArgs a{};
  a.Ys = Ys;
  a.rows = rows;
  a.weights = weights;
  a.base = base;
  a.out = Y;
  a.R = R;
  a.T = T;
  a.D = D;
  a.k = k;
  return status(salr::launch_moe_combine(a, static_cast<hipStream_t>(stream)));
}

int salr_moe_combine_backward(const uint16_t* dY, const uint16_t* Ys, int64_t R, const int32_t* rows,
                              const float* weights, int64_t T, int32_t k, int64_t D, uint16_t* dYs, float* dweights,
                              void* stream) {
  if (!slots_ok(T, k) || R < 0 || R > kMaxSlots || D < 1 || D > kMaxColumns) return SALR_ERR_INVALID_ARG;
  if (T == 0 || (!dYs && !dweights)) return SALR_OK;
  if (!dY || !rows || (R > 0 && dweights && !Ys)) return SALR_ERR_INVALID_ARG;
  if (!all_aligned({dY, Ys, rows, weights, dYs, dweights})) return SALR_ERR_INVALID_ARG;
  const size_t n = (size_t)T * k, row = (size_t)D * 2;
  const Span ys{Ys, R * row};
  if (!writes_apart({{dYs, R * row}, {dweights, n * 4}},
                    {{dY, T * row}, {rows, n * 4}, {weights, n * 4}, {dYs == Ys ? nullptr : Ys, R * row}}) ||
      !apart({dweights, n * 4}, ys))
    return SALR_ERR_INVALID_ARG;
  salr::MoeCombineArgs a{};
  a.dY = dY;
  a.Ys = Ys;
  a.rows = rows;
  a.weights = weights;
  a.out = dYs;
  a.dweights = dweights;
  a.R = R;
  a.T = T;
  a.D = D;
  a.k = k;
  return status(salr::launch_moe_combine_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ----------------------------------------------------------------------------
// AdamW: the plan's table is the tensor records, then the chunk list.
namespace {

static_assert(salr::kAdamwSmallChunk % SALR_ADAMW_BLOCK == 0 && salr::kAdamwLargeChunk % SALR_ADAMW_BLOCK == 0 &&
                  salr::kAdamwLargeChunk >= salr::kAdamwSmallChunk,
              "a chunk holds whole 8-bit runs, and the small one sizes the table");

size_t table_records_bytes(int32_t count) { return align_up((size_t)count * sizeof(salr::AdamwTensor), 256); }
size_t table_bytes_for(int32_t count, int64_t chunks) {
  return table_records_bytes(count) + align_up((size_t)std::max<int64_t>(chunks, 1) * sizeof(salr::AdamwChunk), 256);
}

// Validates the records and, with `table` (host memory of table_bytes_for),
// writes the plan's table.  0, or a negative status.
int adamw_fill(const salr_adamw_tensor_t* t, int32_t count, int32_t p_type, int32_t g_type, bool state8, bool master,
               unsigned char* table, Range* ranges) {
  size_t nw = 0, nr = 0;
  Range* read = ranges + (size_t)count * 6;
  salr::AdamwTensor* rec = reinterpret_cast<salr::AdamwTensor*>(table);
  salr::AdamwChunk* chunk = reinterpret_cast<salr::AdamwChunk*>(table + table_records_bytes(count));
  const size_t pb = p_type == SALR_TYPE_F32 ? 4 : 2, gb = g_type == SALR_TYPE_F32 ? 4 : 2, sb = state8 ? 1 : 4;
  for (int32_t i = 0; i < count; ++i) {
    const salr_adamw_tensor_t& q = t[i];
    rec[i] = salr::AdamwTensor{q.p, q.g, q.m, q.v, q.m_scale, q.v_scale, q.master, q.n};
    if (q.n == 0) continue;
    if (!all_given({q.p, q.g, q.m, q.v})) return SALR_ERR_INVALID_ARG;
    if (state8 && (!q.m_scale || !q.v_scale || !aligned4(q.m_scale) || !aligned4(q.v_scale))) return SALR_ERR_INVALID_ARG;
    if ((q.master != nullptr) != master || !aligned16(q.master)) return SALR_ERR_INVALID_ARG;
    const auto add = [](Range* to, size_t& n, const void* p, size_t bytes) {
      to[n++] = Range{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes};
    };
    const size_t n = (size_t)q.n, runs = (size_t)cdiv(q.n, SALR_ADAMW_BLOCK);
    add(ranges, nw, q.p, n * pb);
    add(ranges, nw, q.m, n * sb);
    add(ranges, nw, q.v, n * sb);
    if (state8) {
      add(ranges, nw, q.m_scale, runs * 4);
      add(ranges, nw, q.v_scale, runs * 4);
    }
    if (master) add(ranges, nw, q.master, n * 4);
    add(read, nr, q.g, n * gb);
    for (int64_t c = 0; c < cdiv(q.n, salr::adamw_chunk(state8, master)); ++c) *chunk++ = salr::AdamwChunk{i, (int32_t)c};
  }
  return overlaps(ranges, nw, read, nr) ? SALR_ERR_INVALID_ARG : SALR_OK;
}

// The chunks of `count` tensors, or -1 (a tensor too long, or too many).
template <class F>
int64_t adamw_chunks(int32_t count, int64_t chunk, F n) {
  int64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (n(i) < 0 || n(i) >= kMaxTensorElements) return -1;
    chunks += cdiv(n(i), chunk);
    if (chunks > max_chunks(chunk)) return -1;
  }
  return chunks;
}

// The chunks in small ones, which size the table, where both kinds can be
// launched, or -1.
template <class F>
int64_t adamw_small_chunks(int32_t count, F n) {
  const int64_t chunks = adamw_chunks(count, salr::kAdamwSmallChunk, n);
  return adamw_chunks(count, salr::kAdamwLargeChunk, n) < 0 ? -1 : chunks;
}

int adamw_step(const salr_adamw_plan_t* plan, const salr_adamw_step_args_t* args, bool random, uint32_t seed,
               const float* dyn, void* stream) {
  if (!plan || !args) return SALR_ERR_INVALID_ARG;
  if (!plan->table || !aligned16(plan->table) || plan->count < 0 || plan->count > kMaxTensors || plan->chunks < 0 ||
      plan->chunks > max_chunks(salr::adamw_chunk(plan->state_type == SALR_STATE_8BIT, plan->has_master != 0)) ||
      !type_ok(plan->p_type) || !type_ok(plan->g_type) ||
      (plan->state_type != SALR_STATE_F32 && plan->state_type != SALR_STATE_8BIT) ||
      (plan->has_master && plan->p_type != SALR_TYPE_BF16))
    return SALR_ERR_INVALID_ARG;
  const auto nonneg = [](double v) { return v >= 0 && std::isfinite(v); };
  if (!nonneg(args->eps) || !nonneg(args->weight_decay)) return SALR_ERR_INVALID_ARG;
  if (!(args->beta1 >= 0 && args->beta1 < 1) || !(args->beta2 >= 0 && args->beta2 < 1)) return SALR_ERR_INVALID_ARG;
  if (!dyn && (args->step < 1 || !nonneg(args->lr))) return SALR_ERR_INVALID_ARG;
  if (!aligned4(dyn)) return SALR_ERR_INVALID_ARG;
  salr::AdamwArgs a{};
  a.tensors = static_cast<const salr::AdamwTensor*>(plan->table);
  a.chunks = reinterpret_cast<const salr::AdamwChunk*>(static_cast<const char*>(plan->table) +
                                                       table_records_bytes(plan->count));
  a.n_chunks = plan->chunks;
  a.dyn = dyn;
  a.beta1 = (float)args->beta1;
  a.beta2 = (float)args->beta2;
  a.rest1 = (float)(1.0 - args->beta1);
  a.rest2 = (float)(1.0 - args->beta2);
  a.eps = (float)args->eps;
  a.weight_decay = (float)args->weight_decay;
  a.seed = seed;
  a.step = (float)args->step;
  if (!dyn) {
    a.grad_scale = (float)args->grad_scale;
    a.decay = (float)(1.0 - args->lr * args->weight_decay);
    a.rate = (float)(args->lr / (1.0 - std::pow(args->beta1, (double)args->step)));
    a.inv_sqrt_bias2 = (float)(1.0 / std::sqrt(1.0 - std::pow(args->beta2, (double)args->step)));
  }
  return status(salr::launch_adamw(a, plan->p_type == SALR_TYPE_F32, plan->g_type == SALR_TYPE_F32,
                                   plan->state_type == SALR_STATE_8BIT, plan->has_master != 0,
                                   random, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int salr_adamw_plan_bytes(const int64_t* n, int32_t count, size_t* out) {
  if (!out || count < 0 || count > kMaxTensors || (count > 0 && !n)) return SALR_ERR_INVALID_ARG;
  const int64_t chunks = adamw_small_chunks(count, [&](int32_t i) { return n[i]; });
  if (chunks < 0) return SALR_ERR_INVALID_ARG;
  *out = table_bytes_for(count, chunks);
  return SALR_OK;
}

int salr_adamw_plan(const salr_adamw_tensor_t* tensors, int32_t count, int32_t p_type, int32_t g_type,
                    int32_t state_type, void* table, size_t table_bytes, salr_adamw_plan_t* out, void* stream) {
  if (!out || count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SALR_ERR_INVALID_ARG;
  if (!type_ok(p_type) || !type_ok(g_type)) return SALR_ERR_INVALID_ARG;
  if (state_type != SALR_STATE_F32 && state_type != SALR_STATE_8BIT) return SALR_ERR_INVALID_ARG;
  const bool state8 = state_type == SALR_STATE_8BIT;
  bool master = false;
  for (int32_t i = 0; i < count && !master; ++i) master = tensors[i].n > 0 && tensors[i].master != nullptr;
  const auto size = [&](int32_t i) { return tensors[i].n; };
  if (adamw_small_chunks(count, size) < 0) return SALR_ERR_INVALID_ARG;  // (as the table's size says)
  const int64_t chunks = adamw_chunks(count, salr::adamw_chunk(state8, master), size);
  if (master && p_type != SALR_TYPE_BF16) return SALR_ERR_INVALID_ARG;
  const size_t bytes = table_bytes_for(count, chunks);
  unsigned char* host = new (std::nothrow) unsigned char[bytes];
  Range* ranges = new (std::nothrow) Range[(size_t)count * 7 + 1];
  int rc = host && ranges ? SALR_OK : SALR_ERR_UNSUPPORTED;
  if (rc == SALR_OK) {
    std::memset(host, 0, bytes);
    rc = adamw_fill(tensors, count, p_type, g_type, state8, master, host, ranges);
  }
  delete[] ranges;
  // (every argument check above comes before the buffer's)
  if (rc == SALR_OK && (!table || !aligned16(table) || table_bytes < bytes)) rc = SALR_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rc == SALR_OK) {
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &cap) != hipSuccess) rc = SALR_ERR_HIP;
    else if (cap != hipStreamCaptureStatusNone) rc = SALR_ERR_UNSUPPORTED;
  }
  if (rc == SALR_OK && (hipMemcpyAsync(table, host, bytes, hipMemcpyHostToDevice, s) != hipSuccess ||
                        hipStreamSynchronize(s) != hipSuccess))
    rc = SALR_ERR_HIP;
  delete[] host;
  if (rc != SALR_OK) return rc;
  out->table = table;
  out->chunks = chunks;
  out->count = count;
  out->p_type = p_type;
  out->g_type = g_type;
  out->state_type = state_type;
  out->has_master = master ? 1 : 0;
  return SALR_OK;
}

int salr_adamw_step(const salr_adamw_plan_t* plan, const salr_adamw_step_args_t* args, const float* dyn,
                    void* stream) {
  return adamw_step(plan, args, false, 0, dyn, stream);
}

int salr_adamw_step_random(const salr_adamw_plan_t* plan, const salr_adamw_step_args_t* args, uint32_t seed,
                           const float* dyn, void* stream) {
  return adamw_step(plan, args, true, seed, dyn, stream);
}

}  // extern "C"

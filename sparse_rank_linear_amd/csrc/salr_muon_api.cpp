// C ABI of the orthogonalised step: argument validation, plan layout and
// dispatch by class.  See include/salr.h for the contract.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "salr.h"
#include "salr_api_checks.hpp"
#include "salr_muon.hpp"

namespace {

using namespace salr;

constexpr int32_t kMaxMatrices = 1 << 20;
constexpr int64_t kMaxSide = int64_t(1) << 30;
constexpr int64_t kMaxMatrix = int64_t(1) << 29;   // elements of one: the kernels' byte offsets have 32 bits
constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int64_t kMaxChunks = (int64_t(1) << 22) - 1;  // of up to 1024 threads: a launch takes 2^32
constexpr int32_t kMaxLarge = 65535;  // matrices of a class that has a grid dimension for them
constexpr double kMinEps = 1e-12;     // far above |u| of elements whose squares a float does not hold
static_assert(SALR_MUON_CLASSES == kMuonClasses, "a plan counts every class");

int class_of(int64_t s) {
  int c = 0;
  while (16 * kMuonTiles[c] < s) ++c;
  return c;
}

struct Shape {
  int64_t s, L;
  int cls;
  int32_t chunk, chunks;
};

// Elements of a chunk of each class.
struct Cut {
  int64_t per[kMuonClasses];
};

// The shape of one matrix; chunks 0 for an empty one.
Shape shape_of(int64_t rows, int64_t cols, const Cut& cut) {
  Shape q{};
  q.s = std::min(rows, cols);
  q.L = std::max(rows, cols);
  if (q.s == 0) return q;
  q.cls = class_of(q.s);
  const int64_t kb = muon_stage(kMuonTiles[q.cls]);
  // (each chunk writes one s x s sum, so it has s columns at least)
  const int64_t chunk = std::min(cdiv(q.L, kb), cdiv(std::max(q.s, cdiv(cut.per[q.cls], q.s)), kb)) * kb;
  q.chunk = (int32_t)chunk;
  q.chunks = (int32_t)cdiv(q.L, chunk);
  return q;
}

// How the matrices are cut, and the chunks that makes in all.  Enough
// workgroups for the CUs, then fewer and longer ones; from ten tiles on a CU
// holds one workgroup at a time, and a few more than there are CUs would take
// half as long again (253 x 67584 columns in 267 chunks 139 us, in 237 ones 100).
// INVALID_ARG, UNSUPPORTED (a short side over the limit, too many pieces) or 0.
constexpr int64_t kCus = 256;
template <class R, class C>
int survey(int32_t count, R rows, C cols, Cut* cut, int64_t* chunks) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (rows(i) < 0 || cols(i) < 0 || rows(i) > kMaxSide || cols(i) > kMaxSide) return SALR_ERR_INVALID_ARG;
    if (std::min(rows(i), cols(i)) > SALR_MUON_MAX_SIDE || rows(i) * cols(i) >= kMaxMatrix) return SALR_ERR_UNSUPPORTED;
    total += rows(i) * cols(i);
    if (total > kMaxElements) return SALR_ERR_UNSUPPORTED;
  }
  for (int64_t& per : cut->per) per = std::min<int64_t>(131072, std::max<int64_t>(8192, total / 1024));
  const auto chunks_of = [&](int64_t (&n)[kMuonClasses]) {
    for (int64_t& v : n) v = 0;
    for (int32_t i = 0; i < count; ++i) {
      const Shape q = shape_of(rows(i), cols(i), *cut);
      n[q.cls] += q.chunks;
    }
  };
  int64_t n[kMuonClasses], matrices[kMuonClasses] = {};
  for (int32_t i = 0; i < count; ++i) {
    const Shape q = shape_of(rows(i), cols(i), *cut);
    matrices[q.cls] += q.chunks > 0;
  }
  for (int cls = kMuonLdsClasses; cls < kMuonClasses; ++cls)
    if (matrices[cls] > kMaxLarge) return SALR_ERR_UNSUPPORTED;
  chunks_of(n);
  for (int cls = 0; cls < kMuonClasses; ++cls)
    for (int k = 0; k < 16 && kMuonTiles[cls] >= 10 && n[cls] > kCus && n[cls] < 2 * kCus; ++k) {
      cut->per[cls] = std::max(cut->per[cls], (int64_t)256 * 16 * kMuonTiles[cls]) * 17 / 16;
      chunks_of(n);
    }
  *chunks = 0;
  for (int64_t v : n) *chunks += v;
  return *chunks > kMaxChunks ? SALR_ERR_UNSUPPORTED : SALR_OK;
}

size_t records_bytes(int64_t count) { return align_up((size_t)count * sizeof(MuonMatrix), 256); }
size_t list_bytes(int64_t chunks) { return align_up((size_t)chunks * sizeof(MuonChunk), 256); }

// One matrix's own memory in the table: its pieces' products, Q, and for
// large classes six matrices to iterate on.
struct Own {
  size_t parts, q, work;
};
Own own_bytes(const Shape& q) {
  if (q.chunks == 0) return {0, 0, 0};
  const size_t S = 16 * (size_t)kMuonTiles[q.cls];
  return {align_up((size_t)q.chunks * muon_lower(kMuonTiles[q.cls]) * 2048, 256), align_up(S * S * 4, 256),
          q.cls < kMuonLdsClasses ? 0 : S * S * 8 * 6};
}

template <class R, class C>
size_t table_bytes_for(int32_t count, R rows, C cols, const Cut& cut, int64_t chunks) {
  size_t bytes = records_bytes(count) + list_bytes(chunks);
  for (int32_t i = 0; i < count; ++i) {
    const Own o = own_bytes(shape_of(rows(i), cols(i), cut));
    bytes += o.parts + o.q + o.work;
  }
  return std::max<size_t>(bytes, 256);
}

}  // namespace

extern "C" {

int salr_muon_plan_bytes(const int64_t* rows, const int64_t* cols, int32_t count, size_t* out) {
  if (!out || count < 0 || count > kMaxMatrices || (count > 0 && (!rows || !cols))) return SALR_ERR_INVALID_ARG;
  const auto r = [&](int32_t i) { return rows[i]; };
  const auto c = [&](int32_t i) { return cols[i]; };
  Cut cut;
  int64_t chunks = 0;
  if (const int e = survey(count, r, c, &cut, &chunks)) return e;
  *out = table_bytes_for(count, r, c, cut, chunks);
  return SALR_OK;
}

int salr_muon_plan(const salr_muon_tensor_t* tensors, int32_t count, int32_t p_type, int32_t g_type, void* table,
                   size_t table_bytes, salr_muon_plan_t* out, void* stream) {
  if (!out || count < 0 || count > kMaxMatrices || (count > 0 && !tensors)) return SALR_ERR_INVALID_ARG;
  if (!type_ok(p_type) || !type_ok(g_type)) return SALR_ERR_INVALID_ARG;
  const auto rows = [&](int32_t i) { return tensors[i].rows; };
  const auto cols = [&](int32_t i) { return tensors[i].cols; };
  Cut cut;
  int64_t chunks = 0;
  if (const int e = survey(count, rows, cols, &cut, &chunks)) return e;
  const auto live = [&](int32_t i) { return tensors[i].rows > 0 && tensors[i].cols > 0; };
  bool master = false;
  for (int32_t i = 0; i < count && !master; ++i) master = live(i) && tensors[i].master != nullptr;
  if (master && p_type != SALR_TYPE_BF16) return SALR_ERR_INVALID_ARG;
  const size_t bytes = table_bytes_for(count, rows, cols, cut, chunks);
  const size_t head = records_bytes(count) + list_bytes(chunks);
  unsigned char* host = new (std::nothrow) unsigned char[std::max<size_t>(head, 1)];
  Range* ranges = new (std::nothrow) Range[(size_t)count * 4 + 2];
  int rc = host && ranges ? SALR_OK : SALR_ERR_UNSUPPORTED;
  salr_muon_plan_t plan{};
  if (rc == SALR_OK) {
    std::memset(host, 0, head);
    MuonMatrix* rec = reinterpret_cast<MuonMatrix*>(host);
    MuonChunk* list = reinterpret_cast<MuonChunk*>(host + records_bytes(count));
    size_t nw = 0, nr = 0, at = head;
    Range* read = ranges + (size_t)count * 3 + 1;
    const size_t pb = p_type == SALR_TYPE_F32 ? 4 : 2, gb = g_type == SALR_TYPE_F32 ? 4 : 2;
    const uintptr_t base = reinterpret_cast<uintptr_t>(table);  // (may be null: refused below)
    int32_t k = 0;
    for (int cls = 0; cls < kMuonClasses && rc == SALR_OK; ++cls) {
      for (int32_t i = 0; i < count; ++i) {
        const Shape q = shape_of(rows(i), cols(i), cut);
        if (q.chunks == 0 || q.cls != cls) continue;
        const salr_muon_tensor_t& t = tensors[i];
        const bool ok = t.p && t.g && t.m && aligned16(t.p) && aligned16(t.g) && aligned16(t.m) &&
                        (t.master != nullptr) == master && aligned16(t.master) && std::isfinite((float)t.lr_scale);
        if (!ok) {
          rc = SALR_ERR_INVALID_ARG;
          break;
        }
        const size_t n = (size_t)t.rows * t.cols;
        const auto add = [](Range* to, size_t& m, const void* p, size_t b) {
          to[m++] = Range{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + b};
        };
        add(ranges, nw, t.p, n * pb);
        add(ranges, nw, t.m, n * 4);
        if (master) add(ranges, nw, t.master, n * 4);
        add(read, nr, t.g, n * gb);
        const Own o = own_bytes(q);
        MuonMatrix& m = rec[k];
        m.p = t.p;
        m.g = t.g;
        m.m = t.m;
        m.master = t.master;
        m.parts = reinterpret_cast<double*>(base + at);
        m.q = reinterpret_cast<float*>(base + at + o.parts);
        m.work = o.work ? reinterpret_cast<double*>(base + at + o.parts + o.q) : nullptr;
        at += o.parts + o.q + o.work;
        m.L = q.L;
        m.s = (int32_t)q.s;
        m.wide = t.cols >= t.rows;
        m.chunks = q.chunks;
        m.chunk = q.chunk;
        m.lr_scale = (float)t.lr_scale;
        for (int32_t c = 0; c < q.chunks; ++c) *list++ = MuonChunk{k, c};
        plan.matrices[cls] += 1;
        plan.chunks[cls] += q.chunks;
        ++k;
      }
    }
    // (a step works in the table too)
    if (table) ranges[nw++] = Range{reinterpret_cast<uintptr_t>(table), reinterpret_cast<uintptr_t>(table) + bytes};
    if (rc == SALR_OK && overlaps(ranges, nw, read, nr)) rc = SALR_ERR_INVALID_ARG;
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
  if (rc == SALR_OK && head > 0 &&
      (hipMemcpyAsync(table, host, head, hipMemcpyHostToDevice, s) != hipSuccess ||
       hipStreamSynchronize(s) != hipSuccess))
    rc = SALR_ERR_HIP;
  delete[] host;
  if (rc != SALR_OK) return rc;
  plan.table = table;
  plan.count = count;
  plan.p_type = p_type;
  plan.g_type = g_type;
  plan.has_master = master ? 1 : 0;
  *out = plan;
  return SALR_OK;
}

int salr_muon_step(const salr_muon_plan_t* plan, const salr_muon_step_args_t* args, const float* dyn, void* stream) {
  if (!plan || !args) return SALR_ERR_INVALID_ARG;
  if (!plan->table || !aligned16(plan->table) || plan->count < 0 || plan->count > kMaxMatrices ||
      !type_ok(plan->p_type) || !type_ok(plan->g_type) || (plan->has_master && plan->p_type != SALR_TYPE_BF16))
    return SALR_ERR_INVALID_ARG;
  int64_t matrices = 0, chunks = 0;
  for (int c = 0; c < kMuonClasses; ++c) {
    if (plan->matrices[c] < 0 || plan->chunks[c] < 0) return SALR_ERR_INVALID_ARG;
    if (c >= kMuonLdsClasses && plan->matrices[c] > kMaxLarge) return SALR_ERR_INVALID_ARG;
    matrices += plan->matrices[c];
    chunks += plan->chunks[c];
  }
  if (matrices > plan->count || chunks > kMaxChunks) return SALR_ERR_INVALID_ARG;
  const auto nonneg = [](double v) { return v >= 0 && std::isfinite((float)v); };
  if (!nonneg(args->weight_decay) || !nonneg(args->eps) || args->eps < kMinEps) return SALR_ERR_INVALID_ARG;
  if (!(args->momentum >= 0 && args->momentum < 1) || args->steps < 1 || args->steps > kMuonMaxSteps)
    return SALR_ERR_INVALID_ARG;
  for (double v : {args->a, args->b, args->c})
    if (!std::isfinite((float)v)) return SALR_ERR_INVALID_ARG;
  if (!dyn && (!nonneg(args->lr) || !std::isfinite((float)args->grad_scale))) return SALR_ERR_INVALID_ARG;
  if (!aligned4(dyn)) return SALR_ERR_INVALID_ARG;
  MuonArgs a{};
  a.matrices = static_cast<const MuonMatrix*>(plan->table);
  a.chunks = reinterpret_cast<const MuonChunk*>(static_cast<const char*>(plan->table) + records_bytes(plan->count));
  a.dyn = dyn;
  a.lr = (float)args->lr;
  a.grad_scale = (float)args->grad_scale;
  a.momentum = (float)args->momentum;
  a.weight_decay = (float)args->weight_decay;
  a.eps = args->eps;
  a.a = args->a;
  a.b = args->b;
  a.c = args->c;
  a.steps = args->steps;
  a.nesterov = args->nesterov != 0;
  a.p_f32 = plan->p_type == SALR_TYPE_F32;
  a.g_f32 = plan->g_type == SALR_TYPE_F32;
  a.master = plan->has_master != 0;
  const auto apply = a.p_f32 ? launch_muon_apply_f32 : a.master ? launch_muon_apply_master : launch_muon_apply_bf16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int32_t m0 = 0;
  int64_t c0 = 0;
  for (int c = 0; c < kMuonClasses; ++c) {
    if (plan->matrices[c] > 0) {
      hipError_t e = launch_muon_gram(a, c, c0, plan->chunks[c], s);
      if (e == hipSuccess) e = launch_muon_iterate(a, c, m0, plan->matrices[c], s);
      if (e == hipSuccess) e = apply(a, c, c0, plan->chunks[c], s);
      if (e != hipSuccess) return SALR_ERR_HIP;
    }
    m0 += plan->matrices[c];
    c0 += plan->chunks[c];
  }
  return SALR_OK;
}

}  // extern "C"

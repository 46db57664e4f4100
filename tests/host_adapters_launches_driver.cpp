// Host-side driver for tests/test_adapters_launches.py: what
// salr_adapters_api.cpp hands to the launchers, for sizes up to the largest that
// the entry points take (whose tensors no card holds).  The launchers are
// stand-ins that check a launch's size and what the kernels write, so no call
// here reaches a device.  Prints "ok" and exits 0 when every expectation holds.
#include <algorithm>
#include <cstdint>
#include <cstdio>

#include "salr.h"
#include "salr_adapters.hpp"

namespace {

constexpr int64_t kLaunchThreads = int64_t(1) << 32;  // a launch has fewer
int failures = 0, launches = 0;
int64_t M, K, N, rank, contracted;
char* const ws = reinterpret_cast<char*>(uintptr_t(1) << 60);
size_t ws_bytes;

void expect(bool ok, const char* what) {
  if (ok) return;
  std::fprintf(stderr, "%s: M %lld, r %lld, K %lld, N %lld\n", what, (long long)M, (long long)rank, (long long)K,
               (long long)N);
  ++failures;
}

// [p, p + bytes) lies in the workspace.
void inside(const void* p, int64_t bytes, const char* what) {
  const char* q = static_cast<const char*>(p);
  expect(q >= ws && q + bytes <= ws + ws_bytes, what);
}

int64_t groups_of(int64_t r) { return (r + 79) / 80; }

}  // namespace

namespace salr {

hipError_t launch_adapter_plan(const int32_t*, const AdapterPlan&, hipStream_t) { return hipSuccess; }

hipError_t launch_adapter_down(const AdapterCommon& c, const AdapterDown* jobs, int n, hipStream_t) {
  ++launches;
  int64_t pieces = 0;
  for (int q = 0; q < n; ++q) {
    pieces += jobs[q].splits;
    contracted += jobs[q].K;
    expect(jobs[q].splits >= 1 && (int64_t)jobs[q].splits * jobs[q].cols >= jobs[q].K &&
               (int64_t)(jobs[q].splits - 1) * jobs[q].cols < jobs[q].K,
           "pieces");
    inside(jobs[q].T, (int64_t)jobs[q].splits * M * rank * 4, "T");
    if (q > 0) expect(jobs[q - 1].T + (int64_t)jobs[q - 1].splits * M * rank <= jobs[q].T, "T and G");
  }
  expect((int64_t)c.plan.max_tiles * groups_of(c.r) * pieces * 256 < kLaunchThreads, "down");
  return hipSuccess;
}
hipError_t launch_adapter_finish(const AdapterCommon& c, const AdapterFinish* jobs, int n, hipStream_t) {
  for (int q = 0; q < n; ++q) inside(jobs[q].planes, 3 * M * rank * 2, "planes");
  expect((int64_t)c.plan.max_tiles * 256 < kLaunchThreads, "finish");
  return hipSuccess;
}
hipError_t launch_adapter_up(const AdapterCommon& c, const AdapterUp& u, hipStream_t) {
  expect((int64_t)c.plan.max_tiles * u.slices * 256 < kLaunchThreads, "up");
  return hipSuccess;
}
hipError_t launch_adapter_transpose(const AdapterCommon& c, const uint16_t*, uint16_t* at, int64_t, const uint16_t*,
                                    uint16_t* bt, int64_t, hipStream_t) {
  inside(at, (int64_t)c.plan.count * rank * K * 2, "A transposed");
  inside(bt, (int64_t)c.plan.count * rank * N * 2, "B transposed");
  return hipSuccess;
}
hipError_t launch_adapter_grads(const AdapterCommon& c, const AdapterGrad& a, const AdapterGrad& b, hipStream_t) {
  const int64_t parts = std::min<int64_t>(c.plan.max_chunks, 2 * M / c.plan.chunk);
  inside(a.parts, parts * rank * K * 4, "dA's sums");
  inside(b.parts, parts * rank * N * 4, "dB's sums");
  return hipSuccess;
}

}  // namespace salr

int main() {
  const int64_t batches[] = {1, 16, 17, 1000, 1024, 1025, 4099, 8192, 65536, 1 << 20, (1 << 27) - 1, 1 << 27};
  const int64_t sides[] = {8, 264, 4096, 11008, 1 << 20};
  for (int64_t count : {1, 7, 4096})
    for (int64_t m : batches)
      for (int64_t r : {8, 32, 40, 80, 88, 160, 168, 240, 248, 256})
        for (int64_t k : sides)
          for (int64_t n : sides)
            for (int backward : {0, 1}) {
              M = m, K = k, N = n, rank = r, launches = 0, contracted = 0;
              const auto at = [](int i) { return (void*)((uintptr_t(1) << 61) + (uintptr_t(i) << 57)); };
              salr_adapters_t A{};
              A.count = (int32_t)count;
              A.r = (int32_t)r;
              A.N = n;
              A.K = k;
              A.a = static_cast<uint16_t*>(at(0));
              A.b = static_cast<uint16_t*>(at(1));
              salr_adapters_plan_t plan{at(2), m, (int32_t)count};
              if (salr_adapters_ws_bytes((int32_t)count, n, k, (int32_t)r, m, backward, &ws_bytes) != SALR_OK) {
                expect(false, "workspace");
                continue;
              }
              const uint16_t *X = static_cast<uint16_t*>(at(3)), *dY = static_cast<uint16_t*>(at(4));
              uint16_t* out = static_cast<uint16_t*>(at(5));
              const int rc = backward ? salr_adapters_backward(&A, &plan, X, dY, nullptr, out, static_cast<float*>(at(6)),
                                                               static_cast<float*>(at(7)), ws, ws_bytes, nullptr)
                                      : salr_adapters_forward(&A, &plan, X, nullptr, out, ws, ws_bytes, nullptr);
              expect(rc == SALR_OK, "status");
              expect(contracted == (backward ? k + n : k), "contractions");
              // (small launches stay together)
              if (m <= (1 << 20)) expect(launches == 1, "launches");
            }
  if (failures) return 1;
  std::puts("ok");
  return 0;
}

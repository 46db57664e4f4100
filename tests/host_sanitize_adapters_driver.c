/* Host-side driver for tests/test_adapters_sanitizers.py: walks the argument
 * validation, size arithmetic and plan layout of the adapters of many requests
 * and of the orthogonalised step, which run on the host before any device
 * work.  Built with AddressSanitizer and UndefinedBehaviorSanitizer around
 * salr_adapters_api.cpp and salr_muon_api.cpp; no call here reaches the device.
 * Prints "ok" and exits 0 when every expectation holds. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "salr.h"

static int failures = 0;

#define EXPECT(cond)                                                                 \
  do {                                                                               \
    if (!(cond)) {                                                                   \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                                    \
    }                                                                                \
  } while (0)

/* Made-up device addresses, 16-byte aligned, never dereferenced. */
static void* at(uint64_t a) { return (void*)(uintptr_t)a; }

static void adapters(void) {
  size_t n = 0;
  EXPECT(salr_adapters_plan_bytes(INT64_C(1) << 27, SALR_ADAPTERS_MAX, &n) == SALR_OK);
  EXPECT(n >= (size_t)(INT64_C(4) << 27));
  EXPECT(salr_adapters_plan_bytes(INT64_MAX, 1, &n) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_adapters_ws_bytes(SALR_ADAPTERS_MAX, 1 << 20, 1 << 20, 256, INT64_C(1) << 27, 1, &n) == SALR_OK);
  EXPECT(salr_adapters_ws_bytes(1, 1, 8, 8, 0, 0, &n) == SALR_OK && n > 0);
  salr_adapters_plan_t plan;
  memset(&plan, 0, sizeof plan);
  EXPECT(salr_adapters_plan(at(0x100000), 100, 4, at(0x200000), 16, &plan, NULL) == SALR_ERR_WORKSPACE);
  EXPECT(salr_adapters_plan(at(0x100000), 100, 4, at(0x100000), 1 << 20, &plan, NULL) == SALR_ERR_INVALID_ARG);
  EXPECT(plan.buffer == NULL);
  plan.buffer = at(0x200000);
  plan.M = INT64_C(1) << 27;
  plan.count = 4096;
  salr_adapters_t a = {4096, 256, 1 << 20, 1 << 20, at(0x10000000000), at(0x20000000000), NULL, NULL};
  /* spans of many terabytes, and at the top of the address space */
  EXPECT(salr_adapters_forward(&a, &plan, at(0x10000000000000), NULL, at(0x30000000000000), at(0x70000000000000), 1,
                               NULL) == SALR_ERR_WORKSPACE);
  EXPECT(salr_adapters_forward(&a, &plan, at(0x10000000000000), NULL, at(0x10000000000010), at(0x70000000000000), 1,
                               NULL) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_adapters_backward(&a, &plan, at(0x10000000000000), at(0x20000000000000), NULL, NULL, at(0x40000000000000),
                                at(0x50000000000000), NULL, 0, NULL) == SALR_ERR_WORKSPACE);
  a.N = 4;
  EXPECT(salr_adapters_backward(&a, &plan, at(16), at(16), NULL, NULL, at(16), at(16), NULL, 0, NULL) ==
         SALR_ERR_UNSUPPORTED);
}

static void muon(void) {
  enum { COUNT = 1000 };
  static int64_t rows[COUNT], cols[COUNT];
  static salr_muon_tensor_t t[COUNT];
  size_t n = 0;
  for (int i = 0; i < COUNT; ++i) {
    rows[i] = i % 257;
    cols[i] = 1 + (i * 37) % 5000;
    if (i % 3 == 0) {
      const int64_t s = rows[i];
      rows[i] = cols[i];
      cols[i] = s;
    }
    const uint64_t base = UINT64_C(0x100000000) * (uint64_t)(i + 1);
    salr_muon_tensor_t q = {at(base), at(base + 0x10000000), at(base + 0x20000000), NULL, rows[i], cols[i], 1.0};
    t[i] = q;
  }
  EXPECT(salr_muon_plan_bytes(rows, cols, COUNT, &n) == SALR_OK && n > COUNT);
  salr_muon_plan_t plan;
  memset(&plan, 0, sizeof plan);
  EXPECT(salr_muon_plan(t, COUNT, SALR_TYPE_F32, SALR_TYPE_BF16, at(0x7000000000000), n - 1, &plan, NULL) ==
         SALR_ERR_WORKSPACE);
  t[500].g = t[499].p;
  EXPECT(salr_muon_plan(t, COUNT, SALR_TYPE_F32, SALR_TYPE_BF16, at(0x7000000000000), n, &plan, NULL) ==
         SALR_ERR_INVALID_ARG);
  t[500].g = at(UINT64_C(0x100000000) * 501 + 0x10000000);
  t[700].m = NULL;
  EXPECT(salr_muon_plan(t, COUNT, SALR_TYPE_F32, SALR_TYPE_BF16, at(0x7000000000000), n, &plan, NULL) ==
         SALR_ERR_INVALID_ARG);
  EXPECT(salr_muon_plan(t, 0, SALR_TYPE_F32, SALR_TYPE_BF16, NULL, 0, &plan, NULL) == SALR_ERR_WORKSPACE);
  rows[3] = INT64_MAX;
  cols[3] = INT64_MAX;
  EXPECT(salr_muon_plan_bytes(rows, cols, COUNT, &n) == SALR_ERR_INVALID_ARG);
  rows[3] = INT64_C(1) << 30;
  cols[3] = 256;
  EXPECT(salr_muon_plan_bytes(rows, cols, COUNT, &n) == SALR_ERR_UNSUPPORTED);
  EXPECT(salr_muon_plan_bytes(rows, cols, INT32_MAX, &n) == SALR_ERR_INVALID_ARG);
  EXPECT(plan.table == NULL);
}

int main(void) {
  adapters();
  muon();
  if (failures) return 1;
  puts("ok");
  return 0;
}

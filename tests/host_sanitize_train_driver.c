/* Host-side driver for tests/test_train_sanitizers.py: walks the argument
 * validation, size arithmetic and plan layout of the routing and AdamW entry
 * points, which run on the host before any device work.  Built with
 * AddressSanitizer and UndefinedBehaviorSanitizer around salr_train_api.cpp;
 * no call here reaches the device.  Prints "ok" and exits 0 when every
 * expectation holds. */
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

static void routing(void) {
  size_t b = 0;
  EXPECT(salr_moe_dispatch_ws_bytes(4096, 6, 64, &b) == SALR_OK && b >= 24 * 64 * 4);
  EXPECT(salr_moe_dispatch_ws_bytes(INT64_MAX, 32, 4096, &b) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_moe_dispatch_ws_bytes((INT64_C(1) << 31) - 65536, 1, 4096, &b) == SALR_OK && b == 64 * 4096 * 4);
  int32_t* ids = at(0x100000);
  float* w = at(0x200000);
  EXPECT(salr_moe_route(at(0x300000), SALR_TYPE_F32, INT64_MAX, 8, 2, 1, ids, w, NULL) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_moe_route(NULL, SALR_TYPE_F32, 4, 8, 2, 1, ids, w, NULL) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_moe_route(ids, SALR_TYPE_BF16, 4, 8, 2, 1, ids, w, NULL) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_moe_dispatch(ids, 1 << 20, 32, 4096, at(0x400000), 1 << 20, at(0x500000), at(0x600000), NULL,
                           at(0x700000), at(0x800000), 1, NULL) == SALR_ERR_INVALID_ARG); /* overlaps */
  EXPECT(salr_moe_dispatch(ids, 4, 2, 8, NULL, 0, at(0x500000), at(0x600000), NULL, NULL, at(0x800000), 1, NULL) ==
         SALR_ERR_WORKSPACE);
  /* spans at the top of the address space */
  EXPECT(salr_moe_combine(at(0x100000), (INT64_C(1) << 31) - 65536, at(0xFFFFFFFFFF000000u), NULL, NULL, 1 << 20, 2,
                          1 << 20, at(0x200000), NULL) == SALR_ERR_INVALID_ARG);
  EXPECT(salr_moe_combine_backward(at(0x100000), NULL, 8, ids, NULL, 4, 2, 64, NULL, w, NULL) == SALR_ERR_INVALID_ARG);
}

static void adamw(void) {
  size_t b = 0;
  int64_t n[3] = {5, 0, 2049};
  EXPECT(salr_adamw_plan_bytes(n, 3, &b) == SALR_OK);
  EXPECT(salr_adamw_plan_bytes(NULL, 0, &b) == SALR_OK);
  n[1] = INT64_MAX;
  EXPECT(salr_adamw_plan_bytes(n, 3, &b) == SALR_ERR_INVALID_ARG);
  /* many tensors: every record and chunk is written before the buffer's size is looked at */
  enum { COUNT = 1000 };
  salr_adamw_tensor_t* t = calloc(COUNT, sizeof *t);
  for (int i = 0; i < COUNT; ++i) {
    const uint64_t base = 0x10000000 + (uint64_t)i * 0x1000000;
    t[i].p = at(base);
    t[i].g = at(base + 0x200000);
    t[i].m = at(base + 0x400000);
    t[i].v = at(base + 0x600000);
    t[i].m_scale = at(base + 0x800000);
    t[i].v_scale = at(base + 0x900000);
    t[i].master = at(base + 0xA00000);
    t[i].n = (i % 3 == 2) ? 0 : 1 + (int64_t)i * 97;
  }
  salr_adamw_plan_t plan;
  memset(&plan, 0x5A, sizeof plan);
  for (int state = 0; state < 2; ++state)
    EXPECT(salr_adamw_plan(t, COUNT, SALR_TYPE_BF16, SALR_TYPE_F32, state, at(0x1000), 64, &plan, NULL) ==
           SALR_ERR_WORKSPACE);
  EXPECT(salr_adamw_plan(t, 0, SALR_TYPE_BF16, SALR_TYPE_F32, 0, NULL, 0, &plan, NULL) == SALR_ERR_WORKSPACE);
  EXPECT(salr_adamw_plan(t, COUNT, SALR_TYPE_F32, SALR_TYPE_F32, 0, at(0x1000), 64, &plan, NULL) ==
         SALR_ERR_INVALID_ARG); /* masters of float parameters */
  t[7].m = t[4].v;
  EXPECT(salr_adamw_plan(t, COUNT, SALR_TYPE_BF16, SALR_TYPE_F32, 0, at(0x1000), 64, &plan, NULL) ==
         SALR_ERR_INVALID_ARG); /* the same state twice */
  free(t);
  salr_adamw_step_args_t a = {1, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0};
  salr_adamw_plan_t empty = {at(0x1000), 0, 0, 0, 0, 0, 0};
  EXPECT(salr_adamw_step(&empty, &a, NULL, NULL) == SALR_OK);
  a.step = INT64_MAX;
  EXPECT(salr_adamw_step(&empty, &a, NULL, NULL) == SALR_OK);
  a.step = -1;
  EXPECT(salr_adamw_step(&empty, &a, NULL, NULL) == SALR_ERR_INVALID_ARG);
}

int main(void) {
  routing();
  adamw();
  if (failures) {
    fprintf(stderr, "%d expectation(s) failed\n", failures);
    return 1;
  }
  printf("ok\n");
  return 0;
}

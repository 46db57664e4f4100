// The router of a mixture-of-experts layer: k experts and their weights from
// each token's logits, and the gradient of the weights (include/salr.h,
// salr_moe_route and salr_moe_route_backward).
//
// Per row of E logits l:  w_j = exp(l_{e_j} - max) / S, where e_0 .. e_{k-1}
// are the k largest (ties to the lower expert) and S is the sum of
// exp(l - max) over all experts, or over the chosen ones (renorm).  Backward,
// with p the same softmax and c = sum_i p_{e_i} dw_i:  dl_e = p_e (dw_e - c).
//
// A group of LANES lanes per row (16 up to 256 experts: four rows a wave),
// PER logits a lane in registers (logit q * LANES + lane), so a row is read
// once.  The k largest are taken one after the other: a maximum over the
// group, then the lowest expert that holds it; within 16 lanes both run on
// DPP row rotations, without the LDS round trips of a shuffle.
//
// Bound by the launch up to a few thousand rows, then by the issue of
// instructions (calls in a graph, over four sets of inputs: 16384 rows of 64
// floats, top 6: 4.4 us, backward 4.3, where reading and writing them takes
// 0.8 and 1.5; 16384 of 256, top 8: 10.4 and 11.2; of 1024, top 8: 28.7 and
// 32.7).  For the first, a wave per row took 18.6 us where 16 lanes took 5.9,
// and float maxima (which quiet NaNs) with the library's exp 4.9 where these
// took 4.2.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "salr.h"
#include "salr_device.hpp"
#include "salr_kernels.hpp"

namespace salr {
namespace {

constexpr int kRouteThreads = 256;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// v combined over the row's lanes, in every one of them.
template <int N>
__device__ __forceinline__ int row_ror(int v) {  // lane i of 16 from lane (i - N) mod 16
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xF, 0xF, true);
}
template <int LANES, class F>
__device__ __forceinline__ int group_all(int v, F f) {
  v = f(v, row_ror<8>(v));
  v = f(v, row_ror<4>(v));
  v = f(v, row_ror<2>(v));
  v = f(v, row_ror<1>(v));
  if constexpr (LANES == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ int group_max(int v) {
  return group_all<LANES>(v, [](int a, int b) { return max(a, b); });
}
template <int LANES>
__device__ __forceinline__ int group_min(int v) {
  return group_all<LANES>(v, [](int a, int b) { return min(a, b); });
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
  return __int_as_float(group_all<LANES>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

template <int LANES>
__device__ __forceinline__ bool group_any(bool v) {
  const uint64_t m = __ballot(v);
  return LANES == 64 ? m != 0 : ((m >> (threadIdx.x & 63 & ~(LANES - 1))) & ((1ull << (LANES & 63)) - 1)) != 0;
}

// Logits as integers in the same order (-0 as 0, NaN as -inf): their maxima
// take one instruction each, where those of floats also quiet NaNs.
constexpr int kLeast = (int)0x807FFFFF;  // order_of(-inf)
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x + 0.f);
  return x == x ? b ^ ((b >> 31) & 0x7FFFFFFF) : kLeast;
}
__device__ __forceinline__ float value_of(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF)); }

// exp(x) for x <= 0 to 2 ulp, 0 below about -87.3, where it is no normal float
// any more (the instruction gives no subnormals; NaN stays): 2^y for y = x
// log2(e), times 1 + ln(2) (x log2(e) - y) for what y's rounding dropped.  x is
// cut at -150, since -inf would leave NaN in the rest.
__device__ __forceinline__ float exp_down(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  x = x < -150.f ? -150.f : x;
  const float y = x * kLog2e;
  const float rest = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(e, rest * kLn2, e);
}

template <class Tl, int LANES, int PER>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const Tl* logits, int64_t T, int32_t E, int32_t k,
                                                                  int32_t renorm, int32_t* ids, float* weights) {
  constexpr int SLOTS = SALR_MOE_MAX_TOPK > LANES ? SALR_MOE_MAX_TOPK / LANES : 1;  // choices kept per lane
  const int lane = threadIdx.x % LANES;
  const int64_t groups = (int64_t)gridDim.x * (kRouteThreads / LANES);
  for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / LANES) + threadIdx.x / LANES; t < T; t += groups) {
    const Tl* row = logits + t * E;
    float l[PER];
    int o[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) l[q] = q * LANES + lane < E ? load_logit(row + q * LANES + lane) : kNegInf;
    int best = kLeast;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      o[q] = order_of(l[q]);
      best = max(best, o[q]);
    }
    best = group_max<LANES>(best);
    const float top = value_of(best);
    float total = 0.f;
    if (!renorm) {
#pragma unroll
      for (int q = 0; q < PER; ++q) total += q * LANES + lane < E ? exp_down(l[q] - top) : 0.f;
      total = group_sum<LANES>(total);
    }
    // lane j % LANES keeps the j-th choice
    int val[SLOTS], id[SLOTS];
#pragma unroll
    for (int c = 0; c < SLOTS; ++c) {
      val[c] = kLeast;
      id[c] = -1;
    }
    for (int j = 0; j < k; ++j) {
      int at = 1 << 30;
#pragma unroll
      for (int q = PER - 1; q >= 0; --q) at = o[q] == best ? q * LANES + lane : at;
      at = group_min<LANES>(at);
      const bool keep = lane == j % LANES && best > kLeast;
#pragma unroll
      for (int c = 0; c < SLOTS; ++c)
        if (keep && j / LANES == c) {
          val[c] = best;
          id[c] = at;
        }
      best = kLeast;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        o[q] = q * LANES + lane == at ? kLeast : o[q];
        best = max(best, o[q]);
      }
      best = group_max<LANES>(best);
    }
    float w[SLOTS], sum = 0.f;
#pragma unroll
    for (int c = 0; c < SLOTS; ++c) {
      w[c] = id[c] >= 0 ? exp_down(value_of(val[c]) - top) : 0.f;
      sum += w[c];
    }
    if (renorm) total = group_sum<LANES>(sum);
#pragma unroll
    for (int c = 0; c < SLOTS; ++c)
      if (c * LANES + lane < k) {
        ids[t * k + c * LANES + lane] = id[c];
        weights[t * k + c * LANES + lane] = id[c] >= 0 ? w[c] / total : 0.f;
      }
  }
}

template <class Tl, int LANES, int PER>
__global__ __launch_bounds__(kRouteThreads) void moe_route_backward_kernel(const Tl* logits, int64_t T, int32_t E,
                                                                           int32_t k, int32_t renorm,
                                                                           const int32_t* ids, const float* dweights,
                                                                           Tl* dlogits) {
  constexpr int SLOTS = SALR_MOE_MAX_TOPK > LANES ? SALR_MOE_MAX_TOPK / LANES : 1;
  constexpr int BATCH = 4;  // choices handed round together
  // From 8 logits a lane on, comparing each with every choice costs more than
  // a row of LDS (rows of 16 lanes 16 banks apart).
  constexpr bool SHARED = PER >= 8;
  constexpr int kStride = LANES * PER + (LANES == 16 ? 16 : 0);
  __shared__ float taken[SHARED ? kRouteThreads / LANES * kStride : 1];
  const int lane = threadIdx.x % LANES;
  const int64_t groups = (int64_t)gridDim.x * (kRouteThreads / LANES);
  for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / LANES) + threadIdx.x / LANES; t < T; t += groups) {
    const Tl* row = logits + t * E;
    int id[SLOTS];
    float dw[SLOTS];
#pragma unroll
    for (int c = 0; c < SLOTS; ++c) {
      const bool in = c * LANES + lane < k;
      id[c] = in ? ids[t * k + c * LANES + lane] : -1;
      dw[c] = in ? dweights[t * k + c * LANES + lane] : 0.f;
    }
    float l[PER], up[PER];  // logit, gradient that reaches its probability
    bool in[PER];           // part of the softmax
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * LANES + lane;
      l[q] = e < E ? load_logit(row + e) : kNegInf;
      up[q] = 0.f;
      in[q] = !renorm && e < E;
    }
    if constexpr (SHARED) {
      // Each choice adds to its expert's place in LDS, one after the other
      // (the same expert twice adds up in order); -0, which no sum of a +0
      // and other values is, marks the places that no choice took.
      volatile float* place = &taken[threadIdx.x / LANES * kStride];
#pragma unroll
      for (int q = 0; q < PER; ++q) place[q * LANES + lane] = -0.f;
      for (int j = 0; j < k; ++j) {
#pragma unroll
        for (int c = 0; c < SLOTS; ++c)
          if (c * LANES + lane == j && (uint32_t)id[c] < (uint32_t)E) {
            const float sum = place[id[c]];
            place[id[c]] = (sum + 0.f) + dw[c];
          }
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const float sum = place[q * LANES + lane];
        in[q] = in[q] || __float_as_int(sum) != __float_as_int(-0.f);
        up[q] = sum;
      }
    } else {
#pragma unroll
      for (int c = 0; c < SLOTS; ++c)
        for (int j0 = c * LANES; j0 < min(k, (c + 1) * LANES); j0 += BATCH) {
          int ej[BATCH];
          float dj[BATCH];
#pragma unroll
          for (int b = 0; b < BATCH; ++b) {  // (past k: id -1, which no lane has)
            ej[b] = __shfl(id[c], (j0 + b) % LANES, LANES);
            dj[b] = __shfl(dw[c], (j0 + b) % LANES, LANES);
          }
#pragma unroll
          for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int q = 0; q < PER; ++q) {
              const bool hit = ej[b] == q * LANES + lane && ej[b] < E;
              up[q] += hit ? dj[b] : 0.f;
              in[q] = in[q] || hit;
            }
        }
    }
    int best = kLeast;
#pragma unroll
    for (int q = 0; q < PER; ++q) best = max(best, in[q] ? order_of(l[q]) : kLeast);
    best = group_max<LANES>(best);
    const float top = value_of(best);
    // (a row without any choice gets zeros whatever its logits are, NaN too)
    bool any = false;
#pragma unroll
    for (int c = 0; c < SLOTS; ++c) any = any || (uint32_t)id[c] < (uint32_t)E;
    const bool live = group_any<LANES>(any) && best > kLeast;
    float total = 0.f, c = 0.f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      l[q] = in[q] && live ? exp_down(l[q] - top) : 0.f;
      total += l[q];
      c += l[q] * up[q];
    }
    total = group_sum<LANES>(total);
    c = group_sum<LANES>(c);
    const float inv = total != 0.f ? 1.f / total : 0.f;
    c *= inv;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * LANES + lane;
      if (e < E) store_logit(dlogits + t * E + e, l[q] * inv * (up[q] - c));
    }
  }
}

// f(lanes, per) for the first form that holds E logits.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <class F>
void with_form(int32_t E, F f) {
  if (E <= 16) f(Int<16>{}, Int<1>{});
  else if (E <= 32) f(Int<16>{}, Int<2>{});
  else if (E <= 64) f(Int<16>{}, Int<4>{});
  else if (E <= 128) f(Int<16>{}, Int<8>{});
  else if (E <= 256) f(Int<16>{}, Int<16>{});
  else if (E <= 512) f(Int<64>{}, Int<8>{});
  else if (E <= 1024) f(Int<64>{}, Int<16>{});
  else if (E <= 2048) f(Int<64>{}, Int<32>{});
  else f(Int<64>{}, Int<64>{});
}

// Workgroups for T rows (more than kMaxBlocks: they loop).
constexpr int64_t kMaxBlocks = int64_t(1) << 22;
dim3 route_grid(int64_t T, int lanes) {
  const int64_t rows = kRouteThreads / lanes;
  return dim3((unsigned)std::min(kMaxBlocks, (T + rows - 1) / rows));
}

}  // namespace

hipError_t launch_moe_route(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renorm, int32_t* ids,
                            float* weights, hipStream_t s) {
  if (T == 0) return hipSuccess;
  with_form(E, [&](auto lanes, auto per) {
    constexpr int LANES = decltype(lanes)::value, PER = decltype(per)::value;
    const dim3 grid = route_grid(T, LANES);
    if (f32)
      hipLaunchKernelGGL((moe_route_kernel<float, LANES, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const float*>(logits), T, E, k, (int32_t)renorm, ids, weights);
    else
      hipLaunchKernelGGL((moe_route_kernel<uint16_t, LANES, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const uint16_t*>(logits), T, E, k, (int32_t)renorm, ids, weights);
  });
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renorm,
                                     const int32_t* ids, const float* dweights, void* dlogits, hipStream_t s) {
  if (T == 0) return hipSuccess;
  with_form(E, [&](auto lanes, auto per) {
    constexpr int LANES = decltype(lanes)::value, PER = decltype(per)::value;
    const dim3 grid = route_grid(T, LANES);
    if (f32)
      hipLaunchKernelGGL((moe_route_backward_kernel<float, LANES, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const float*>(logits), T, E, k, (int32_t)renorm, ids, dweights,
                         static_cast<float*>(dlogits));
    else
      hipLaunchKernelGGL((moe_route_backward_kernel<uint16_t, LANES, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const uint16_t*>(logits), T, E, k, (int32_t)renorm, ids, dweights,
                         static_cast<uint16_t*>(dlogits));
  });
  return hipGetLastError();
}

}  // namespace salr

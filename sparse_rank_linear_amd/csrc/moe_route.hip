// The router of a mixture-of-experts layer: k experts and their weights from
// each token's logits, and the gradient of the weights (include/salr.h,
// salr_moe_route and salr_moe_route_backward).
//
// Per row of E logits l:  w_j = exp(l_{e_j} - max) / S, where e_0 .. e_{k-1}
// are the k largest (ties to the lower expert) and S is the sum of
// exp(l - max) over all experts, or over the chosen ones (renorm).  Backward,
// with p the same softmax and c = sum_i p_{e_i} dw_i:  dl_e = p_e (dw_e - c).
//
// One wave per row, PER logits a lane in registers (logit q * 64 + lane), so
// a row is read once.  The k largest are taken one after the other: a
// wave-wide maximum, then the lowest expert that holds it.
#include <hip/hip_runtime.h>

#include <algorithm>

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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = min(v, __shfl_xor(v, d, 64));
  return v;
}

template <class Tl, int PER>
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(const Tl* logits, int64_t T, int32_t E, int32_t k,
                                                                  int32_t renorm, int32_t* ids, float* weights) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * (kRouteThreads / 64);
  for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 64) + (threadIdx.x >> 6); t < T; t += waves) {
    float l[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * 64 + lane;
      l[q] = e < E ? load_logit(logits + t * E + e) : kNegInf;
    }
    float top = kNegInf;  // (fmaxf leaves NaN aside)
#pragma unroll
    for (int q = 0; q < PER; ++q) top = fmaxf(top, l[q]);
    top = wave_max(top);
    float total = 0.f;
    if (!renorm) {
#pragma unroll
      for (int q = 0; q < PER; ++q) total += q * 64 + lane < E ? expf(l[q] - top) : 0.f;
      total = wave_sum(total);
    }
    // lane j keeps the j-th choice
    float mine = 0.f;
    int my_id = -1;
    float best = top;
    for (int j = 0; j < k; ++j) {
      if (!(best > kNegInf)) break;
      int at = 1 << 30;
#pragma unroll
      for (int q = PER - 1; q >= 0; --q) at = l[q] == best ? q * 64 + lane : at;
      at = wave_min(at);
      const float w = expf(best - top);
      if (renorm) total += w;
      if (lane == j) {
        mine = w;
        my_id = at;
      }
      float next = kNegInf;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (q * 64 + lane == at) l[q] = kNegInf;
        next = fmaxf(next, l[q]);
      }
      best = wave_max(next);
    }
    if (lane < k) {
      ids[t * k + lane] = my_id;
      weights[t * k + lane] = my_id >= 0 ? mine / total : 0.f;
    }
  }
}

template <class Tl, int PER>
__global__ __launch_bounds__(kRouteThreads) void moe_route_backward_kernel(const Tl* logits, int64_t T, int32_t E,
                                                                           int32_t k, int32_t renorm,
                                                                           const int32_t* ids, const float* dweights,
                                                                           Tl* dlogits) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * (kRouteThreads / 64);
  for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 64) + (threadIdx.x >> 6); t < T; t += waves) {
    float l[PER], up[PER];  // logit, gradient that reaches its probability
    bool chosen[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * 64 + lane;
      l[q] = e < E ? load_logit(logits + t * E + e) : kNegInf;
      up[q] = 0.f;
      chosen[q] = false;
    }
    int id = -1;
    float dw = 0.f;
    if (lane < k) {
      id = ids[t * k + lane];
      dw = dweights[t * k + lane];
    }
    for (int j = 0; j < k; ++j) {
      const int e = __shfl(id, j, 64);
      const float d = __shfl(dw, j, 64);
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (e == q * 64 + lane && e < E) {
          up[q] += d;
          chosen[q] = true;
        }
    }
    float top = kNegInf;
#pragma unroll
    for (int q = 0; q < PER; ++q) top = fmaxf(top, !renorm || chosen[q] ? l[q] : kNegInf);
    top = wave_max(top);
    float total = 0.f, c = 0.f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const bool in = q * 64 + lane < E && (!renorm || chosen[q]);
      l[q] = in && top > kNegInf ? expf(l[q] - top) : 0.f;
      total += l[q];
      c += l[q] * up[q];
    }
    total = wave_sum(total);
    c = wave_sum(c);
    const float inv = total != 0.f ? 1.f / total : 0.f;
    c *= inv;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = q * 64 + lane;
      if (e < E) store_logit(dlogits + t * E + e, l[q] * inv * (up[q] - c));
    }
  }
}

// f(std::integral_constant<int, PER>) for the least PER with 64 PER >= E.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <class F>
void with_per(int32_t E, F f) {
  if (E <= 64) f(Int<1>{});
  else if (E <= 128) f(Int<2>{});
  else if (E <= 256) f(Int<4>{});
  else if (E <= 512) f(Int<8>{});
  else if (E <= 1024) f(Int<16>{});
  else if (E <= 2048) f(Int<32>{});
  else f(Int<64>{});
}

// Workgroups for T rows, a wave a row (more than kMaxBlocks: they loop).
constexpr int64_t kMaxBlocks = int64_t(1) << 22;
unsigned route_blocks(int64_t T) {
  return (unsigned)std::min(kMaxBlocks, (T + kRouteThreads / 64 - 1) / (kRouteThreads / 64));
}

}  // namespace

hipError_t launch_moe_route(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renorm, int32_t* ids,
                            float* weights, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const dim3 grid(route_blocks(T));
  with_per(E, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    if (f32)
      hipLaunchKernelGGL((moe_route_kernel<float, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const float*>(logits), T, E, k, (int32_t)renorm, ids, weights);
    else
      hipLaunchKernelGGL((moe_route_kernel<uint16_t, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const uint16_t*>(logits), T, E, k, (int32_t)renorm, ids, weights);
  });
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renorm,
                                     const int32_t* ids, const float* dweights, void* dlogits, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const dim3 grid(route_blocks(T));
  with_per(E, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    if (f32)
      hipLaunchKernelGGL((moe_route_backward_kernel<float, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const float*>(logits), T, E, k, (int32_t)renorm, ids, dweights,
                         static_cast<float*>(dlogits));
    else
      hipLaunchKernelGGL((moe_route_backward_kernel<uint16_t, PER>), grid, dim3(kRouteThreads), 0, s,
                         static_cast<const uint16_t*>(logits), T, E, k, (int32_t)renorm, ids, dweights,
                         static_cast<uint16_t*>(dlogits));
  });
  return hipGetLastError();
}

}  // namespace salr

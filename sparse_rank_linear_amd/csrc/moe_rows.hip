// The way of the tokens to their experts' rows and back (include/salr.h,
// salr_moe_dispatch, salr_moe_combine and its gradient).
//
// Slot s = t * k + j is token t's j-th choice.  The sort is a stable counting
// sort:  rows[s] = #{s' : id_s' < id_s} + #{s' < s : id_s' = id_s},  counted
// per chunk of slots (moe_count_kernel), then placed (moe_place_kernel: each
// workgroup adds up the chunks before its own, so no scan launch sits
// between).  The copies run token-major: a token's row is read once and
// written to its k rows (or its k rows are read and one written), 16 bytes a
// thread; they are bound by HBM.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "salr_device.hpp"
#include "salr_kernels.hpp"

namespace salr {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kCopyThreads = 256;

// ---- sort ----

// hist[chunk][e] = slots of the chunk with id e.
__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(MoeDispatchArgs a) {
  extern __shared__ uint32_t sm[];
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) sm[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * a.chunk, s1 = min(s0 + a.chunk, (int64_t)a.n);
  for (int64_t s = s0 + threadIdx.x; s < s1; s += kSortThreads) {
    const uint32_t id = (uint32_t)a.ids[s];
    if (id < (uint32_t)a.E) atomicAdd(&sm[id], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.hist[(size_t)blockIdx.x * a.E + e] = sm[e];
}

// Exclusive prefix sum of v over the workgroup's kSortThreads threads.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* part, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortThreads / 64; ++w) {
    if (w < wave) before += part[w];
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

// Lanes of the wave that hold the same id (bits: the id's bits in use).
__device__ __forceinline__ uint64_t same_id(uint32_t id, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool set = (id >> b) & 1u;
    const uint64_t v = __ballot(set);
    m &= set ? v : ~v;
  }
  return m;
}

// rows and slots of one chunk of slots; workgroup 0 writes the offsets.
// LDS: first[E] (the row where the chunk's slots of e begin), then
// next[waves][E]: each wave's running row of e.
__global__ __launch_bounds__(kSortThreads) void moe_place_kernel(MoeDispatchArgs a, int waves, int bits) {
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t part[kSortThreads / 64];
  uint32_t* first = sm;
  uint32_t* next = sm + a.E;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < a.E * (waves + 1); e += kSortThreads) sm[e] = 0;
  __syncthreads();
  // next[0][e]: all slots of e; first[e]: those of the chunks before
  for (int c = tid; c < a.E * a.chunks; c += kSortThreads) {
    const uint32_t h = a.hist[c];
    const int e = c % a.E;
    if (h) {
      atomicAdd(&next[e], h);
      if (c / a.E < (int)blockIdx.x) atomicAdd(&first[e], h);
    }
  }
  __syncthreads();
  uint32_t run = 0;
  for (int e0 = 0; e0 < a.E; e0 += kSortThreads) {
    const int e = e0 + tid;
    uint32_t total;
    const uint32_t off = run + block_prefix(e < a.E ? next[e] : 0u, part, &total);
    if (e < a.E) {
      first[e] += off;
      next[e] = 0;
      if (blockIdx.x == 0) a.off[e] = (int32_t)off;
    }
    run += total;
  }
  if (blockIdx.x == 0 && tid == 0) a.off[a.E] = (int32_t)run;
  __syncthreads();
  // each wave counts its run of the chunk's slots, the counts become rows
  const int per = (a.chunk / waves + 63) / 64 * 64;
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk, c1 = min(c0 + a.chunk, (int64_t)a.n);
  const int64_t w0 = c0 + (int64_t)wave * per, w1 = wave < waves ? min(w0 + per, c1) : w0;
  for (int64_t s = w0 + lane; s < w1; s += 64) {
    const uint32_t id = (uint32_t)a.ids[s];
    if (id < (uint32_t)a.E) atomicAdd(&next[wave * a.E + id], 1u);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kSortThreads) {
    uint32_t r = first[e];
    for (int w = 0; w < waves; ++w) {
      const uint32_t c = next[w * a.E + e];
      next[w * a.E + e] = r;
      r += c;
    }
  }
  __syncthreads();
  // (a wave's LDS accesses stay in order, so a counter that its last lane
  // advances is read advanced in the next 64 slots)
  for (int64_t base = w0; base < w1; base += 64) {
    const int64_t s = base + lane;
    const uint32_t id = s < w1 ? (uint32_t)a.ids[s] : 0xFFFFFFFFu;
    const bool ok = id < (uint32_t)a.E;
    const uint64_t m = same_id(ok ? id : 0u, bits) & __ballot(ok);
    volatile uint32_t* cell = &next[wave * a.E + (ok ? id : 0u)];
    const uint32_t r = *cell;
    const uint32_t rank = (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
    __builtin_amdgcn_wave_barrier();
    if (ok && (m >> lane) == 1ull) *cell = r + rank + 1;
    __builtin_amdgcn_wave_barrier();
    if (s < w1) a.rows[s] = ok ? (int32_t)(r + rank) : -1;
    if (ok && a.slots) a.slots[r + rank] = (int32_t)s;
  }
}

// ---- rows ----

template <int VEC>
struct Piece;  // VEC bf16 values
template <>
struct Piece<8> {
  u32x4_t w;
};
template <>
struct Piece<1> {
  uint16_t w;
};
template <int VEC>
__device__ __forceinline__ Piece<VEC> load_piece(const uint16_t* p) {
  return *reinterpret_cast<const Piece<VEC>*>(p);
}
template <int VEC>
__device__ __forceinline__ void store_piece(uint16_t* p, Piece<VEC> v) {
  *reinterpret_cast<Piece<VEC>*>(p) = v;
}
__device__ __forceinline__ void add_piece(float* acc, Piece<8> v, float w) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    acc[2 * c] += w * bf16_to_f32((uint16_t)v.w[c]);
    acc[2 * c + 1] += w * bf16_to_f32((uint16_t)(v.w[c] >> 16));
  }
}
__device__ __forceinline__ void add_piece(float* acc, Piece<1> v, float w) { acc[0] += w * bf16_to_f32(v.w); }
__device__ __forceinline__ Piece<8> round_piece8(const float* f) {
  Piece<8> v;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    v.w[c] = (uint32_t)f32_to_bf16(f[2 * c]) | ((uint32_t)f32_to_bf16(f[2 * c + 1]) << 16);
  return v;
}
template <int VEC>
__device__ __forceinline__ Piece<VEC> round_piece(const float* f) {
  if constexpr (VEC == 8) return round_piece8(f);
  else return Piece<1>{f32_to_bf16(f[0])};
}

// Xs[rows[t][j]] = X[t]: one thread per (token, piece).
template <int VEC>
__global__ __launch_bounds__(kCopyThreads) void moe_gather_kernel(MoeDispatchArgs a, int64_t pieces, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kCopyThreads) {
    const int64_t t = i / pieces, d = (i - t * pieces) * VEC;
    const Piece<VEC> v = load_piece<VEC>(a.X + t * a.D + d);
    for (int j = 0; j < a.k; ++j) {
      const int32_t r = a.rows[t * a.k + j];
      if (r >= 0) store_piece<VEC>(a.Xs + (int64_t)r * a.D + d, v);
    }
  }
}

// Y[t] = base[t] + sum_j w[t][j] Ys[rows[t][j]]: one thread per (token, piece).
template <int VEC>
__global__ __launch_bounds__(kCopyThreads) void moe_combine_kernel(MoeCombineArgs a, int64_t pieces, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kCopyThreads) {
    const int64_t t = i / pieces, d = (i - t * pieces) * VEC;
    float acc[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] = 0.f;
    if (a.base) add_piece(acc, load_piece<VEC>(a.base + t * a.D + d), 1.f);
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = a.rows[t * a.k + j];
      if (r < 0 || r >= a.R) continue;
      const float w = a.weights ? a.weights[t * a.k + j] : 1.f;
      add_piece(acc, load_piece<VEC>(a.Ys + r * a.D + d), w);
    }
    store_piece<VEC>(a.out + t * a.D + d, round_piece<VEC>(acc));
  }
}

// A workgroup per token: each slot's row is read for its dot product and
// written (dYs) in turn.
template <int VEC>
__global__ __launch_bounds__(kCopyThreads) void moe_combine_backward_kernel(MoeCombineArgs a, int64_t pieces) {
  __shared__ float part[kCopyThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = a.rows[t * a.k + j];
      const bool ok = r >= 0 && r < a.R;
      const float w = a.weights ? a.weights[t * a.k + j] : 1.f;
      float dot = 0.f;
      if (ok) {
        for (int64_t p = threadIdx.x; p < pieces; p += kCopyThreads) {
          float g[VEC], o[VEC];
#pragma unroll
          for (int c = 0; c < VEC; ++c) g[c] = o[c] = 0.f;
          add_piece(g, load_piece<VEC>(a.dY + t * a.D + p * VEC), 1.f);
          if (a.dweights) {
            float y[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) y[c] = 0.f;
            add_piece(y, load_piece<VEC>(a.Ys + r * a.D + p * VEC), 1.f);
#pragma unroll
            for (int c = 0; c < VEC; ++c) dot += g[c] * y[c];
          }
          if (a.out) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) o[c] = w * g[c];
            store_piece<VEC>(a.out + r * a.D + p * VEC, round_piece<VEC>(o));
          }
        }
      }
      if (a.dweights) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
        if (lane == 0) part[wave] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
          float sum = 0.f;
          for (int q = 0; q < kCopyThreads / 64; ++q) sum += part[q];
          a.dweights[t * a.k + j] = ok ? sum : 0.f;
        }
        __syncthreads();
      }
    }
  }
}

// Workgroups for n items, `per` each (more than kMaxBlocks: they loop).
constexpr int64_t kMaxBlocks = int64_t(1) << 22;
inline unsigned blocks_for(int64_t n, int64_t per) { return (unsigned)std::min(kMaxBlocks, (n + per - 1) / per); }

}  // namespace

int32_t moe_sort_chunk(int64_t n) {
  const int64_t c = (n + kMoeSortChunks - 1) / kMoeSortChunks;
  return (int32_t)std::max<int64_t>(1024, (c + 1023) / 1024 * 1024);
}

hipError_t launch_moe_dispatch(const MoeDispatchArgs& a, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
  // (each wave's counters: 4 waves keep E = 4096 within 80 KB of LDS)
  const int waves = a.E <= 1024 ? 16 : 4;
  const int chunks = std::max(a.chunks, 1);  // (no slots: workgroup 0 still writes the offsets)
  hipLaunchKernelGGL(moe_count_kernel, dim3((unsigned)chunks), dim3(kSortThreads), (size_t)a.E * 4, s, a);
  hipLaunchKernelGGL(moe_place_kernel, dim3((unsigned)chunks), dim3(kSortThreads), (size_t)a.E * (waves + 1) * 4, s,
                     a, waves, bits);
  if (a.X && a.n > 0) {
    const int64_t T = a.n / a.k;
    if (a.D % 8 == 0) {
      const int64_t p = a.D / 8;
      hipLaunchKernelGGL(moe_gather_kernel<8>, dim3(blocks_for(T * p, kCopyThreads)), dim3(kCopyThreads), 0, s, a, p,
                         T * p);
    } else {
      hipLaunchKernelGGL(moe_gather_kernel<1>, dim3(blocks_for(T * a.D, kCopyThreads)), dim3(kCopyThreads), 0, s, a,
                         a.D, T * a.D);
    }
  }
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.D % 8 == 0) {
    const int64_t p = a.D / 8;
    hipLaunchKernelGGL(moe_combine_kernel<8>, dim3(blocks_for(a.T * p, kCopyThreads)), dim3(kCopyThreads), 0, s, a, p,
                       a.T * p);
  } else {
    hipLaunchKernelGGL(moe_combine_kernel<1>, dim3(blocks_for(a.T * a.D, kCopyThreads)), dim3(kCopyThreads), 0, s, a,
                       a.D, a.T * a.D);
  }
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const MoeCombineArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.D % 8 == 0)
    hipLaunchKernelGGL(moe_combine_backward_kernel<8>, dim3(blocks_for(a.T, 1)), dim3(kCopyThreads), 0, s, a, a.D / 8);
  else
    hipLaunchKernelGGL(moe_combine_backward_kernel<1>, dim3(blocks_for(a.T, 1)), dim3(kCopyThreads), 0, s, a, a.D);
  return hipGetLastError();
}

}  // namespace salr

// The way of the tokens to their experts' rows and back (include/salr.h,
// salr_moe_dispatch, salr_moe_combine and its gradient).
//
// Slot s = t * k + j is token t's j-th choice.  The sort is a stable counting
// sort:  rows[s] = #{s' : id_s' < id_s} + #{s' < s : id_s' = id_s}.
//
// moe_dispatch_kernel sorts and copies in one launch: every workgroup counts
// the ids for itself (all of them, and those before its own few tokens),
// places its slots and copies its tokens' rows.  Each workgroup reads all n
// ids, so from a few thousand slots on moe_count_kernel counts them in chunks
// first and the workgroups add up the chunks' counts; with many chunks of
// many experts moe_place_kernel does that once per chunk and
// moe_gather_kernel copies.  The copies run token-major: a token's row is read
// once and written to its k rows (or its k rows are read and one written), 16
// bytes a thread; they are bound by HBM.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "salr_device.hpp"
#include "salr_kernels.hpp"

namespace salr {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kDispatchThreads = 512;

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

// Exclusive prefix sum of v over the workgroup's THREADS threads.
template <int THREADS>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* part, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) part[wave] = incl;
  lds_barrier();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += part[w];
    all += part[w];
  }
  lds_barrier();
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

// Adds the chunks' counts: all[e] over every chunk, first[e] over those
// before `chunk` (both at e << shift).  Threads share an expert's chunks as far
// as they go round.
template <int THREADS>
__device__ __forceinline__ void add_chunks(const MoeDispatchArgs& a, int chunk, int shift, uint32_t* all,
                                           uint32_t* first) {
  const int groups = max(1, THREADS / a.E), g = (int)threadIdx.x / a.E;
  for (int e = (int)threadIdx.x - g * a.E; e < a.E && g < groups; e += THREADS) {
    uint32_t sum = 0, before = 0;
#pragma unroll 4
    for (int c = g; c < a.chunks; c += groups) {
      const uint32_t h = a.hist[(size_t)c * a.E + e];
      sum += h;
      before += c < chunk ? h : 0u;
    }
    if (sum) atomicAdd(&all[e << shift], sum);
    if (before) atomicAdd(&first[e << shift], before);
  }
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
  add_chunks<kSortThreads>(a, blockIdx.x, 0, next, first);
  __syncthreads();
  uint32_t run = 0;
  for (int e0 = 0; e0 < a.E; e0 += kSortThreads) {
    const int e = e0 + tid;
    uint32_t total;
    const uint32_t off = run + block_prefix<kSortThreads>(e < a.E ? next[e] : 0u, part, &total);
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

// VEC bf16 values of a row, as wide as the row's length allows.
template <int VEC>
struct Piece;
template <>
struct Piece<8> {
  u32x4_t w;
};
template <>
struct Piece<4> {
  u32x2_t w;
};
template <>
struct Piece<2> {
  uint32_t w;
};
template <>
struct Piece<1> {
  uint16_t w;
};
// NT: data that is not read again soon, past the caches.
template <int VEC, bool NT = false>
__device__ __forceinline__ Piece<VEC> load_piece(const uint16_t* p) {
  Piece<VEC> v;
  const auto* q = reinterpret_cast<const decltype(v.w)*>(p);
  if constexpr (NT) v.w = __builtin_nontemporal_load(q);
  else v.w = *q;
  return v;
}
template <int VEC, bool NT = false>
__device__ __forceinline__ void store_piece(uint16_t* p, Piece<VEC> v) {
  auto* q = reinterpret_cast<decltype(v.w)*>(p);
  if constexpr (NT) __builtin_nontemporal_store(v.w, q);
  else *q = v.w;
}
template <int VEC>
__device__ __forceinline__ void expand_piece(float* x, Piece<VEC> v) {
  if constexpr (VEC == 1) {
    x[0] = bf16_to_f32(v.w);
  } else {
    uint32_t w[VEC / 2];
    __builtin_memcpy(w, &v, sizeof(v));
#pragma unroll
    for (int c = 0; c < VEC / 2; ++c) {
      x[2 * c] = bf16_to_f32((uint16_t)w[c]);
      x[2 * c + 1] = bf16_to_f32((uint16_t)(w[c] >> 16));
    }
  }
}
template <int VEC>
__device__ __forceinline__ Piece<VEC> round_piece(const float* f) {
  Piece<VEC> v;
  if constexpr (VEC == 1) {
    v.w = f32_to_bf16(f[0]);
  } else {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int c = 0; c < VEC / 2; ++c)
      w[c] = (uint32_t)f32_to_bf16(f[2 * c]) | ((uint32_t)f32_to_bf16(f[2 * c + 1]) << 16);
    __builtin_memcpy(&v, w, sizeof(v));
  }
  return v;
}

// Sort and copy in one launch, after moe_count_kernel where there are more
// chunks than one: the workgroup's tokens are [G * blockIdx.x, + G), G * k <=
// 64.  LDS: all (slots of each expert), then first (in the end the row where the
// workgroup's slots of e begin), 1 << shift counters an expert each, which a
// wave's lanes share out: few experts would make them queue at one.
template <int VEC>
__global__ __launch_bounds__(kDispatchThreads) void moe_dispatch_kernel(MoeDispatchArgs a, int64_t T, int G, int bits,
                                                                        int shift, int pieces) {
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t part[kDispatchThreads / 64];
  __shared__ int32_t row[64];
  uint32_t* all = sm;
  uint32_t* first = sm + (a.E << shift);
  const int tid = threadIdx.x, mine_of = tid & ((1 << shift) - 1);
  const int64_t t0 = (int64_t)blockIdx.x * G, t1 = min(t0 + G, T);
  const int s0 = (int)(t0 * a.k), s1 = (int)(t1 * a.k);
  // (what does not wait for the sort is requested before it, and the barriers
  // wait for LDS alone: 16 tokens, 6 of 64, 2048 columns 3.8 us, without 4.0)
  const uint32_t mine = tid < 64 && s0 + tid < s1 ? (uint32_t)a.ids[s0 + tid] : 0xFFFFFFFFu;
  const int total = a.X ? (int)(t1 - t0) * pieces : 0;
  Piece<VEC> ahead;
  if (tid < total) ahead = load_piece<VEC>(a.X + t0 * a.D + (int64_t)tid * VEC);
  for (int e = tid; e < 2 * (a.E << shift); e += kDispatchThreads) sm[e] = 0;
  lds_barrier();
  if (a.chunks == 1) {
    // (four ids requested at a time; one atomic each: those from the
    // workgroup's slots on go to `all`, which takes the others after)
    for (int base = tid; base < a.n; base += 4 * kDispatchThreads) {
      uint32_t id[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int s = base + q * kDispatchThreads;
        id[q] = s < a.n ? (uint32_t)a.ids[s] : 0xFFFFFFFFu;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (id[q] < (uint32_t)a.E)
          atomicAdd(&(base + q * kDispatchThreads < s0 ? first : all)[(id[q] << shift) + mine_of], 1u);
    }
  } else {
    const int chunk = s0 / a.chunk;
    add_chunks<kDispatchThreads>(a, chunk, shift, all, first);
    for (int s = chunk * a.chunk + tid; s < s0; s += kDispatchThreads) {
      const uint32_t id = (uint32_t)a.ids[s];
      if (id < (uint32_t)a.E) atomicAdd(&first[(id << shift) + mine_of], 1u);
    }
  }
  lds_barrier();
  uint32_t run = 0;
  for (int e0 = 0; e0 < a.E; e0 += kDispatchThreads) {
    const int e = e0 + tid;
    uint32_t total;
    uint32_t before = 0, rest = 0;
    for (int c = e << shift; e < a.E && c < (e + 1) << shift; ++c) {
      before += first[c];
      rest += all[c];
    }
    const uint32_t off = run + block_prefix<kDispatchThreads>(a.chunks == 1 ? before + rest : rest, part, &total);
    if (e < a.E) {
      first[e << shift] = before + off;
      if (blockIdx.x == 0) a.off[e] = (int32_t)off;
    }
    run += total;
  }
  if (blockIdx.x == 0 && tid == 0) a.off[a.E] = (int32_t)run;
  lds_barrier();
  if (tid < 64) {
    const int s = s0 + tid;
    const bool ok = mine < (uint32_t)a.E;
    const uint64_t m = same_id(ok ? mine : 0u, bits) & __ballot(ok);
    const int32_t r = ok ? (int32_t)(first[mine << shift] + (uint32_t)__popcll(m & ((1ull << tid) - 1ull))) : -1;
    row[tid] = r;
    if (s < s1) a.rows[s] = r;
    if (ok && a.slots) a.slots[r] = s;
  }
  lds_barrier();
  for (int i = tid; i < total; i += kDispatchThreads) {
    const int g = i / pieces;
    const int64_t d = (int64_t)(i - g * pieces) * VEC;
    const Piece<VEC> v = i == tid ? ahead : load_piece<VEC>(a.X + (t0 + g) * a.D + d);
    for (int j = 0; j < a.k; ++j) {
      const int32_t r = row[g * a.k + j];
      if (r >= 0) store_piece<VEC, true>(a.Xs + (int64_t)r * a.D + d, v);
    }
  }
}

// i / n for n < 2^32 (in 32 bits wherever i allows it).
__device__ __forceinline__ int64_t divide(int64_t i, int64_t n) {
  return (uint64_t)i >> 32 ? i / n : (int64_t)((uint32_t)i / (uint32_t)n);
}

// Xs[rows[t][j]] = X[t]: one thread per (token, piece).
template <int VEC>
__global__ __launch_bounds__(kCopyThreads) void moe_gather_kernel(MoeDispatchArgs a, int64_t pieces, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kCopyThreads) {
    const int64_t t = divide(i, pieces), d = (i - t * pieces) * VEC;
    const Piece<VEC> v = load_piece<VEC>(a.X + t * a.D + d);
    for (int j = 0; j < a.k; ++j) {
      const int32_t r = a.rows[t * a.k + j];
      if (r >= 0) store_piece<VEC, true>(a.Xs + (int64_t)r * a.D + d, v);
    }
  }
}

// Y[t] = base[t] + sum_j w[t][j] Ys[rows[t][j]], a piece a thread; KB rows are
// requested before the first is used.  WAVE: a wave has `width` = 64
// consecutive pieces of one token (row starts and weights become scalar
// loads), the last of a token's `parts` waves maybe fewer; else thread i has
// piece i of all (parts = 1, width = pieces).
template <int VEC, int KB, bool NT, bool WAVE>
__global__ __launch_bounds__(kCopyThreads) void moe_combine_kernel(MoeCombineArgs a, int parts, int width,
                                                                   int64_t total) {
  const int lane = threadIdx.x & 63;
  const int per = WAVE ? kCopyThreads / 64 : kCopyThreads;  // items a workgroup: waves' shares, or pieces
  const int mine = WAVE ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : (int)threadIdx.x;
  for (int64_t i = (int64_t)blockIdx.x * per + mine; i < total; i += (int64_t)gridDim.x * per) {
    const int64_t t = divide(i, WAVE ? parts : width);
    const int64_t d = (WAVE ? (i - t * parts) * 64 + lane : i - t * width) * VEC;
    if (WAVE && d >= a.D) continue;
    float acc[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc[c] = 0.f;
    Piece<VEC> b;
    if (a.base) b = load_piece<VEC, NT>(a.base + t * a.D + d);
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      Piece<VEC> v[KB];
      float w[KB];
      bool ok[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t r = j0 + j < a.k ? a.rows[t * a.k + j0 + j] : -1;
        ok[j] = r >= 0 && r < a.R;
        w[j] = ok[j] && a.weights ? a.weights[t * a.k + j0 + j] : 1.f;
        if (ok[j]) v[j] = load_piece<VEC, NT>(a.Ys + r * a.D + d);
      }
      if (j0 == 0 && a.base) expand_piece(acc, b);
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (ok[j]) {
          float x[VEC];
          expand_piece(x, v[j]);
#pragma unroll
          for (int c = 0; c < VEC; ++c) acc[c] += w[j] * x[c];
        }
    }
    store_piece<VEC, true>(a.out + t * a.D + d, round_piece<VEC>(acc));
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// dYs and dweights of one token by THREADS threads (a wave, or the workgroup
// for long rows): a piece of dY is loaded once for KB slots, whose
// rows' pieces are requested together.
template <int VEC, int THREADS, int KB, bool NT>
__global__ __launch_bounds__(kCopyThreads) void moe_combine_backward_kernel(MoeCombineArgs a, int pieces) {
  constexpr int kTokens = kCopyThreads / THREADS;
  __shared__ float part[kCopyThreads / 64][KB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = threadIdx.x % THREADS;
  for (int64_t t = (int64_t)blockIdx.x * kTokens + (kTokens > 1 ? wave : 0); t < a.T; t += (int64_t)gridDim.x * kTokens) {
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      int64_t r[KB];
      float w[KB], dot[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        r[j] = j0 + j < a.k ? a.rows[t * a.k + j0 + j] : -1;
        if (r[j] >= a.R) r[j] = -1;
        w[j] = r[j] >= 0 && a.weights ? a.weights[t * a.k + j0 + j] : 1.f;
        dot[j] = 0.f;
      }
      for (int p = tid; p < pieces; p += THREADS) {
        float g[VEC];
        const Piece<VEC> gp = load_piece<VEC>(a.dY + t * a.D + (int64_t)p * VEC);
        Piece<VEC> y[KB];
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (r[j] >= 0) y[j] = load_piece<VEC, NT>(a.Ys + r[j] * a.D + (int64_t)p * VEC);
        }
        expand_piece(g, gp);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (r[j] < 0) continue;
          if (a.dweights) {
            float f[VEC];
            expand_piece(f, y[j]);
#pragma unroll
            for (int c = 0; c < VEC; ++c) dot[j] += g[c] * f[c];
          }
          if (a.out) {
            float o[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) o[c] = w[j] * g[c];
            store_piece<VEC, true>(a.out + r[j] * a.D + (int64_t)p * VEC, round_piece<VEC>(o));
          }
        }
      }
      if (!a.dweights) continue;
#pragma unroll
      for (int j = 0; j < KB; ++j) dot[j] = wave_sum(dot[j]);
      if constexpr (THREADS == 64) {
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (lane == j && j0 + j < a.k) a.dweights[t * a.k + j0 + j] = dot[j];
      } else {
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < KB; ++j) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (tid < KB && j0 + tid < a.k) {
          float sum = 0.f;
          for (int q = 0; q < THREADS / 64; ++q) sum += part[q][tid];
          a.dweights[t * a.k + j0 + tid] = sum;
        }
        __syncthreads();
      }
    }
  }
}

// The widest pieces that rows of D values start on (the pointers are 16-byte
// aligned), and f with that as a template argument.
inline int piece_width(int64_t D) { return D % 8 == 0 ? 8 : D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1; }
template <int N>
struct Int {
  static constexpr int value = N;
};
template <class F>
void with_width(int vec, F f) {
  if (vec == 8) f(Int<8>{});
  else if (vec == 4) f(Int<4>{});
  else if (vec == 2) f(Int<2>{});
  else f(Int<1>{});
}

// Workgroups for n items, `per` each (more than kMaxBlocks: they loop).
constexpr int64_t kMaxBlocks = int64_t(1) << 22;
inline unsigned blocks_for(int64_t n, int64_t per) { return (unsigned)std::min(kMaxBlocks, (n + per - 1) / per); }

}  // namespace

int32_t moe_sort_chunk(int64_t n) {
  const int64_t c = (n + kMoeSortChunks - 1) / kMoeSortChunks;
  return (int32_t)std::max<int64_t>(1024, (c + 1023) / 1024 * 1024);
}

// Which form of the dispatch, and how many tokens a workgroup takes in the
// first two (measured in us on random experts, sort and copy unless said):
//  - one launch up to 12288 slots: every workgroup reads all of them (of 64
//    experts, 1024 columns: 4092 slots 5.4, counted first 7.6; 12288 8.7 and
//    9.9; 16380 11.2 and 11.8, but of 8 experts, 4096 columns 36.5 and 35.3;
//    of 2000 experts, 1024 columns: 12000 slots 10.5, counted and placed 19.3);
//  - counted first while the chunks' counts are few enough for every
//    workgroup to add up (16384 tokens, 2 of 256, 512 columns: 13.0; placed in
//    a launch of their own 15.7; 8 of 128, 1024 columns: 56.5 and 61.2),
//    without rows to copy only for as many workgroups as the CUs hold (those
//    131072 slots sorted alone: 15.0, and 9.4 placed);
//  - else counted, placed and copied in a launch each.
// A workgroup's share of the sort does not shrink with its tokens, so there
// are about kDispatchGroups workgroups (two a CU), not more (1000 tokens, 2
// of 8, 4096 columns: 7.5, with a workgroup a token 9.6; 6.0 since).
constexpr int64_t kOneLaunchSlots = 12288;
constexpr int64_t kFusedTable = 16384;     // counts
constexpr int64_t kFusedSlots = 1 << 20;   // (a chunk is then 2^14 slots, read by each of its workgroups)
constexpr int64_t kFusedSortGroups = 1024;
constexpr int64_t kDispatchGroups = 512;

hipError_t launch_moe_dispatch(const MoeDispatchArgs& args, hipStream_t s) {
  MoeDispatchArgs a = args;
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
  const int64_t T = a.n / a.k;
  const int vec = piece_width(a.D);
  const int64_t p = a.X ? a.D / vec : 0;
  if (a.n <= kOneLaunchSlots) a.chunks = 1;
  else
    hipLaunchKernelGGL(moe_count_kernel, dim3((unsigned)a.chunks), dim3(kSortThreads), (size_t)a.E * 4, s, a);
  const int G = (int)std::min<int64_t>(64 / a.k, std::max<int64_t>(1, (T + kDispatchGroups - 1) / kDispatchGroups));
  const int64_t fused_groups = std::max<int64_t>(1, (T + G - 1) / G);
  if (a.n <= kFusedSlots && (int64_t)a.chunks * a.E <= kFusedTable &&
      (a.X || fused_groups <= kFusedSortGroups)) {
    const dim3 grid((unsigned)fused_groups);
    // (up to 64 counters, one a bank, for few experts; chunks leave few ids to count)
    const int shift = a.chunks == 1 ? std::min(3, std::max(0, 6 - bits)) : 0;
    const size_t lds = ((size_t)a.E << shift) * 8;
    with_width(vec, [&](auto v) {
      hipLaunchKernelGGL(moe_dispatch_kernel<decltype(v)::value>, grid, dim3(kDispatchThreads), lds, s, a, T, G, bits,
                         shift, (int)p);
    });
    return hipGetLastError();
  }
  // (each wave's counters: 4 waves keep E = 4096 within 80 KB of LDS)
  const int waves = a.E <= 1024 ? 16 : 4;
  hipLaunchKernelGGL(moe_place_kernel, dim3((unsigned)a.chunks), dim3(kSortThreads), (size_t)a.E * (waves + 1) * 4, s,
                     a, waves, bits);
  if (a.X && a.n > 0) {
    const dim3 grid(blocks_for(T * p, kCopyThreads));
    with_width(vec, [&](auto v) {
      hipLaunchKernelGGL(moe_gather_kernel<decltype(v)::value>, grid, dim3(kCopyThreads), 0, s, a, p, T * p);
    });
  }
  return hipGetLastError();
}

// f with the row batch, and with or without caching, as template arguments.
template <class F>
void with_form(int k, bool nt, F f) {
  const auto go = [&](auto kb) { nt ? f(kb, Int<1>{}) : f(kb, Int<0>{}); };
  if (k <= 2) go(Int<2>{});
  else if (k <= 4) go(Int<4>{});
  else go(Int<8>{});
}

// A wave per token up to this many pieces of a row, a workgroup from there on
// (8192 tokens, 2 of 4096 columns: 58.5 us, a wave each 77; 20000 tokens, 8
// of 256 columns: 80.7 us, a wave each 40.1; equal at 1024 columns).
constexpr int kWavePieces = 96;

// From here on the gathered rows do not stay in the caches between the
// kernel that wrote them and this one, and reading them past the caches is
// faster (combine of 8192 tokens, 2 of 4096 columns, 134 MB: 34.9 against 37.4
// us); below, they do and it is slower (500 tokens, 8 of 4096 columns, 33
// MB: 10.4 against 8.3 us).
constexpr int64_t kStreamRowBytes = int64_t(64) << 20;

hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const int vec = piece_width(a.D);
  const int64_t p = a.D / vec, parts = (p + 63) / 64;
  const dim3 threads(kCopyThreads);
  with_form(a.k, a.T * a.k * a.D * 2 >= kStreamRowBytes, [&](auto kb, auto nt) {
    constexpr int KB = decltype(kb)::value;
    constexpr bool NT = decltype(nt)::value;
    if (vec == 8 && 4 * p >= 3 * 64 * parts) {  // (waves at least three quarters full)
      hipLaunchKernelGGL((moe_combine_kernel<8, KB, NT, true>), dim3(blocks_for(a.T * parts, kCopyThreads / 64)),
                         threads, 0, s, a, (int)parts, 64, a.T * parts);
    } else {
      with_width(vec, [&](auto v) {
        hipLaunchKernelGGL((moe_combine_kernel<decltype(v)::value, KB, NT, false>),
                           dim3(blocks_for(a.T * p, kCopyThreads)), threads, 0, s, a, 1, (int)p, a.T * p);
      });
    }
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const MoeCombineArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const int vec = piece_width(a.D);
  const int p = (int)(a.D / vec);
  const dim3 threads(kCopyThreads);
  with_form(a.k, a.T * a.k * a.D * 2 >= kStreamRowBytes, [&](auto kb, auto nt) {
    constexpr int KB = decltype(kb)::value;
    constexpr bool NT = decltype(nt)::value;
    with_width(vec, [&](auto v) {
      constexpr int VEC = decltype(v)::value;
      if (p > kWavePieces)
        hipLaunchKernelGGL((moe_combine_backward_kernel<VEC, 256, KB, NT>), dim3(blocks_for(a.T, 1)), threads, 0, s, a,
                           p);
      else
        hipLaunchKernelGGL((moe_combine_backward_kernel<VEC, 64, KB, NT>), dim3(blocks_for(a.T, 4)), threads, 0, s, a,
                           p);
    });
  });
  return hipGetLastError();
}

}  // namespace salr

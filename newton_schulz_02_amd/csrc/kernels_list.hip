// Kernels over lists of tensors for gfx950: the global gradient norm, clipping by it, and
// AdamW (muon_grad.h).
//
// A list is a table of tensors cut into chunks (list_plan.h); a workgroup takes chunks
// blockIdx.x, blockIdx.x + gridDim.x, ... and finds each one's tensor by a search over the
// tensors' first chunks.  All three kernels are HBM-bound: the norm reads every gradient once
// (one 4096-hidden layer in bf16, 405 MB: 69.6 us, 5.8 TB/s; 512 small fp32 matrices, 1.4 GB:
// 221 us, 6.4 TB/s), clipping reads and writes it once more (144 us, 5.6 TB/s; 488 us, 5.8
// TB/s), AdamW reads and writes its state once.  The squares' 64-bit sums hide under the
// loads: the inf norm, an integer maximum, takes 69.0 us on the same layer.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "list_math.h"
#include "muon_internal.h"

using namespace muon;

namespace {

__device__ __forceinline__ float ld_f(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float ld_f(const float* p) { return *p; }
__device__ __forceinline__ void st_f(uint16_t* p, float f) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ void st_f(float* p, float f) { *p = f; }

// The last entry whose first chunk is <= c (entries have at least one chunk each, the first
// entry's is 0).  The 64 lanes of a wave probe evenly spaced entries at once: a list of up to
// 64 tensors takes one round of loads, 4096 two.
template <typename Rec>
__device__ __forceinline__ int find(const Rec* recs, int count, uint32_t c) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = count;
  while (len > 1) {
    const int step = (len + 63) >> 6;
    const int at = lane * step;
    const bool below = at < len && recs[lo + at].first <= c;
    const int k = __popcll(__ballot(below)) - 1;
    lo += k * step;
    len = min(step, len - k * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// 16 bytes of S elements, read and written with one access wherever they lie: a tensor may
// start at any element (gfx950 takes unaligned 16-byte accesses; the address space keeps them
// global, since FLAT ones would also hold up the LDS waits).
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef u32x4 __attribute__((aligned(4))) u32x4_at4;
template <typename S>
struct Vec {
  static constexpr int N = 16 / sizeof(S);
  u32x4 v;
  __device__ __forceinline__ void load(const S* p) {
    if constexpr (sizeof(S) == 2) v = *(__attribute__((address_space(1))) const u32x4_at2*)(p);
    else v = *(__attribute__((address_space(1))) const u32x4_at4*)(p);
  }
  __device__ __forceinline__ void store(S* p) const {
    if constexpr (sizeof(S) == 2) *(__attribute__((address_space(1))) u32x4_at2*)(p) = v;
    else *(__attribute__((address_space(1))) u32x4_at4*)(p) = v;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(S) == 4) return __uint_as_float(v[e]);
    else return __uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
  }
  // All N elements, rounded to S.
  __device__ __forceinline__ void set(const float (&f)[N]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(S) == 4) {
        v[q] = __float_as_uint(f[q]);
      } else {
        v[q] = uint32_t(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f[2 * q]))) |
               uint32_t(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f[2 * q + 1]))) << 16;
      }
    }
  }
};

// Partial result: squares and sums in 64 bits, so that neither the smallest nor the largest
// fp32 gradient leaves the range (two sums, so that one addition need not wait for the last);
// for the inf norm the magnitudes' bits, whose order as integers puts infinity above all
// numbers and NaN above infinity.
struct Part {
  double sum[2] = {0.0, 0.0};
  uint32_t top = 0;
  template <bool INF>
  __device__ __forceinline__ void take(float g, int e) {
    if constexpr (INF) top = max(top, __float_as_uint(g) & 0x7fffffffu);
    else sum[e & 1] = fma(double(g), double(g), sum[e & 1]);
  }
};

// A piece of a chunk: the elements [lo, hi) of the BYTES bytes behind p.  Chunks start on line
// boundaries, the first one at or before its tensor, so lanes read and write whole lines
// wherever the tensor starts (with chunks counted from the tensor's own start, an odd one cost
// 13 % on a bf16 norm).
template <typename S, int BYTES>
struct Piece {
  S* p;
  int lo, hi;
  static constexpr int kAll = BYTES / int(sizeof(S));
};
// Piece h of chunk c of the tensor; empty (hi <= lo) behind the tensor's end.
template <typename S, int BYTES>
__device__ __forceinline__ Piece<S, BYTES> piece_of(const GradRec& r, uint32_t c, int h = 0) {
  const int shift = int(r.ptr % kLine / sizeof(S));
  const int64_t at = int64_t(c - r.first) * (kGradChunk / int64_t(sizeof(S))) + h * Piece<S, BYTES>::kAll - shift;
  Piece<S, BYTES> x;
  x.p = reinterpret_cast<S*>(r.ptr) + at;
  x.lo = at < 0 ? int(-at) : 0;
  x.hi = int(min(int64_t(Piece<S, BYTES>::kAll), r.n - at));
  return x;
}

// f(vector) for each of this thread's vectors of a piece; STORE: write them back.  A whole
// piece has all its loads in flight before the first vector is used; else vectors that reach
// outside go element by element (with zeros for what is outside, which change neither a sum
// nor a maximum).
template <bool STORE, typename S, int BYTES, typename F>
__device__ __forceinline__ void each_vec(const Piece<S, BYTES>& x, F&& f) {
  constexpr int N = Vec<S>::N, U = BYTES / (256 * 16);
  const int tid = threadIdx.x;
  if (x.lo == 0 && x.hi == x.kAll) {
    Vec<S> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u].load(x.p + (u * 256 + tid) * N);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f(v[u]);
      if (STORE) v[u].store(x.p + (u * 256 + tid) * N);
    }
    return;
  }
  for (int i = tid * N; i < x.hi; i += 256 * N) {
    Vec<S> v;
    if (i >= x.lo && i + N <= x.hi) {
      v.load(x.p + i);
      f(v);
      if (STORE) v.store(x.p + i);
      continue;
    }
    float e[N];
#pragma unroll
    for (int k = 0; k < N; ++k) e[k] = i + k >= x.lo && i + k < x.hi ? ld_f(x.p + i + k) : 0.0f;
    v.set(e);
    f(v);
    if (STORE) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (i + k >= x.lo && i + k < x.hi) st_f(x.p + i + k, v.get(k));
    }
  }
}

template <bool INF>
__device__ __forceinline__ Part norm_chunks(const GradArgs& a) {
  Part part;
  auto take = [&](const auto& v) {
#pragma unroll
    for (int e = 0; e < std::decay_t<decltype(v)>::N; ++e) part.template take<INF>(v.get(e), e);
  };
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const GradRec r = a.recs[find(a.recs, a.count, c)];
    if (r.dtype == kBF16) each_vec<false>(piece_of<uint16_t, kGradChunk>(r, c), take);
    else each_vec<false>(piece_of<float, kGradChunk>(r, c), take);
  }
  return part;
}

// Sum, or maximum, over a workgroup in a fixed order; the result is thread 0's.
__device__ __forceinline__ double combine(double x, double y, bool inf) { return inf ? (x > y ? x : y) : x + y; }
__device__ __forceinline__ double reduce(double x, bool inf, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = combine(x, __shfl_xor(x, off, 64), inf);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  return combine(combine(red[0], red[1], inf), combine(red[2], red[3], inf), inf);
}

// The workgroup that finishes last adds up all partial results, always in the same order, so
// one launch does the whole norm.  Partial results pass between XCDs, whose L2s are not
// coherent with each other: they are stored and loaded at device scope, and a store is
// complete (s_waitcnt) before its workgroup counts itself.  No device-wide release: it writes
// back a whole L2, and one per workgroup took 36 us over 1024 workgroups.  Counts of one
// address are made one after another (10 ns each), so a workgroup counts itself among those
// with its index modulo kTickets, and the last of each of these among the last ones.  All
// counts are back at 0 at the end.
__device__ __forceinline__ uint32_t count_self(uint32_t* ticket) {
  return __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__global__ __launch_bounds__(256) void k_grad_norm(GradArgs a) {
  __shared__ double red[4], red_all[4];
  __shared__ bool last;
  const bool inf = a.inf;
  const Part part = inf ? norm_chunks<true>(a) : norm_chunks<false>(a);
  double x = reduce(inf ? double(part.top) : part.sum[0] + part.sum[1], inf, red);
  const unsigned grid = gridDim.x;
  if (grid > 1) {
    if (threadIdx.x == 0) {
      __hip_atomic_store(a.parts + blockIdx.x, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __builtin_amdgcn_s_waitcnt(0);
      const unsigned mine = blockIdx.x % kTickets;
      uint32_t* ticket = a.tickets + (1 + mine) * (kLine / 4);
      last = count_self(ticket) == (grid - mine - 1) / kTickets;
      if (last) {
        __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = count_self(a.tickets) == min(grid, unsigned(kTickets)) - 1;
        if (last) __hip_atomic_store(a.tickets, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    __syncthreads();
    if (!last) return;
    x = 0.0;
    for (unsigned i = threadIdx.x; i < grid; i += 256)
      x = combine(x, __hip_atomic_load(a.parts + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), inf);
    x = reduce(x, inf, red_all);
  }
  if (threadIdx.x == 0) *a.norm = inf ? __uint_as_float(uint32_t(x)) : float(sqrt(x));
}

template <typename S>
__device__ __forceinline__ void scale_vec(Vec<S>& x, float coef) {
  float f[Vec<S>::N];
#pragma unroll
  for (int e = 0; e < Vec<S>::N; ++e) f[e] = coef * x.get(e);
  x.set(f);
}

__global__ __launch_bounds__(256) void k_grad_clip(GradArgs a) {
  const float coef = clip_coef(a.clip);
  if (coef == 1.0f) return;
  auto scale = [=](auto& v) { scale_vec(v, coef); };
  // By half chunks (512 small fp32 matrices, 1.4 GB: 488 us by 16 KiB, 534 by 32 KiB, 576 by
  // 8 KiB), a workgroup each up to 65536 of them (2048 looping ones: 538), and backwards, since
  // what the norm read last may still be in the memory-side cache (1 % of a layer's clipping).
  for (uint32_t b = blockIdx.x; b < 2 * a.chunks; b += gridDim.x) {
    const uint32_t h = 2 * a.chunks - 1 - b;
    const uint32_t c = h >> 1;
    const GradRec r = a.recs[find(a.recs, a.count, c)];
    if (r.dtype == kBF16) each_vec<true>(piece_of<uint16_t, kGradChunk / 2>(r, c, h & 1), scale);
    else each_vec<true>(piece_of<float, kGradChunk / 2>(r, c, h & 1), scale);
  }
}

// n elements from element `at` of one tensor; a master takes the place of the param as what
// is updated.
template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void adamw_chunk(const AdamRec& r, int64_t at, int64_t n, float coef,
                                            const AdamListArgs& a) {
  P* p = reinterpret_cast<P*>(r.param) + at;
  const G* g = reinterpret_cast<const G*>(r.grad) + at;
  float* m = reinterpret_cast<float*>(r.m) + at;
  float* v = reinterpret_cast<float*>(r.v) + at;
  float* w = reinterpret_cast<float*>(r.master) + at;
  const float wd = a.wd * r.decay;
  for (int64_t i = threadIdx.x; i < n; i += 256) {
    float x = MASTER ? w[i] : ld_f(p + i), mi = m[i], vi = v[i];
    adamw_one(x, coef * ld_f(g + i), mi, vi, a, wd);
    m[i] = mi;
    v[i] = vi;
    if (MASTER) w[i] = x;
    st_f(p + i, x);
  }
}

__global__ __launch_bounds__(256) void k_adamw_list(AdamListArgs a) {
  const float coef = clip_coef(a.clip);
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const AdamRec& r = a.recs[find(a.recs, a.count, c)];
    const int64_t at = int64_t(c - r.first) * kAdamChunk;
    const int64_t n = min(kAdamChunk, r.n - at);
    if (!r.param_bf16) {
      if (r.grad_bf16) adamw_chunk<float, uint16_t, false>(r, at, n, coef, a);
      else adamw_chunk<float, float, false>(r, at, n, coef, a);
    } else if (r.master) {
      if (r.grad_bf16) adamw_chunk<uint16_t, uint16_t, true>(r, at, n, coef, a);
      else adamw_chunk<uint16_t, float, true>(r, at, n, coef, a);
    } else {
      if (r.grad_bf16) adamw_chunk<uint16_t, uint16_t, false>(r, at, n, coef, a);
      else adamw_chunk<uint16_t, float, false>(r, at, n, coef, a);
    }
  }
}

unsigned grid_of(uint32_t chunks, uint32_t most) { return chunks < most ? chunks : most; }

}  // namespace

int muon_launch_grad_norm(const GradArgs& a, void* stream) {
  const unsigned grid = a.chunks ? grid_of(a.chunks, kNormParts) : 1;  // no gradients: the norm is 0
  hipLaunchKernelGGL(k_grad_norm, dim3(grid), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

int muon_launch_grad_clip(const GradArgs& a, void* stream) {
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_clip, dim3(grid_of(2 * a.chunks, 1u << 16)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

int muon_launch_adamw_list(const AdamListArgs& a, void* stream) {
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_adamw_list, dim3(grid_of(a.chunks, 1u << 16)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

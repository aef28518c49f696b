// Kernels over lists of tensors for gfx950: the global gradient norm, clipping by it, and
// AdamW (muon_grad.h).
//
// A list is a table of tensors cut into chunks (list_plan.h); a workgroup takes chunks
// blockIdx.x, blockIdx.x + gridDim.x, ... and finds each one's tensor by a search over the
// tensors' first chunks.  All three kernels are HBM-bound: the norm reads every gradient once,
// clipping reads and writes it once more, AdamW reads and writes its state once.
#include <hip/hip_runtime.h>

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

// The last entry whose first chunk is <= c (entries have at least one chunk each).
template <typename Rec>
__device__ __forceinline__ int find(const Rec* recs, int count, uint32_t c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (recs[mid].first <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
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

// One chunk: kGradChunk bytes as four 16-byte loads per thread, all in flight before the first
// is used; the last chunk of a tensor vector by vector, then element by element.
template <typename S, bool INF>
__device__ __forceinline__ void norm_chunk(const S* p, int64_t n, Part& part) {
  constexpr int N = Vec<S>::N, U = kGradChunk / (256 * 16);
  const int tid = threadIdx.x;
  if (n == kGradChunk / int64_t(sizeof(S))) {
    Vec<S> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(p + (u * 256 + tid) * N);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) part.template take<INF>(x[u].get(e), e);
    return;
  }
  const int vecs = int(n) / N;
  for (int i = tid; i < vecs; i += 256) {
    Vec<S> x;
    x.load(p + i * N);
#pragma unroll
    for (int e = 0; e < N; ++e) part.template take<INF>(x.get(e), e);
  }
  const int i = vecs * N + tid;
  if (i < int(n)) part.template take<INF>(ld_f(p + i), 0);
}

template <bool INF>
__device__ __forceinline__ Part norm_chunks(const GradArgs& a) {
  Part part;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const GradRec r = a.recs[find(a.recs, a.count, c)];
    const int64_t per = r.dtype == kBF16 ? kGradChunk / 2 : kGradChunk / 4;
    const int64_t at = int64_t(c - r.first) * per;
    const int64_t n = min(per, r.n - at);
    if (r.dtype == kBF16) norm_chunk<uint16_t, INF>(reinterpret_cast<const uint16_t*>(r.ptr) + at, n, part);
    else norm_chunk<float, INF>(reinterpret_cast<const float*>(r.ptr) + at, n, part);
  }
  return part;
}

__global__ __launch_bounds__(256) void k_grad_norm(GradArgs a) {
  const Part part = a.inf ? norm_chunks<true>(a) : norm_chunks<false>(a);
  __shared__ double red[256];
  red[threadIdx.x] = a.inf ? double(part.top) : part.sum[0] + part.sum[1];
  __syncthreads();
  for (int s = 128; s > 0; s >>= 1) {
    if (int(threadIdx.x) < s) {
      const double x = red[threadIdx.x], y = red[threadIdx.x + s];
      red[threadIdx.x] = a.inf ? (x > y ? x : y) : x + y;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) a.parts[blockIdx.x] = red[0];
}

// The partial results' sum (or maximum) in a fixed order, and the norm.
__global__ __launch_bounds__(256) void k_grad_norm_end(GradArgs a) {
  __shared__ double red[256];
  double x = 0.0;
  for (int i = threadIdx.x; i < a.nparts; i += 256) x = a.inf ? (a.parts[i] > x ? a.parts[i] : x) : x + a.parts[i];
  red[threadIdx.x] = x;
  __syncthreads();
  for (int s = 128; s > 0; s >>= 1) {
    if (int(threadIdx.x) < s) {
      const double u = red[threadIdx.x], w = red[threadIdx.x + s];
      red[threadIdx.x] = a.inf ? (u > w ? u : w) : u + w;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.norm = a.inf ? __uint_as_float(uint32_t(red[0])) : float(sqrt(red[0]));
}

template <typename S>
__device__ __forceinline__ void scale_vec(Vec<S>& x, float coef) {
  float f[Vec<S>::N];
#pragma unroll
  for (int e = 0; e < Vec<S>::N; ++e) f[e] = coef * x.get(e);
  x.set(f);
}

template <typename S>
__device__ __forceinline__ void clip_chunk(S* p, int64_t n, float coef) {
  constexpr int N = Vec<S>::N, U = kGradChunk / (256 * 16);
  const int tid = threadIdx.x;
  if (n == kGradChunk / int64_t(sizeof(S))) {
    Vec<S> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(p + (u * 256 + tid) * N);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      scale_vec(x[u], coef);
      x[u].store(p + (u * 256 + tid) * N);
    }
    return;
  }
  const int vecs = int(n) / N;
  for (int i = tid; i < vecs; i += 256) {
    Vec<S> x;
    x.load(p + i * N);
    scale_vec(x, coef);
    x.store(p + i * N);
  }
  const int i = vecs * N + tid;
  if (i < int(n)) st_f(p + i, coef * ld_f(p + i));
}

__global__ __launch_bounds__(256) void k_grad_clip(GradArgs a) {
  const float coef = clip_coef(a.clip);
  if (coef == 1.0f) return;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const GradRec r = a.recs[find(a.recs, a.count, c)];
    const int64_t per = r.dtype == kBF16 ? kGradChunk / 2 : kGradChunk / 4;
    const int64_t at = int64_t(c - r.first) * per;
    const int64_t n = min(per, r.n - at);
    if (r.dtype == kBF16) clip_chunk(reinterpret_cast<uint16_t*>(r.ptr) + at, n, coef);
    else clip_chunk(reinterpret_cast<float*>(r.ptr) + at, n, coef);
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

int muon_launch_grad_norm(const GradArgs& args, void* stream) {
  GradArgs a = args;
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.nparts = int32_t(grid_of(a.chunks, kNormParts));
  if (a.nparts > 0) {
    hipLaunchKernelGGL(k_grad_norm, dim3(unsigned(a.nparts)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_grad_norm_end, dim3(1), dim3(256), 0, s, a);
  return hipGetLastError();
}

int muon_launch_grad_clip(const GradArgs& a, void* stream) {
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_clip, dim3(grid_of(a.chunks, 1u << 16)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

int muon_launch_adamw_list(const AdamListArgs& a, void* stream) {
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_adamw_list, dim3(grid_of(a.chunks, 1u << 16)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

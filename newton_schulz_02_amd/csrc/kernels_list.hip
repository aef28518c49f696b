// Kernels over lists of tensors for gfx950: the global gradient norm, clipping by it, and
// AdamW (muon_grad.h).
//
// A list is a table of tensors cut into chunks (list_plan.h); a workgroup takes chunks
// blockIdx.x, blockIdx.x + gridDim.x, ... and finds each one's tensor in the list's map.  All
// three kernels are HBM-bound:
//   norm   reads every gradient once: one 4096-hidden layer in bf16 (405 MB) in 64 us, 6.3
//          TB/s; 512 small fp32 matrices (1.4 GB) in 197 us, 7.2 TB/s.  The squares' 64-bit
//          sums hide under the loads: the inf norm, an integer maximum, takes as long.
//   clip   reads and writes them: 128 us, 6.3 TB/s; 476 us, 5.9 TB/s.
//   AdamW  reads and writes its state once: two 32000 x 4096 embeddings with masters and bf16
//          gradients (7.3 GB) in 1.19 ms, 6.2 TB/s.
// (Medians of each kernel alone, launched in turn over three sets of tensors.  Times beside a
// choice below are of calls queued one behind the other, a few per cent shorter, and of one run
// each.  A copy by the runtime's own kernel moves 4.9 TB/s on the same card.)
#include <hip/hip_runtime.h>

#include <type_traits>

#include "list_math.h"

using namespace muon;

namespace {

__device__ __forceinline__ float ld_f(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float ld_f(const float* p) { return *p; }
__device__ __forceinline__ void st_f(uint16_t* p, float f) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ void st_f(float* p, float f) { *p = f; }

// map[c] <- the tensor of chunk c: the last entry whose first chunk is <= c (entries have at
// least one chunk each, the first entry's is 0).  Run once per list, so that the kernels below
// find a chunk's tensor by one load: a search there, three loads one behind the other, was a
// third of a workgroup's time in AdamW over 1000 tensors.
template <typename Rec>
__global__ __launch_bounds__(256) void k_list_map(const Rec* recs, int count, uint32_t chunks, uint32_t* map) {
  const uint32_t step = gridDim.x * 256u;
  for (uint64_t c = blockIdx.x * 256u + threadIdx.x; c < chunks; c += step) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (recs[mid].first <= c) lo = mid; else hi = mid - 1;
    }
    map[c] = uint32_t(lo);
  }
}

// 16 bytes of S elements, read and written with one access.  Chunks start on line boundaries, so
// the accesses of norm and clip are aligned wherever a tensor starts; the types say no more than
// an element's alignment (which gfx950 takes too, and which AdamW's load4 and store4 need, whose
// buffers lie differently).  The address space keeps them global, since FLAT ones would also
// hold up the LDS waits.  Non-temporal, as every list
// access below: nothing is used twice by one kernel.  That is worth a tenth: the norm of a bf16
// layer takes 63.6 us with it and 70.4 us without, its clipping 126 and 145 us.
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef u32x4 __attribute__((aligned(4))) u32x4_at4;
template <typename S>
struct Vec {
  static constexpr int N = 16 / sizeof(S);
  u32x4 v;
  __device__ __forceinline__ void load(const S* p) {
    if constexpr (sizeof(S) == 2) v = __builtin_nontemporal_load((__attribute__((address_space(1))) const u32x4_at2*)(p));
    else v = __builtin_nontemporal_load((__attribute__((address_space(1))) const u32x4_at4*)(p));
  }
  __device__ __forceinline__ void store(S* p) const {
    if constexpr (sizeof(S) == 2) __builtin_nontemporal_store(v, (__attribute__((address_space(1))) u32x4_at2*)(p));
    else __builtin_nontemporal_store(v, (__attribute__((address_space(1))) u32x4_at4*)(p));
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

// The elements of [lo, hi) that no whole vector of n elements covers, up to n - 1 at each end:
// one per thread, -1 for a thread without one.
__device__ __forceinline__ int edge_of(int lo, int hi, int n) {
  const int head = min(hi, (lo + n - 1) / n * n), tail = max(head, hi / n * n);
  const int i = lo + int(threadIdx.x);
  if (i < head) return i;
  return i - head + tail < hi ? i - head + tail : -1;
}

// f on each of this thread's vectors of a piece (and on single elements at the ends of one that
// is not whole); STORE: write them back.  All loads are in flight before the first use, in a
// piece that is not whole, too: one vector after the other there, the norm of 23 ragged
// tensors took 10.0 us instead of 6.5.
template <bool STORE, typename S, int BYTES, typename F>
__device__ __forceinline__ void each_vec(const Piece<S, BYTES>& x, F&& f) {
  constexpr int N = Vec<S>::N, U = BYTES / (256 * 16);
  const int tid = threadIdx.x;
  Vec<S> v[U];
  if (x.lo == 0 && x.hi == x.kAll) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u].load(x.p + (u * 256 + tid) * N);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f(v[u]);
      if (STORE) v[u].store(x.p + (u * 256 + tid) * N);
    }
    return;
  }
  if (x.hi <= x.lo) return;
  const int at = edge_of(x.lo, x.hi, N);
  float edge = at >= 0 ? ld_f(x.p + at) : 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * 256 + tid) * N;
    v[u].v = 0;  // zeros change neither a sum nor a maximum
    if (i >= x.lo && i + N <= x.hi) v[u].load(x.p + i);
  }
  f(edge);
  if (STORE && at >= 0) st_f(x.p + at, edge);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * 256 + tid) * N;
    f(v[u]);
    if (STORE && i >= x.lo && i + N <= x.hi) v[u].store(x.p + i);
  }
}

template <bool INF>
struct Take {
  Part& part;
  template <typename S>
  __device__ __forceinline__ void operator()(const Vec<S>& v) {
#pragma unroll
    for (int e = 0; e < Vec<S>::N; ++e) part.template take<INF>(v.get(e), e);
  }
  __device__ __forceinline__ void operator()(float g) { part.template take<INF>(g, 0); }
};

template <bool INF>
__device__ __forceinline__ Part norm_chunks(const GradArgs& a) {
  Part part;
  Take<INF> take{part};
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const GradRec r = a.recs[a.map[c]];
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
// with its index modulo kTickets, and the last of each of these among the last ones; up to 64
// workgroups count themselves at once.  A count goes back to 0 by the increment that completes
// it, not by a store: also where two norms of a list overlap, against the rule, every count is 0
// when both have ended, and the list's next norm is right.
__device__ __forceinline__ bool count_self(uint32_t* ticket, uint32_t all) {
  return atomicInc(ticket, all - 1) == all - 1;  // device scope, relaxed
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
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const bool few = grid <= 64;
      bool done = true;
      if (!few) {
        const unsigned mine = blockIdx.x % kTickets;
        uint32_t* ticket = a.tickets + (1 + mine) * (kLine / 4);
        done = count_self(ticket, (grid - mine - 1) / kTickets + 1);
      }
      if (done) done = count_self(a.tickets, few ? grid : unsigned(kTickets));
      last = done;
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

struct Scale {
  float coef;
  template <typename S>
  __device__ __forceinline__ void operator()(Vec<S>& v) {
    float f[Vec<S>::N];
#pragma unroll
    for (int e = 0; e < Vec<S>::N; ++e) f[e] = coef * v.get(e);
    v.set(f);
  }
  __device__ __forceinline__ void operator()(float& g) { g *= coef; }
};

__global__ __launch_bounds__(256) void k_grad_clip(GradArgs a) {
  const float coef = clip_coef(a.clip);
  if (coef == 1.0f) return;
  Scale scale{coef};
  // By half chunks (512 small fp32 matrices, 1.4 GB, a workgroup for each: 450 us by 16 KiB, 475
  // by 32 KiB and by 8 KiB; 468 by 16 KiB in the grid below), and backwards, since what the norm
  // read last may still be in the memory-side cache (1 % of a layer's clipping).
  for (uint32_t b = blockIdx.x; b < 2 * a.chunks; b += gridDim.x) {
    const uint32_t h = 2 * a.chunks - 1 - b;
    const uint32_t c = h >> 1;
    const GradRec r = a.recs[a.map[c]];
    if (r.dtype == kBF16) each_vec<true>(piece_of<uint16_t, kGradChunk / 2>(r, c, h & 1), scale);
    else each_vec<true>(piece_of<float, kGradChunk / 2>(r, c, h & 1), scale);
  }
}

// Four neighbouring elements, as one access at any alignment (16 bytes of fp32, 8 of bf16), or
// those of them in [lo, hi) one by one.
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 __attribute__((aligned(2))) u32x2_at2;
typedef uint16_t bf16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const u32x4 v = __builtin_nontemporal_load((__attribute__((address_space(1))) const u32x4_at4*)(p));
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(v[k]);
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&f)[4]) {
  const u32x2 v = __builtin_nontemporal_load((__attribute__((address_space(1))) const u32x2_at2*)(p));
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(k & 1 ? v[k >> 1] & 0xffff0000u : v[k >> 1] << 16);
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
  u32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __float_as_uint(f[k]);
  __builtin_nontemporal_store(v, (__attribute__((address_space(1))) u32x4_at4*)(p));
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&f)[4]) {
  bf16x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f[k]));
  __builtin_nontemporal_store(__builtin_bit_cast(u32x2, v), (__attribute__((address_space(1))) u32x2_at2*)(p));
}
// The elements of chunk c of one tensor; a master takes the place of the param as what is
// updated.  Chunks start where m lies on a line boundary, so buffers that lie alike (those of
// one flat bucket per type) are all read and written by whole lines.
// All loads of a whole chunk are in flight before the first update: 16 bytes of fp32 per lane
// and load, two of each buffer.  Non-temporal loads and stores together are worth a tenth
// (embeddings with masters 1.36 -> 1.21 ms), either alone nothing.  Dividing by reciprocals
// instead changes nothing: the arithmetic hides under the loads.
template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void adamw_chunk(const AdamRec& r, uint32_t c, float coef, const AdamListArgs& a) {
  typedef std::conditional_t<MASTER, float, P> X;
  const int64_t at = int64_t(c - r.first) * kAdamChunk - int64_t(r.m % kLine / 4);
  P* p = reinterpret_cast<P*>(r.param) + at;
  X* x = reinterpret_cast<X*>(MASTER ? r.master : r.param) + at;
  const G* g = reinterpret_cast<const G*>(r.grad) + at;
  float* m = reinterpret_cast<float*>(r.m) + at;
  float* v = reinterpret_cast<float*>(r.v) + at;
  const float wd = a.wd * r.decay;
  const int tid = threadIdx.x;
  constexpr int U = int(kAdamChunk) / 1024;
  float xs[U][4], gs[U][4], ms[U][4], vs[U][4];
  if (at >= 0 && r.n - at >= kAdamChunk) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (u * 256 + tid) * 4;
      load4(x + i, xs[u]);
      load4(g + i, gs[u]);
      load4(m + i, ms[u]);
      load4(v + i, vs[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (u * 256 + tid) * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) adamw_one(xs[u][k], coef * gs[u][k], ms[u][k], vs[u][k], a, a.betas, wd);
      store4(m + i, ms[u]);
      store4(v + i, vs[u]);
      store4(x + i, xs[u]);
      if (MASTER) store4(p + i, xs[u]);
    }
    return;
  }
  // The first or last chunk of a tensor: vectors inside it, and up to three single elements at
  // each end.
  const int lo = at < 0 ? int(-at) : 0;
  const int hi = int(min(kAdamChunk, r.n - at));
  const int e = edge_of(lo, hi, 4);
  float xe = 0.0f, ge = 0.0f, me = 0.0f, ve = 0.0f;
  if (e >= 0) {
    xe = ld_f(x + e);
    ge = ld_f(g + e);
    me = m[e];
    ve = v[e];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * 256 + tid) * 4;
    if (i < lo || i + 4 > hi) continue;
    load4(x + i, xs[u]);
    load4(g + i, gs[u]);
    load4(m + i, ms[u]);
    load4(v + i, vs[u]);
  }
  if (e >= 0) {
    adamw_one(xe, coef * ge, me, ve, a, a.betas, wd);
    m[e] = me;
    v[e] = ve;
    st_f(x + e, xe);
    if (MASTER) st_f(p + e, xe);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * 256 + tid) * 4;
    if (i < lo || i + 4 > hi) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) adamw_one(xs[u][k], coef * gs[u][k], ms[u][k], vs[u][k], a, a.betas, wd);
    store4(m + i, ms[u]);
    store4(v + i, vs[u]);
    store4(x + i, xs[u]);
    if (MASTER) store4(p + i, xs[u]);
  }
}

// Workgroups go to the eight XCDs in turn: each round of 128 chunks gives every XCD 16
// neighbouring ones, longer runs of each of the nine streams.  us with 1 / 8 / 16 / 32:
// embeddings with masters 1211 / 1227 / 1161 / 1162, fp32 303 / 303 / 296 / 307, bf16 467 / 466 /
// 456 / 456; the norm and clipping, of one stream or two, gain nothing.
__device__ __forceinline__ uint32_t chunk_of(uint32_t b, uint32_t chunks) {
  constexpr uint32_t kRun = 16, kRound = 8 * kRun;
  const uint32_t base = b / kRound * kRound, i = b - base;
  return base + kRound > chunks ? b : base + i % 8 * kRun + i / 8;
}

__global__ __launch_bounds__(256) void k_adamw_list(AdamListArgs a) {
  const float coef = clip_coef(a.clip);
  for (uint32_t b = blockIdx.x; b < a.chunks; b += gridDim.x) {
    const uint32_t c = chunk_of(b, a.chunks);
    const AdamRec& r = a.recs[a.map[c]];
    if (!r.param_bf16) {
      if (r.grad_bf16) adamw_chunk<float, uint16_t, false>(r, c, coef, a);
      else adamw_chunk<float, float, false>(r, c, coef, a);
    } else if (r.master) {
      if (r.grad_bf16) adamw_chunk<uint16_t, uint16_t, true>(r, c, coef, a);
      else adamw_chunk<uint16_t, float, true>(r, c, coef, a);
    } else {
      if (r.grad_bf16) adamw_chunk<uint16_t, uint16_t, false>(r, c, coef, a);
      else adamw_chunk<uint16_t, float, false>(r, c, coef, a);
    }
  }
}

// AdamW: a workgroup for each chunk; 2048 or 4096 looping ones took a tenth longer (loading a
// chunk ahead of the last one's stores did not help clipping, which is alike).  Clipping: at
// most 32768, since a launch that finds nothing to clip, the usual one in a settled run, costs
// 20 us by 86000 workgroups and 8 by 32768; clipping those 1.4 GB takes 459 and 468 us.
constexpr uint32_t kMostGroups = 1u << 20, kMostClipGroups = 1u << 15;
unsigned grid_of(uint32_t chunks, uint32_t most) { return chunks < most ? chunks : most; }

template <typename Rec>
int launch_map(const Rec* recs, int count, uint32_t chunks, uint32_t* map, void* stream) {
  if (chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_list_map<Rec>, dim3(grid_of(uint32_t(ceil_div(chunks, 256)), 4096)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), recs, count, chunks, map);
  return hipGetLastError();
}

}  // namespace

int muon_launch_grad_map(const GradRec* recs, int count, uint32_t chunks, uint32_t* map, void* stream) {
  return launch_map(recs, count, chunks, map, stream);
}
int muon_launch_adamw_map(const AdamRec* recs, int count, uint32_t chunks, uint32_t* map, void* stream) {
  return launch_map(recs, count, chunks, map, stream);
}

int muon_launch_grad_norm(const GradArgs& a, void* stream) {
  const unsigned grid = a.chunks ? grid_of(a.chunks, kNormParts) : 1;  // no gradients: the norm is 0
  hipLaunchKernelGGL(k_grad_norm, dim3(grid), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

int muon_launch_grad_clip(const GradArgs& a, void* stream) {
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_clip, dim3(grid_of(2 * a.chunks, kMostClipGroups)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

int muon_launch_adamw_list(const AdamListArgs& a, void* stream) {
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_adamw_list, dim3(grid_of(a.chunks, kMostGroups)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return hipGetLastError();
}

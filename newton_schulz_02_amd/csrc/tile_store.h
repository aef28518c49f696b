// From accumulators to rows of the result, for the products of the 8-bit linear operators.
//
// A wave's block of FM x FN matrix-instruction results (32 x 32 each): operand order is chosen so
// that lane l holds, of result row 32 i + l % 32, the columns 32 j + 8 g + 4 (l / 32) + 0..3 in
// acc[i][j][4 g .. 4 g + 3].  32 rows at a time go through LDS (each wave its own part, so no
// barrier), and come back as runs of 16 bytes of the result, neighbouring lanes on neighbouring
// runs, so that whole lines are read and written.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_math.h"

namespace muon {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>).
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// 16 bytes of a result of T: E values of one row.
template <typename T>
struct Run {
  static constexpr int E = 16 / int(sizeof(T));
  u32x4 v;
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(v[e]);
    else return __uint_as_float(e & 1 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(f[i]);
      else v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    }
  }
  // At any alignment of T.  Non-temporal as the stores, but not for bf16, where a run is half of what
  // the lane beside it will ask for again (an fp32 gradient of 4096 x 4096 added to: 33.4 -> 30.0
  // us for 128 tokens; a bf16 one 16.5 -> 17.9).
  using At = typename std::conditional<sizeof(T) == 4, u32x4_at4, u32x4_at2>::type;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) == 4) v = __builtin_nontemporal_load((global_ptr<const At>)(p));
    else v = *(global_ptr<const At>)(p);
  }
  // A run of a row of `cols` values that may end before it.  Of a row of E values or more the load
  // is one access, that of the row's last E values where the run passes the end, and `settle` moves
  // them into place when they are used: no branch, so that loads are not waited for one by one.
  __device__ __forceinline__ void load_edge(const T* row, int col, int cols) {
    if (cols >= E) {
      load(row + min(col, cols - E));
    } else {
      v = 0;
#pragma unroll
      for (int e = 0; e < E - 1; ++e)
        if (col + e < cols) {
          if constexpr (sizeof(T) == 4) v[e] = *(global_ptr<const uint32_t>)(row + col + e);
          else v[e / 2] |= uint32_t(*(global_ptr<const uint16_t>)(row + col + e)) << (16 * (e & 1));
        }
    }
  }
  __device__ __forceinline__ void settle(int col, int cols) {
    int by = cols >= E ? max(0, col + E - cols) : 0;  // values to move down
    if constexpr (sizeof(T) == 2) {
      if (by & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
      by >>= 1;
    }
    if (by & 1) v = u32x4{v[1], v[2], v[3], 0};
    if (by & 2) v = u32x4{v[2], v[3], 0, 0};
  }
  template <bool WHOLE>
  __device__ __forceinline__ void store(T* row, int col, int cols) const {
    if (WHOLE || col + E <= cols) {
      __builtin_nontemporal_store(v, (global_ptr<At>)(row + col));
    } else {
#pragma unroll
      for (int e = 0; e < E - 1; ++e)
        if (col + e < cols) {
          if constexpr (sizeof(T) == 4) *(global_ptr<uint32_t>)(row + col + e) = v[e];
          else *(global_ptr<uint16_t>)(row + col + e) = uint16_t(v[e / 2] >> (16 * (e & 1)));
        }
    }
  }
};

// Floats of a wave's part: 32 rows of FN * 32 columns and 4 floats (so that rows start in
// different banks).
template <int FN>
constexpr int store_floats() {
  return 32 * (FN * 32 + 4);
}

// Column of a lane's runs (of E values) within its wave's block.
template <int FN, int E>
__device__ __forceinline__ int store_col() {
  return int(threadIdx.x & 63) % (FN * 32 / E) * E;
}

// For every run of a wave's block: put(row, its E accumulators, fetch(row)), with the row within the
// block; the fetches of 32 rows are in flight while the 32 before are put.  DRAIN: put has branches,
// behind which the compiler no longer knows which loads are done and waits for all accesses, the
// stores among them, at every run; the loads are waited for once, before the stores, instead.
template <int FM, int FN, int E, bool DRAIN, typename V, typename Fetch, typename Put>
__device__ __forceinline__ void store_block(const V (&acc)[FM][FN], float* part, Fetch&& fetch, Put&& put) {
  constexpr int kLd = FN * 32 + 4, kRuns = FN * 32 / E, kU = 32 * kRuns / 64, kRows = 64 / kRuns;
  const int lane = threadIdx.x & 63, lr = lane & 31, lk = lane >> 5;
  const int r0 = lane / kRuns, c = lane % kRuns * E;
  decltype(fetch(0)) got[2][kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) got[0][u] = fetch(u * kRows + r0);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i + 1 < FM) {
#pragma unroll
      for (int u = 0; u < kU; ++u) got[(i + 1) & 1][u] = fetch(32 * (i + 1) + u * kRows + r0);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const auto x = acc[i][j][4 * g + q];  // a value: the cast of a vector's element in place takes element 0
          v[q] = __builtin_bit_cast(float, x);
        }
        *reinterpret_cast<f32x4*>(part + lr * kLd + 32 * j + 8 * g + 4 * lk) = v;
      }
    if constexpr (DRAIN) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float v[E];
#pragma unroll
      for (int h = 0; h < E / 4; ++h) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(part + (u * kRows + r0) * kLd + c + 4 * h);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[4 * h + q] = x[q];
      }
      put(32 * i + u * kRows + r0, v, got[i & 1][u]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace muon

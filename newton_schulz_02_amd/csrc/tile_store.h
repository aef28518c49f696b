// From accumulators to rows of the result, for the products of the 8-bit linear operators.
//
// A wave's block of FM x FN matrix-instruction results (32 x 32 each): operand order is chosen so
// that lane l holds, of result row 32 i + l % 32, the columns 32 j + 8 g + 4 (l / 32) + 0..3 in
// acc[i][j][4 g .. 4 g + 3].  32 rows at a time go through LDS (each wave its own part, so no
// barrier), and come back as runs of 8 columns: f(row, column, the 8 values).
#pragma once

#include <hip/hip_runtime.h>

namespace muon {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Floats of a wave's part: 32 rows of FN * 32 columns and 4 floats (so that rows start in
// different banks).
template <int FN>
constexpr int store_floats() {
  return 32 * (FN * 32 + 4);
}

template <int FM, int FN, typename V, typename F>
__device__ __forceinline__ void store_block(const V (&acc)[FM][FN], float* part, F&& f) {
  constexpr int kLd = FN * 32 + 4, kRuns = FN * 4;
  const int lane = threadIdx.x & 63, lr = lane & 31, lk = lane >> 5;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
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
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < 32 * kRuns / 64; ++u) {
      const int r = (u * 64 + lane) / kRuns, c = (u * 64 + lane) % kRuns * 8;
      const f32x4* p = reinterpret_cast<const f32x4*>(part + r * kLd + c);
      const f32x4 lo = p[0], hi = p[1];
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      f(32 * i + r, c, v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace muon

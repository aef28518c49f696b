// Products of 8-bit codes for gfx950 (muon_linear.h): out = (A B^T) with a scale for each row of A
// and of B, both stored with the columns that are summed over contiguous and padded with zeros
// to 128.
//
// Main loop: as in the bf16 products of kernels_gemm.hip (a k-step holds 128 bytes of each operand
// row; rows go straight from global memory to LDS, two stages, 16-byte chunks swizzled by row),
// with v_mfma_i32_32x32x32_i8: a fragment is the same 16 bytes a lane, and the sums are exact.
#include <hip/hip_runtime.h>

#include "linear_math.h"
#include "linear_types.h"
#include "tile_order.h"
#include "tile_store.h"

using namespace muon;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kRowBytes = 128;

// Chunk position of 16-byte chunk c in LDS row r is c ^ swz(r): the 16 lanes that the LDS serves at
// once have 16 consecutive rows at the same chunk, two of which share the 64 banks.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

template <int n>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}

// Barrier of the main loop: each wave has waited for its loads, and its reads of the stage before
// were complete when their matrix instructions ran, so no fence is needed.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// WM x WN waves, each with FM x FN results of 32 x 32.
template <int WM, int WN, int FM, int FN>
__device__ __forceinline__ void int8_tile(const IntArgs& a) {
  constexpr int kWaves = WM * WN, kTM = WM * FM * 32, kTN = WN * FN * 32;
  constexpr int kStage = (kTM + kTN) * kRowBytes;
  constexpr int kInstA = kTM / 8 / kWaves, kInstB = kTN / 8 / kWaves;  // 8 rows an instruction
  constexpr int kPart = store_floats<FN>() * 4;
  static_assert(kInstA * 8 * kWaves == kTM && kInstB * 8 * kWaves == kTN, "whole instructions per wave");
  static_assert(kStage * 2 >= kWaves * kPart, "the stages hold the waves' parts of the store pass");
  static_assert(kStage % kPart == 0 || kWaves * kPart <= kStage || kWaves / 2 * kPart <= kStage, "parts lie in one stage");
  __shared__ __attribute__((aligned(1024))) char lds0[kStage];
  __shared__ __attribute__((aligned(1024))) char lds1[kStage];

  const int tm = (a.rows + kTM - 1) / kTM, tn = (a.cols + kTN - 1) / kTN;
  int ti, tj;
  full_band_decode(xcd_remap(int(blockIdx.x), int(gridDim.x)), tm, tn, ti, tj);
  const int row0 = ti * kTM, col0 = tj * kTN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / WN, wn = wave % WN, lr = lane & 31, lk = lane >> 5;

  i32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = 0;

  // Lane l of an instruction fills chunk position l % 8 of row l / 8 of its 8 rows.  Offsets are
  // relative to the tile's first row, so they fit 32 bits whatever the operand's size; rows
  // behind the operand's end are clamped to its last one and feed results that are not stored.
  const int rows_a = min(kTM, a.rows - row0), rows_b = min(kTN, a.cols - col0);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.a + int64_t(row0) * a.pitch), (short)0, rows_a * a.pitch, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + int64_t(col0) * a.pitch), (short)0, rows_b * a.pitch, 0x00020000);
  uint32_t off_a[kInstA], off_b[kInstB];
#pragma unroll
  for (int j = 0; j < kInstA; ++j) {
    const int r = (wave * kInstA + j) * 8 + (lane >> 3);
    off_a[j] = uint32_t(min(r, rows_a - 1) * a.pitch + (((lane & 7) ^ swz(r)) << 4));
  }
#pragma unroll
  for (int j = 0; j < kInstB; ++j) {
    const int r = (wave * kInstB + j) * 8 + (lane >> 3);
    off_b[j] = uint32_t(min(r, rows_b - 1) * a.pitch + (((lane & 7) ^ swz(r)) << 4));
  }
  auto issue = [&](int ks, char* st) {
#pragma unroll
    for (int j = 0; j < kInstA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (wave * kInstA + j) * 1024), 16, off_a[j],
                                               ks * kRowBytes, 0, 0);
#pragma unroll
    for (int j = 0; j < kInstB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(st + kTM * kRowBytes + (wave * kInstB + j) * 1024), 16,
                                               off_b[j], ks * kRowBytes, 0, 0);
  };
  const int steps = a.pitch / kRowBytes;
  auto step = [&](int ks, const char* st, char* next) {
    wait_vm<0>();
    stage_barrier();  // all waves' loads of this stage have landed, and the other one is free
    if (ks + 1 < steps) issue(ks + 1, next);
    __builtin_amdgcn_iglp_opt(1);
#pragma unroll
    for (int kk = 0; kk < kRowBytes / 32; ++kk) {
      const int c = 2 * kk + lk;
      i32x4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = (wm * FM + i) * 32 + lr;
        fa[i] = *reinterpret_cast<const i32x4*>(st + r * kRowBytes + ((c ^ swz(r)) << 4));
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int r = (wn * FN + j) * 32 + lr;
        fb[j] = *reinterpret_cast<const i32x4*>(st + kTM * kRowBytes + r * kRowBytes + ((c ^ swz(r)) << 4));
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  };
  if (steps > 0) issue(0, lds0);
  int ks = 0;
  for (; ks + 2 <= steps; ks += 2) {
    step(ks, lds0, lds1);
    step(ks + 1, lds1, lds0);
  }
  if (ks < steps) step(ks, lds0, lds1);
  __syncthreads();  // the store pass uses the LDS

  constexpr bool kOne = kWaves * kPart <= kStage;
  char* base = kOne || wave < kWaves / 2 ? lds0 : lds1;
  float* part = reinterpret_cast<float*>(base + (kOne ? wave : wave % (kWaves / 2)) * kPart);
  store_block(acc, part, [&](int r, int c, const float (&v)[8]) {
    const int row = row0 + wm * FM * 32 + r, col = col0 + wn * FN * 32 + c;
    if (row >= a.rows || col >= a.cols) return;
    const float sa = a.a_scale[row];
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f[e] = float(__float_as_int(v[e])) * sa * a.b_scale[min(col + e, a.cols - 1)];
    if (a.out_bf16) Eight<uint16_t>::store(static_cast<uint16_t*>(a.out) + int64_t(row) * a.ldo, col, a.cols, f);
    else Eight<float>::store(static_cast<float*>(a.out) + int64_t(row) * a.ldo, col, a.cols, f);
  });
}

template <int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(WM * WN * 64, 1) void k_int8(IntArgs a) {
  int8_tile<WM, WN, FM, FN>(a);
}

// At most 16 rows: out's columns are B's rows, read once, so the product is bound by them.  A
// workgroup of 8 waves takes 16 columns; wave w takes the k-steps w, w + 8, ... of 128 bytes, a
// lane 32 bytes of one row.  Partial sums are integers and meet in LDS.  With FUSED the rows come
// as values and every workgroup makes their codes itself, in LDS.
constexpr int kFewRows = 16, kFewWaves = 8;
template <bool FUSED, typename T>
__global__ __launch_bounds__(kFewWaves * 64) void k_int8_few(IntArgs a) {
  extern __shared__ __attribute__((aligned(16))) char codes[];  // FUSED: rows x pitch
  __shared__ int sums[kFewWaves][16][kFewRows + 1];
  __shared__ uint32_t tops[2][kFewWaves];
  __shared__ float scales[kFewRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col0 = int(blockIdx.x) * 16;
  const int l16 = lane & 15, part = lane >> 4;
  const int8_t* b = a.b + int64_t(min(col0 + l16, a.cols - 1)) * a.pitch + part * 32;
  const int steps = a.pitch / 128;
  i32x4 acc = 0;

  if constexpr (FUSED) {
    // The waves in groups of `team`, each with one row at a time.
    const int team = a.rows == 1 ? 8 : a.rows == 2 ? 4 : a.rows <= 4 ? 2 : 1;
    const int at_once = kFewWaves / team;
    for (int r0 = 0, turn = 0; r0 < a.rows; r0 += at_once, ++turn) {
      const int row = r0 + wave / team;
      const T* x = static_cast<const T*>(a.x) + int64_t(min(row, a.rows - 1)) * a.ldx;
      const int first = (wave % team) * 64 + lane, stride = team * 64;
      uint32_t top = 0;
      for (int c = first; c * 8 < a.pitch; c += stride) {
        Eight<T> v;
        v.load(x, c * 8, a.k);
        top = max(top, v.top());
      }
#pragma unroll
      for (int d = 1; d < 64; d *= 2) top = max(top, uint32_t(__shfl_xor(int(top), d)));
      if (lane == 0) tops[turn & 1][wave] = top;
      __syncthreads();
      for (int w = 0; w < team; ++w) top = max(top, tops[turn & 1][wave / team * team + w]);
      if (row < a.rows) {
        const RowCoder code(top);
        if (first == 0) scales[row] = code.scale();
        for (int c = first; c * 8 < a.pitch; c += stride) {
          Eight<T> v;
          v.load(x, c * 8, a.k);
          store_codes(reinterpret_cast<int8_t*>(codes) + row * a.pitch + c * 8, code.eight(v));
        }
      }
    }
    __syncthreads();
  }
  const char* mine = FUSED ? codes : reinterpret_cast<const char*>(a.a);
  mine += min(l16, a.rows - 1) * a.pitch + part * 32;
  for (int ks = wave; ks < steps; ks += kFewWaves) {
    const i32x4* p = reinterpret_cast<const i32x4*>(b + ks * 128);
    const i32x4* q = reinterpret_cast<const i32x4*>(mine + ks * 128);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(p[0], q[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(p[1], q[1], acc, 0, 0, 0);
  }
  // acc[r] is the sum of out's column 4 part + r (of 16) and row l16.
#pragma unroll
  for (int r = 0; r < 4; ++r) sums[wave][4 * part + r][l16] = acc[r];
  __syncthreads();
  if (threadIdx.x < 16 * kFewRows) {
    const int c = threadIdx.x & 15, row = threadIdx.x >> 4;
    if (row < a.rows && col0 + c < a.cols) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) sum += sums[w][c][row];
      const float f = float(sum) * (FUSED ? scales[row] : a.a_scale[row]) * a.b_scale[col0 + c];
      if (a.out_bf16) static_cast<uint16_t*>(a.out)[int64_t(row) * a.ldo + col0 + c] = uint16_t(pack_bf16(f, 0.0f));
      else static_cast<float*>(a.out)[int64_t(row) * a.ldo + col0 + c] = f;
    }
  }
}

template <int WM, int WN, int FM, int FN>
int launch(const IntArgs& a, hipStream_t s) {
  const int64_t tm = (a.rows + WM * FM * 32 - 1) / (WM * FM * 32), tn = (a.cols + WN * FN * 32 - 1) / (WN * FN * 32);
  hipLaunchKernelGGL((k_int8<WM, WN, FM, FN>), dim3(uint32_t(tm * tn)), dim3(WM * WN * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int muon_launch_int8(const IntArgs& a, int tile, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return tile == 256 ? launch<2, 4, 4, 2>(a, s) : launch<2, 2, 2, 2>(a, s);
}

int muon_launch_int8_few(const IntArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(uint32_t((a.cols + 15) / 16)), block(kFewWaves * 64);
  const uint32_t lds = a.fused ? uint32_t(a.rows) * uint32_t(a.pitch) : 0;
  if (!a.fused) hipLaunchKernelGGL((k_int8_few<false, float>), grid, block, 0, s, a);
  else if (a.x_bf16) hipLaunchKernelGGL((k_int8_few<true, uint16_t>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_int8_few<true, float>), grid, block, lds, s, a);
  return hipGetLastError();
}

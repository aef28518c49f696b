// Products of 8-bit codes for gfx950 (muon_linear.h): out = (A B^T) with a scale for each row of A
// and of B, both stored with the columns that are summed over contiguous and padded with zeros
// to 128.
//
// Main loop: a k-step holds 64 bytes of each operand row.  Rows go straight from global memory to
// one of five stages in LDS, so loads have three steps to arrive, and step ks + 1 is complete
// when step ks begins: the last group of step ks reads the first fragments of the next one, and
// matrix instructions (v_mfma_i32_32x32x32_i8; the sums are exact) go on over the barrier.
//
// 16384 x 11008 x 4096 take 640 to 690 us by card and by how long it has run (2.1 to 2.3 POP/s), 8192^3 454
// (2.4): power holds the clock at 1.65 GHz, with the matrix units busy 64 % of the time.
// 2048 x 4096 x 4096 take 39 to 43 us in 256 x 128 tiles, at 2.36 GHz: the loads decide.  Of the time that the
// compute units are busy the matrix units are for 37 %, LDS reads take 21 % and the L1 caches wait for
// L2 60 %: rows of 64 bytes are requests of 64 bytes, about 118 of them in flight for 430 cycles each, so
// 18 bytes a cycle and compute unit arrive.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_math.h"
#include "linear_types.h"
#include "tile_order.h"
#include "tile_store.h"

using namespace muon;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kRowBytes = 64, kStages = 5;

// Chunk position of 16-byte chunk c in LDS row r is c ^ swz(r): the 16 lanes that the LDS serves at
// once have 16 consecutive rows at the same chunk, four of which share the 64 banks.
__device__ __forceinline__ int swz(int r) { return (r >> 2) & 3; }

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

// WM x WN waves, each with FM x FN results of 32 x 32; T is the result's type.
template <typename T, int WM, int WN, int FM, int FN>
__device__ __forceinline__ void int8_tile(const IntArgs& a) {
  constexpr int kWaves = WM * WN, kTM = WM * FM * 32, kTN = WN * FN * 32;
  constexpr int kStage = (kTM + kTN) * kRowBytes;
  constexpr int kInstA = kTM / 16 / kWaves, kInstB = kTN / 16 / kWaves;  // 16 rows an instruction
  constexpr int kLoads = kInstA + kInstB, kGroups = kRowBytes / 32;
  constexpr int kPart = store_floats<FN>() * 4;
  constexpr int kPartWaves = (kWaves + 3) / 4;
  static_assert(kInstA * 16 * kWaves == kTM && kInstB * 16 * kWaves == kTN, "whole instructions per wave");
  static_assert(kStage >= kPartWaves * kPart, "a stage holds a quarter of the waves' parts of the store pass");
  __shared__ __attribute__((aligned(1024))) char s0[kStage];
  __shared__ __attribute__((aligned(1024))) char s1[kStage];
  __shared__ __attribute__((aligned(1024))) char s2[kStage];
  __shared__ __attribute__((aligned(1024))) char s3[kStage];
  __shared__ __attribute__((aligned(1024))) char s4[kStage];

  const int tm = (a.rows + kTM - 1) / kTM, tn = (a.cols + kTN - 1) / kTN;
  int ti, tj;
  full_band_decode(xcd_remap(int(blockIdx.x), int(gridDim.x)), tm, tn, ti, tj);
  const int row0 = ti * kTM, col0 = tj * kTN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, lr = lane & 31, lk = lane >> 5;

  i32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = 0;

  // Lane l of an instruction fills chunk position l % 4 of row l / 4 of its 16 rows.  Offsets are
  // relative to the tile's first row, so they fit 32 bits whatever the operand's size; rows
  // behind the operand's end are clamped to its last one and feed results that are not stored.
  const int rows_a = min(kTM, a.rows - row0), rows_b = min(kTN, a.cols - col0);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.a + int64_t(row0) * a.pitch), (short)0, rows_a * a.pitch, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.b + int64_t(col0) * a.pitch), (short)0, rows_b * a.pitch, 0x00020000);
  uint32_t off[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = (j < kInstA ? wave * kInstA + j : wave * kInstB + j - kInstA) * 16 + (lane >> 2);
    off[j] = uint32_t(min(r, (j < kInstA ? rows_a : rows_b) - 1) * a.pitch + (((lane & 3) ^ swz(r)) << 4));
  }
  const int steps = a.pitch / kRowBytes;
  // Load j of k-step ks; steps behind the last one load that again, which nothing reads.
  auto issue = [&](int ks, int j, char* st) {
    const int at = min(ks, steps - 1) * kRowBytes;
    if (j < kInstA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (wave * kInstA + j) * 1024), 16, off[j], at, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(st + kTM * kRowBytes + (wave * kInstB + j - kInstA) * 1024),
                                               16, off[j], at, 0, 0);
  };
  i32x4 fa[2][FM], fb[2][FN];
  auto read = [&](const char* st, int kk, int to) {
    const int c = 2 * kk + lk;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int r = (wn * FN + j) * 32 + lr;
      fb[to][j] = *reinterpret_cast<const i32x4*>(st + kTM * kRowBytes + r * kRowBytes + ((c ^ swz(r)) << 4));
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = (wm * FM + i) * 32 + lr;
      fa[to][i] = *reinterpret_cast<const i32x4*>(st + r * kRowBytes + ((c ^ swz(r)) << 4));
    }
  };
  // In flight when step ks begins: the loads of steps ks + 1 to ks + 3; those of ks + 1 are waited
  // for.  Those of ks + 4 go where step ks - 1 was.
  auto step = [&](int ks, const char* st, const char* next, char* free) {
    wait_vm<2 * kLoads>();
    stage_barrier();
    static_for<kGroups>([&](auto kc) {
      constexpr int kk = decltype(kc)::value, cur = kk & 1;
#pragma unroll
      for (int j = kk * kLoads / kGroups; j < (kk + 1) * kLoads / kGroups; ++j) issue(ks + 4, j, free);
      if constexpr (kk + 1 < kGroups) read(st, kk + 1, cur ^ 1);
      else read(next, 0, cur ^ 1);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
      // Between two matrix instructions: one load and one read.
      static_for<FM * FN>([&](auto) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, (FM + FN + FM * FN - 1) / (FM * FN), 0);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  static_assert(kGroups % 2 == 0, "a step begins with the same half of the fragment registers");
  if (steps > 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) issue(q, j, q == 0 ? s0 : q == 1 ? s1 : q == 2 ? s2 : s3);
    wait_vm<3 * kLoads>();
    stage_barrier();
    read(s0, 0, 0);
    auto step_at = [&](int ks, auto at) {
      constexpr int i = decltype(at)::value;
      char* const st[kStages] = {s0, s1, s2, s3, s4};
      step(ks, st[i], st[(i + 1) % kStages], st[(i + 4) % kStages]);
    };
    // Five steps until the stages come round, and the rest behind the loop: with exits inside it the
    // compiler joined their states with the next round's, and waited for all loads there.
    int ks = 0;
    for (; ks + kStages <= steps; ks += kStages) static_for<kStages>([&](auto at) { step_at(ks + decltype(at)::value, at); });
    if (ks < steps) {
      step_at(ks, std::integral_constant<int, 0>{});
      if (ks + 1 < steps) {
        step_at(ks + 1, std::integral_constant<int, 1>{});
        if (ks + 2 < steps) {
          step_at(ks + 2, std::integral_constant<int, 2>{});
          if (ks + 3 < steps) step_at(ks + 3, std::integral_constant<int, 3>{});
        }
      }
    }
    wait_vm<0>();  // what the last steps loaded
  }
  __syncthreads();  // the store pass uses the LDS

  const int array = wave / kPartWaves;
  char* base = array == 0 ? s0 : array == 1 ? s1 : array == 2 ? s2 : s3;
  float* part = reinterpret_cast<float*>(base + wave % kPartWaves * kPart);
  const int wrow = row0 + wm * FM * 32, wcol = col0 + wn * FN * 32;
  constexpr int E = Run<T>::E;
  const int col = wcol + store_col<FN, E>();
  float sb[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sb[e] = *(global_ptr<const float>)(a.b_scale + min(col + e, a.cols - 1));
  auto store = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    store_block<FM, FN, E, !kWhole>(
        acc, part,
        [&](int r) { return *(global_ptr<const float>)(a.a_scale + (kWhole ? wrow + r : min(wrow + r, a.rows - 1))); },
        [&](int r, const float (&v)[E], float sa) {
          if (!kWhole && (wrow + r >= a.rows || col >= a.cols)) return;
          float f[E];
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = float(__float_as_int(v[e])) * sa * sb[e];
          Run<T> x;
          x.set(f);
          x.template store<kWhole>(static_cast<T*>(a.out) + int64_t(wrow + r) * a.ldo, col, a.cols);
        });
  };
  if (wrow + FM * 32 <= a.rows && wcol + FN * 32 <= a.cols) store(std::true_type{});
  else store(std::false_type{});
}

template <typename T, int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(WM * WN * 64, 1) void k_int8(IntArgs a) {
  int8_tile<T, WM, WN, FM, FN>(a);
}

// Few rows: out's columns are B's rows, read once, so the product is bound by them.  A workgroup of
// 8 waves takes 16 C columns and up to 16 G rows; wave w takes the k-steps w, w + 8, ... of 128
// bytes, a lane 16 bytes of each half of one row of each operand, kAhead steps before they are
// multiplied.
// Partial sums are integers and meet in LDS.  One row of 4096 for 11008 columns takes 12 us (3.8 TB/s):
// the weights, and about 3 us until the first arrive and the sums have met.
// With FUSED the rows come as values and every workgroup makes their codes itself, in LDS, while its
// first loads of B are on their way.
constexpr int kFewWaves = 8;
template <bool FUSED, typename T, int G, int C>
__global__ __launch_bounds__(kFewWaves * 64) void k_int8_few(IntArgs a) {
  constexpr int kAhead = C == 1 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) char codes[];  // FUSED: rows x pitch
  __shared__ int sums[kFewWaves][16 * C][16 * G + 1];
  __shared__ uint32_t tops[kFewWaves];
  __shared__ float scales[16 * G];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col0 = int(blockIdx.x) * 16 * C;
  const int l16 = lane & 15, part = lane >> 4;
  const int steps = a.pitch / 128;
  const int8_t* b[C];
#pragma unroll
  for (int c = 0; c < C; ++c) b[c] = a.b + int64_t(min(col0 + 16 * c + l16, a.cols - 1)) * a.pitch + part * 16;
  i32x4 w[kAhead][C][2];
  auto load_b = [&](int ks, int u) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const global_ptr<const i32x4> p = (global_ptr<const i32x4>)(b[c] + ks * 128);
      w[u][c][0] = __builtin_nontemporal_load(p);
      w[u][c][1] = __builtin_nontemporal_load(p + 4);
    }
  };
  auto load_first = [&] {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (wave + u * kFewWaves < steps) load_b(wave + u * kFewWaves, u);
  };
  if constexpr (FUSED) {
    // The waves in groups of `team`, each with one row at a time, whose first kHold chunks of 8 values a
    // lane are kept between the maximum and the codes.  Where a team is more than a wave (up to 4 rows)
    // there is a team for each row, so the loop runs once and `tops` is written once.  Loads arrive in
    // their order, so the first rows are asked for before B (behind it, the codes were begun when all
    // of B had come).
    constexpr int kHold = 2;
    const int team = a.rows == 1 ? kFewWaves : a.rows == 2 ? kFewWaves / 2 : a.rows <= 4 ? kFewWaves / 4 : 1;
    const int at_once = kFewWaves / team;
    const int first = (wave % team) * 64 + lane, stride = team * 64;
    Eight<T> v[kHold];
    auto row_of = [&](int row) { return static_cast<const T*>(a.x) + int64_t(min(row, a.rows - 1)) * a.ldx; };
    auto load_row = [&](const T* x) {
#pragma unroll
      for (int i = 0; i < kHold; ++i) v[i].load(x, (first + i * stride) * 8, a.k);
    };
    load_row(row_of(wave / team));
    load_first();
    for (int r0 = 0; r0 < a.rows; r0 += at_once) {
      const int row = r0 + wave / team;
      const T* x = row_of(row);
      if (r0 > 0) load_row(x);
      typename Eight<T>::Tops tops_of;
#pragma unroll
      for (int i = 0; i < kHold; ++i) tops_of.take(v[i]);
      for (int c = first + kHold * stride; c * 8 < a.pitch; c += stride) {
        Eight<T> y;
        y.load(x, c * 8, a.k);
        tops_of.take(y);
      }
      uint32_t top = max64(tops_of.all());
      if (team > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        for (int i = 0; i < team; ++i) top = max(top, tops[wave / team * team + i]);
      }
      if (row < a.rows) {
        const RowCoder code(top);
        if (first == 0) scales[row] = code.scale();
        uint2* q = reinterpret_cast<uint2*>(codes + row * a.pitch);
#pragma unroll
        for (int i = 0; i < kHold; ++i)
          if ((first + i * stride) * 8 < a.pitch) q[first + i * stride] = code.eight(v[i]);
        for (int c = first + kHold * stride; c * 8 < a.pitch; c += stride) {
          Eight<T> y;
          y.load(x, c * 8, a.k);
          q[c] = code.eight(y);
        }
      }
    }
    __syncthreads();
  } else {
    load_first();
  }
  const char* rows = FUSED ? codes : reinterpret_cast<const char*>(a.a);
  int at[G];  // few rows: 64 * 131072 bytes at most
#pragma unroll
  for (int g = 0; g < G; ++g) at[g] = min(16 * g + l16, a.rows - 1) * a.pitch + part * 16;
  i32x4 acc[G][C];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[g][c] = 0;
  for (int k0 = wave; k0 < steps; k0 += kAhead * kFewWaves) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int ks = k0 + u * kFewWaves;
      if (ks >= steps) break;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const i32x4* q = reinterpret_cast<const i32x4*>(rows + at[g] + ks * 128);
        const i32x4 q0 = q[0], q1 = q[4];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          acc[g][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][c][0], q0, acc[g][c], 0, 0, 0);
          acc[g][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][c][1], q1, acc[g][c], 0, 0, 0);
        }
      }
      if (ks + kAhead * kFewWaves < steps) load_b(ks + kAhead * kFewWaves, u);
    }
  }
  // acc[g][c][r] is the sum of out's column 16 c + 4 part + r and row 16 g + l16.
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][16 * c + 4 * part + r][16 * g + l16] = acc[g][c][r];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * C * 16 * G; i += kFewWaves * 64) {
    const int c = i % (16 * C), row = i / (16 * C);
    if (row >= a.rows || col0 + c >= a.cols) continue;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) sum += sums[v][c][row];
    const float f = float(sum) * (FUSED ? scales[row] : a.a_scale[row]) * a.b_scale[col0 + c];
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[int64_t(row) * a.ldo + col0 + c] = uint16_t(pack_bf16(f, 0.0f));
    else static_cast<float*>(a.out)[int64_t(row) * a.ldo + col0 + c] = f;
  }
}

template <bool FUSED, typename T, int G, int C>
int launch_few(const IntArgs& a, hipStream_t s) {
  const uint32_t lds = FUSED ? uint32_t(a.rows) * uint32_t(a.pitch) : 0;
  hipLaunchKernelGGL((k_int8_few<FUSED, T, G, C>), dim3(uint32_t((a.cols + 16 * C - 1) / (16 * C))), dim3(kFewWaves * 64),
                     lds, s, a);
  return hipGetLastError();
}

template <int WM, int WN, int FM, int FN>
int launch(const IntArgs& a, hipStream_t s) {
  const int64_t tm = (a.rows + WM * FM * 32 - 1) / (WM * FM * 32), tn = (a.cols + WN * FN * 32 - 1) / (WN * FN * 32);
  const dim3 grid(uint32_t(tm * tn)), block(WM * WN * 64);
  if (a.out_bf16) hipLaunchKernelGGL((k_int8<uint16_t, WM, WN, FM, FN>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_int8<float, WM, WN, FM, FN>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

int muon_launch_int8(const IntArgs& a, int tile, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (tile == kTile256) return launch<2, 4, 4, 2>(a, s);
  return tile == kTile256x128 ? launch<4, 2, 2, 2>(a, s) : launch<2, 2, 2, 2>(a, s);
}

int muon_launch_int8_few(const IntArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.fused) return a.x_bf16 ? launch_few<true, uint16_t, 1, 1>(a, s) : launch_few<true, float, 1, 1>(a, s);
  if (a.rows <= 16) return launch_few<false, float, 1, 1>(a, s);
  if (a.rows <= 32) return launch_few<false, float, 2, 2>(a, s);
  return launch_few<false, float, 4, 2>(a, s);
}

// Weight gradients from 8-bit checkpoints for gfx950 (muon_linear.h): dw = dy^T x, summed over the
// tokens, which are the rows of both operands.
//
// bf16 dy.  A k-step is 64 tokens.  dy's rows go straight from global memory to LDS; the codes
// come through registers, where one token's 16 codes are decoded by its block's scale to bf16
// (exactly) before they are written next to them.  Both lie in LDS as they lie in memory,
// tokens as rows, and ds_read_b64_tr_b16 turns them as they are read: of each group of 16 lanes,
// lane i gives the address of 4 columns of token i / 4, and gets 4 tokens of column i.
//
// 16384 tokens x 11008 x 4096 take 1210 to 1275 us by card (1.2 PFLOP/s): bound by power, at 1.7 GHz with the matrix
// units busy 66 % of the time that the 688 tiles of 256 x 256 take.  In a tile of 128 x 128 a step takes
// 0.63 us, of which LDS accesses are the most.
//
// fp32 dy.  v_mfma_f32_32x32x2_f32 takes one value a lane and operand, which is how the rows lie
// in LDS already.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_math.h"
#include "linear_types.h"
#include "tile_order.h"
#include "tile_store.h"

using namespace muon;

namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

constexpr int kStep = 64;  // tokens of a k-step

template <int n>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}

__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14)); }

// Barrier of the main loop: each wave has waited for what it wrote or loaded itself, and its reads
// of the stage before were complete when their matrix instructions ran.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A wave's block of results, from row wrow and column wcol on, less the rows before row_lo: to the
// output (T), added to what is there with ADD, or to a piece's partial results.
template <typename T, bool ADD, int FM, int FN>
__device__ __forceinline__ void put_block(const WgradArgs& a, const f32x16 (&acc)[FM][FN], float* part, int wrow, int wcol,
                                          int row_lo) {
  constexpr int E = Run<T>::E;
  const bool pieces = a.splits > 1;  // T is float then
  T* out = pieces ? reinterpret_cast<T*>(a.parts) + int64_t(blockIdx.y) * a.n * a.k : static_cast<T*>(a.out);
  const int64_t ld = pieces ? a.k : a.ldo;
  const int col = wcol + store_col<FN, E>();
  auto store = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    store_block<FM, FN, E, !kWhole>(
        acc, part,
        [&](int r) {
          Run<T> old;
          old.v = 0;
          if (ADD && kWhole) old.load(out + int64_t(wrow + r) * ld + col);
          else if (ADD) old.load_edge(out + int64_t(min(wrow + r, a.n - 1)) * ld, min(col, a.k - 1), a.k);
          return old;
        },
        [&](int r, const float (&v)[E], Run<T> old) {
          if (!kWhole && (wrow + r < row_lo || wrow + r >= a.n || col >= a.k)) return;
          if (ADD && !kWhole) old.settle(col, a.k);
          float f[E];
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = ADD ? old.get(e) + v[e] : v[e];
          Run<T> x;
          x.set(f);
          x.template store<kWhole>(out + int64_t(wrow + r) * ld, col, a.k);
        });
  };
  if (wrow >= row_lo && wrow + FM * 32 <= a.n && wcol + FN * 32 <= a.k) store(std::true_type{});
  else store(std::false_type{});
}

// Place of 16-byte chunk c of token t's row in LDS.  A transposing read takes 64 bytes (4 chunks) of
// each of 4 consecutive tokens at a time: bits 2 and 3 put these on different banks.  Bit 0 puts
// the two chunks that a lane decodes on other banks for odd tokens than for even ones.
__device__ __forceinline__ int place(int c, int t) { return c ^ (((t & 3) << 2) | (t & 1)); }

// WM x WN waves of FM x FN results: a tile of WM FM 32 rows (columns of dy) by WN FN 32 (inputs).
//
// dy has three stages in LDS, x two.  While step ks is multiplied, dy of step ks + 2 is on its way to
// LDS and the codes of step ks + 2 to registers; those of step ks + 1, in registers, are decoded
// into x's other stage between the matrix instructions.  Each stage is an array of its own, so
// that the compiler does not take the writes of one for the loads of another.
//
// THROUGH: dy's rows are not 16-byte aligned, which loads to LDS have to be, and come through
// registers, written to LDS a step after they were asked for.  The last tile begins early enough to
// be whole (n is at least a tile then), and leaves the rows that it shares to the tile before.
template <typename T, bool ADD, bool THROUGH, int WM, int WN, int FM, int FN>
__device__ __forceinline__ void wgrad_tile(const WgradArgs& a) {
  constexpr int kWaves = WM * WN, kThreads = kWaves * 64, kTM = WM * FM * 32, kTN = WN * FN * 32;
  constexpr int kRowA = kTM * 2, kRowB = kTN * 2;  // bytes of a token's row in LDS
  constexpr int kA = kStep * kRowA, kB = kStep * kRowB;
  constexpr int kInstA = kA / 1024 / kWaves;                // instructions of 1 KB a wave and step
  constexpr int kUnits = kStep * kTN / 16 / kThreads;       // 16 codes a lane and unit
  constexpr int kPart = store_floats<FN>() * 4;
  static_assert(kInstA * 1024 * kWaves == kA && kUnits * kThreads * 16 == kStep * kTN, "whole loads per lane");
  constexpr int kGroups = kStep / 16;                       // fragment groups of 16 tokens
  constexpr int kPieces = kUnits * 2 / kGroups;             // half units that a lane decodes with each
  static_assert(kPieces * kGroups == kUnits * 2, "whole pieces with each fragment group");
  // The store pass: an array each for up to a quarter of the waves.
  constexpr int kPartWaves = (kWaves + 3) / 4;
  constexpr int kArrA = kA > kPartWaves * kPart ? kA : kPartWaves * kPart;
  constexpr int kArrB = kB > kPartWaves * kPart ? kB : kPartWaves * kPart;
  __shared__ __attribute__((aligned(1024))) char a0[kArrA];
  __shared__ __attribute__((aligned(1024))) char a1[kArrA];
  __shared__ __attribute__((aligned(1024))) char a2[kArrA];
  __shared__ __attribute__((aligned(1024))) char b0[kArrB];
  __shared__ __attribute__((aligned(1024))) char b1[kArrB];

  const int tm = (a.n + kTM - 1) / kTM, tn = (a.k + kTN - 1) / kTN;
  int ti, tj;
  full_band_decode(xcd_remap(int(blockIdx.x), int(gridDim.x)), tm, tn, ti, tj);
  const int row_lo = ti * kTM, row0 = THROUGH ? min(row_lo, a.n - kTM) : row_lo, col0 = tj * kTN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int t0 = int(blockIdx.y) * a.piece, tokens = min(a.piece, a.tokens - t0);
  const int steps = (tokens + kStep - 1) / kStep;

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = 0.0f;

  // dy: lane l of a wave's instruction fills chunk position l % (chunks a row) of one of its rows.
  // Columns behind dy's end are clamped to its last chunk (n_read is a multiple of 8), tokens to
  // the last token; the rows of tokens that are not there are cleared below.  Offsets are relative
  // to the step's first token, so they fit 32 bits.
  constexpr int kChunksA = kRowA / 16, kRowsInst = 64 / kChunksA;
  const char* dy = static_cast<const char*>(a.dy) + int64_t(t0) * a.lddy * 2;
  const int ld2 = int(a.lddy * 2);
  int src[kInstA], tok[kInstA];
#pragma unroll
  for (int j = 0; j < kInstA; ++j) {
    tok[j] = (wave * kInstA + j) * kRowsInst + lane / kChunksA;
    src[j] = min(row0 + place(lane % kChunksA, tok[j]) * 8, a.n_read - 8) * 2;
  }
  u32x4 through[THROUGH ? kInstA : 1] = {};
  auto load_dy = [&](int ks, int j, char* st) {
    const int first = min(ks * kStep, tokens - 1), left = tokens - 1 - first;
    if constexpr (THROUGH) {
      through[j] = *(global_ptr<const u32x4_at2>)(dy + int64_t(first) * ld2 + uint32_t(min(tok[j], left) * ld2 + src[j]));
      return;
    }
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(dy + int64_t(first) * ld2), (short)0, min(left, kStep - 1) * ld2 + a.n_read * 2, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(st + (wave * kInstA + j) * 1024), 16,
                                             min(tok[j], left) * ld2 + src[j], 0, 0, 0);
  };
  // Codes: a lane has 16 codes of one token, which share a scale.
  constexpr int kChunksB = kTN / 16;  // 16-code units of a token's row
  u32x4 xq[2][kUnits];
  float xs[2][kUnits];
  const int8_t* q0 = a.q + int64_t(t0) * a.pitch;
  const float* s0 = a.scale + int64_t(t0) * a.groups;
  const int col = min(col0 + tid % kChunksB * 16, a.pitch - 16);  // kThreads is a multiple of kChunksB
  const int group = min(col / kCodeBlock, a.groups - 1);
  auto load_x = [&](int ks, auto set, int u) {
    constexpr int r = decltype(set)::value;
    const int first = min(ks * kStep, tokens - 1);
    const int8_t* q = q0 + int64_t(first) * a.pitch;
    const float* s = s0 + int64_t(first) * a.groups;
    const uint32_t t = uint32_t(min((u * kThreads + tid) / kChunksB, tokens - 1 - first));
    xq[r][u] = *(global_ptr<const u32x4>)(q + (t * uint32_t(a.pitch) + uint32_t(col)));
    xs[r][u] = *(global_ptr<const float>)(s + (t * uint32_t(a.groups) + uint32_t(group)));
  };
  // The share of a step's loads that goes with fragment group kk.  A wave's loads of 1 KB each keep
  // the address unit busy for 16 cycles: together at the step's start, they held all waves up.
  auto load_share = [&](int ks, int kk, char* st, auto set, char* before) {
#pragma unroll
    for (int j = 0; j < kInstA; ++j)
      if (j * kGroups / kInstA == kk) {
        // What step ks - 1 will read.
        if constexpr (THROUGH) *reinterpret_cast<u32x4*>(before + (wave * kInstA + j) * 1024 + lane * 16) = through[j];
        load_dy(ks, j, st);
      }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (u * kGroups / kUnits == kk) load_x(ks, set, u);
  };
  // Half h of unit u, of step ks: decoded, to LDS; zero for tokens behind the last one.
  auto put_x = [&](int ks, auto set, int u, int h, char* st) {
    constexpr int r = decltype(set)::value;
    const int t = (u * kThreads + tid) / kChunksB, c = tid % kChunksB * 2 + h;
    const float s = ks * kStep + t < tokens ? xs[r][u] : 0.0f;
    float f[8];
    decode8(make_uint2(xq[r][u][2 * h], xq[r][u][2 * h + 1]), s, f);
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
    *reinterpret_cast<u32x4*>(st + t * kRowB + place(c, t) * 16) = o;
  };

  // Fragments.  Of a 32 x 16 fragment (columns x tokens), lane l has column l % 32 and the tokens
  // 8 (l / 32) .. + 7, as two transposing reads of 4.
  const int g = lane >> 4, i16 = lane & 15;
  auto frag_at = [&](int col) {  // byte of the first read's address within a stage's operand, less the row's
    const int n = col + 16 * (g & 1) + (i16 & 3) * 4;
    return place(n / 8, i16 >> 2) * 16 + (n & 4) * 2;
  };
  const int t_lane = 8 * (g >> 1) + (i16 >> 2);
  int at_a[FM], at_b[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) at_a[i] = t_lane * kRowA + frag_at((wm * FM + i) * 32);
#pragma unroll
  for (int j = 0; j < FN; ++j) at_b[j] = t_lane * kRowB + frag_at((wn * FN + j) * 32);
  auto frag = [&](char* st, int at, int row_bytes, int kk) {
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(st + at + kk * 16 * row_bytes));
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(st + at + (kk * 16 + 4) * row_bytes));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  auto load_frags = [&](char* sa, char* sb, int kk, bf16x8 (&fa)[FM], bf16x8 (&fb)[FN]) {
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = frag(sb, at_b[j], kRowB, kk);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = frag(sa, at_a[i], kRowA, kk);
  };

  // Loads are counted in their order: when step ks begins, behind dy of step ks there are codes of
  // step ks (used already), and dy and the codes of step ks + 1 in flight: kInstA loads and 2 a
  // unit (the barrier's empty asm statements keep a step's loads in it).  The last steps, too, load
  // and decode what would come next (the last token, and nothing reads it): without branches the
  // compiler mixes a step's parts, and keeps the results where they are.  next_a, next_b: where dy
  // of step ks + 2 and x of step ks + 1 go; mid_a: dy of step ks + 1.
  auto step = [&](int ks, char* sa, char* sb, char* mid_a, char* next_a, char* next_b, auto set, auto other) {
    if constexpr (!THROUGH) wait_vm<kInstA + 2 * kUnits>();
    wait_lds();
    stage_barrier();  // all waves' dy and codes of this step are there, and what step ks - 1 read is free
    if (tokens - ks * kStep < kStep) {
      // Tokens behind the last one: x is zero there; so that infinities in dy's last row are not
      // multiplied with it, dy is cleared too.
      for (int b = tokens % kStep * kRowA + tid * 16; b < kA; b += kThreads * 16) *reinterpret_cast<u32x4*>(sa + b) = 0;
      __syncthreads();
    }
    // The fragments of a group of 16 tokens are read while the group before is multiplied.
    bf16x8 fa[2][FM], fb[2][FN];
    load_frags(sa, sb, 0, fa[0], fb[0]);
    __builtin_amdgcn_sched_barrier(0);
    static_for<kGroups>([&](auto kc) {
      constexpr int kk = decltype(kc)::value, cur = kk & 1;
      constexpr bool kNext = kk + 1 < kGroups;
      load_share(ks + 2, kk, next_a, set, mid_a);
      if constexpr (kNext) load_frags(sa, sb, kk + 1, fa[cur ^ 1], fb[cur ^ 1]);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int p = kk * kPieces; p < (kk + 1) * kPieces; ++p) put_x(ks + 1, other, p >> 1, p & 1, next_b);
      // Between two matrix instructions: a few of the loads, the reads and the decoding's instructions.
      static_for<FM * FN>([&](auto) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        if constexpr (kNext) __builtin_amdgcn_sched_group_barrier(0x100, (2 * (FM + FN) + FM * FN - 1) / (FM * FN), 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      });
      __builtin_amdgcn_sched_group_barrier(0x200, kPieces + (THROUGH ? kInstA / kGroups : 0), 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  if (steps > 0) {
    constexpr std::integral_constant<int, 0> x0{};
    constexpr std::integral_constant<int, 1> x1{};
#pragma unroll
    for (int kk = 0; kk < kGroups; ++kk) load_share(0, kk, a0, x0, a2);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int p = 0; p < 2 * kUnits; ++p) put_x(0, x0, p >> 1, p & 1, b0);
#pragma unroll
    for (int kk = 0; kk < kGroups; ++kk) load_share(1, kk, a1, x1, a0);
    auto step_at = [&](int ks, auto at) {
      constexpr int i = decltype(at)::value;
      char* const st[3] = {a0, a1, a2};
      char* const sx[2] = {b0, b1};
      const std::integral_constant<int, i % 2> set{};
      const std::integral_constant<int, 1 - i % 2> other{};
      step(ks, st[i % 3], sx[i % 2], st[(i + 1) % 3], st[(i + 2) % 3], sx[1 - i % 2], set, other);
    };
    // Six steps until stages and registers come round, and the rest behind the loop: with exits inside
    // it the compiler joined their states with the next round's, and waited for all loads there.
    int ks = 0;
    for (; ks + 6 <= steps; ks += 6) static_for<6>([&](auto at) { step_at(ks + decltype(at)::value, at); });
    if (ks < steps) {
      step_at(ks, std::integral_constant<int, 0>{});
      if (ks + 1 < steps) {
        step_at(ks + 1, std::integral_constant<int, 1>{});
        if (ks + 2 < steps) {
          step_at(ks + 2, std::integral_constant<int, 2>{});
          if (ks + 3 < steps) {
            step_at(ks + 3, std::integral_constant<int, 3>{});
            if (ks + 4 < steps) step_at(ks + 4, std::integral_constant<int, 4>{});
          }
        }
      }
    }
    wait_vm<0>();  // what the last step loaded
  }
  __syncthreads();  // the store pass uses the LDS

  const int array = wave / kPartWaves;
  char* base = array == 0 ? a0 : array == 1 ? a1 : array == 2 ? b0 : b1;
  put_block<T, ADD>(a, acc, reinterpret_cast<float*>(base + wave % kPartWaves * kPart), row0 + wm * FM * 32,
                    col0 + wn * FN * 32, row_lo);
}

template <typename T, bool ADD, bool THROUGH, int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(WM * WN * 64, 1) void k_wgrad(WgradArgs a) {
  wgrad_tile<T, ADD, THROUGH, WM, WN, FM, FN>(a);
}

// fp32 dy: 128 x 128 tiles of 4 waves, 32 tokens a step, through registers; two workgroups share a
// compute unit, so that one multiplies while the other writes to LDS.  4096^3 takes 1175 us (117 TFLOP/s).
template <typename T, bool ADD>
__global__ __launch_bounds__(256, 2) void k_wgrad_f32(WgradArgs a) {
  constexpr int kT = 128, kTok = 32, kLd = kT + 4, kUnits = kTok / 16;
  __shared__ __attribute__((aligned(16))) float lds[2][2][kTok * kLd];
  static_assert(sizeof(lds) >= 4 * store_floats<2>() * 4, "the stages hold the waves' parts of the store pass");
  const int tm = (a.n + kT - 1) / kT, tn = (a.k + kT - 1) / kT;
  int ti, tj;
  full_band_decode(xcd_remap(int(blockIdx.x), int(gridDim.x)), tm, tn, ti, tj);
  const int row0 = ti * kT, col0 = tj * kT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 31, lk = lane >> 5;
  const int t0 = int(blockIdx.y) * a.piece, tokens = min(a.piece, a.tokens - t0);
  const int steps = (tokens + kTok - 1) / kTok;
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = 0.0f;

  // A lane has 8 columns of tokens tid / 16 and tid / 16 + 16.
  const int t = tid >> 4, c = (tid & 15) * 8;
  const int col = min(col0 + c, a.pitch - 8), group = min(col / kCodeBlock, a.groups - 1);
  Eight<float> dy[kUnits];
  u32x2 codes[kUnits];
  float scale[kUnits];
  auto load = [&](int ks) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = ks * kTok + t + 16 * u;
      const int64_t row = t0 + min(at, tokens - 1);
      dy[u].clear();
      if (at < tokens) dy[u].load(static_cast<const float*>(a.dy) + row * a.lddy, row0 + c, a.n);
      codes[u] = *(global_ptr<const u32x2>)(a.q + row * a.pitch + col);
      scale[u] = *(global_ptr<const float>)(a.scale + row * a.groups + group);
    }
  };
  auto put = [&](int ks) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float f[8];
      decode8(make_uint2(codes[u][0], codes[u][1]), ks * kTok + t + 16 * u < tokens ? scale[u] : 0.0f, f);
      f32x4* pa = reinterpret_cast<f32x4*>(&lds[ks & 1][0][(t + 16 * u) * kLd + c]);
      f32x4* pb = reinterpret_cast<f32x4*>(&lds[ks & 1][1][(t + 16 * u) * kLd + c]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pa[h] = f32x4{dy[u].get(4 * h), dy[u].get(4 * h + 1), dy[u].get(4 * h + 2), dy[u].get(4 * h + 3)};
        pb[h] = f32x4{f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
      }
    }
  };
  if (steps > 0) load(0);
  for (int ks = 0; ks < steps; ++ks) {
    put(ks);
    __syncthreads();
    if (ks + 1 < steps) load(ks + 1);
    const float* pa = lds[ks & 1][0] + lk * kLd + wm * 64 + lr;
    const float* pb = lds[ks & 1][1] + lk * kLd + wn * 64 + lr;
#pragma unroll
    for (int kk = 0; kk < kTok / 2; ++kk) {
      float fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = pa[kk * 2 * kLd + 32 * i], fb[i] = pb[kk * 2 * kLd + 32 * i];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();  // the store pass uses the LDS
  float* parts = &lds[0][0][0];
  put_block<T, ADD>(a, acc, parts + wave * store_floats<2>(), row0 + wm * 64, col0 + wn * 64, row0);
}

// Partial results of the pieces, in their order, to the output; a lane has 8 values.  Only results of
// few tiles are cut, so a launch has a few thousand workgroups at most.  3 pieces of 517 x 1031, added
// to: 5.4 us.
template <typename T, bool ADD>
__global__ __launch_bounds__(256) void k_wgrad_join(WgradArgs a) {
  const int chunks = (a.k + 7) / 8;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= int64_t(a.n) * chunks) return;
  const int row = int(i / chunks), col = int(i - int64_t(row) * chunks) * 8;
  T* out = static_cast<T*>(a.out) + int64_t(row) * a.ldo;
  Eight<T> old;
  old.clear();
  if (ADD) old.load(out, col, a.k);
  float sum[8] = {};
  for (int s0 = 0; s0 < a.splits; s0 += 4) {  // four pieces' loads in flight
    Eight<float> v[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v[s].clear();
      if (s0 + s < a.splits) v[s].load(a.parts + (int64_t(s0 + s) * a.n + row) * a.k, col, a.k);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[s].get(e);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = ADD ? old.get(e) + sum[e] : sum[e];
  Eight<T>::store(out, col, a.k, sum);
}

template <typename T, bool ADD>
void launch(const WgradArgs& a, bool dy_bf16, int tile, hipStream_t s) {
  const int edge = tile == kTile256 ? 256 : 128;
  const int64_t tiles = int64_t((a.n + edge - 1) / edge) * ((a.k + edge - 1) / edge);
  const dim3 grid(uint32_t(tiles), uint32_t(a.splits));
  if (!dy_bf16) hipLaunchKernelGGL((k_wgrad_f32<T, ADD>), grid, dim3(256), 0, s, a);
  else if (tile == kTile256) hipLaunchKernelGGL((k_wgrad<T, ADD, false, 2, 4, 4, 2>), grid, dim3(512), 0, s, a);
  else if (a.through) hipLaunchKernelGGL((k_wgrad<T, ADD, true, 2, 2, 2, 2>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_wgrad<T, ADD, false, 2, 2, 2, 2>), grid, dim3(256), 0, s, a);
}

template <typename T, bool ADD>
void join(const WgradArgs& a, hipStream_t s) {
  const int64_t work = (int64_t(a.n) * ((a.k + 7) / 8) + 255) / 256;
  hipLaunchKernelGGL((k_wgrad_join<T, ADD>), dim3(uint32_t(work)), dim3(256), 0, s, a);
}

}  // namespace

int muon_launch_wgrad(const WgradArgs& a, bool dy_bf16, int tile, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool pieces = a.splits > 1, add = a.accumulate != 0;
  if (pieces || (!a.out_bf16 && !add)) launch<float, false>(a, dy_bf16, tile, s);
  else if (!a.out_bf16) launch<float, true>(a, dy_bf16, tile, s);
  else if (add) launch<uint16_t, true>(a, dy_bf16, tile, s);
  else launch<uint16_t, false>(a, dy_bf16, tile, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !pieces) return e;
  if (a.out_bf16 && add) join<uint16_t, true>(a, s);
  else if (a.out_bf16) join<uint16_t, false>(a, s);
  else if (add) join<float, true>(a, s);
  else join<float, false>(a, s);
  return hipGetLastError();
}

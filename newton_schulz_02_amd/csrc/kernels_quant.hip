// Quantising to 8-bit codes and reading them back, for gfx950 (muon_linear.h).  All of it is
// HBM-bound: a value is read once (twice where the columns' maxima come first), its code
// written once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "linear_math.h"
#include "linear_types.h"
#include "tile_store.h"

using namespace muon;

namespace {

// Codes of rows.  L lanes take a row together: a wave (four rows to a workgroup), or a workgroup of
// 256 or 1024 lanes.  The first KEEP chunks of 8 values of each lane stay in registers between the
// maximum and the codes; longer rows are read again (they come from L2).  16384 x 4096 bf16 take 36 us
// (5.6 TB/s), 16384 x 11008 100 us (5.4).
template <typename T, int L, int KEEP>
__global__ __launch_bounds__(L < 256 ? 256 : L) void k_quant_rows(QuantArgs a) {
  constexpr int kThreads = L < 256 ? 256 : L, kRows = kThreads / L;
  __shared__ uint32_t tops[2][L > 64 ? L / 64 : 1];
  const int lane = threadIdx.x % L;
  const int chunks = a.pitch / 8;
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / L; row < a.rows; row += int64_t(gridDim.x) * kRows) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld;
    Eight<T> v[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) v[i].load(x, (lane + i * L) * 8, a.cols);
    typename Eight<T>::Tops tops_of;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) tops_of.take(v[i]);
    for (int c = lane + KEEP * L; c < chunks; c += L) {
      Eight<T> w;
      w.load(x, c * 8, a.cols);
      tops_of.take(w);
    }
    uint32_t top = max64(tops_of.all());
    if constexpr (L > 64) {
      // The two halves of `tops` take turns, so one barrier a row is enough.
      if ((threadIdx.x & 63) == 0) tops[turn & 1][threadIdx.x / 64] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < L / 64; ++w) top = max(top, tops[turn & 1][w]);
      ++turn;
    }
    const RowCoder code(top);
    if (lane == 0) a.scale[row] = code.scale();
    int8_t* q = a.q + row * a.pitch;
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (lane + i * L < chunks) store_codes(q + (lane + i * L) * 8, code.eight(v[i]));
    for (int c = lane + KEEP * L; c < chunks; c += L) {
      Eight<T> w;
      w.load(x, c * 8, a.cols);
      store_codes(q + c * 8, code.eight(w));
    }
  }
}

// Codes of blocks: 16 lanes take a block of 128 values, so a wave reads 1 KB (bf16) at once.  A
// workgroup takes kUnits x 256 consecutive chunks of 8 values, all in flight together.  16384 x 11008
// bf16 take 92 us (5.9 TB/s).
constexpr int kUnits = 4;
template <typename T>
__global__ __launch_bounds__(256) void k_quant_blocks(QuantArgs a, int64_t total) {
  const int chunks = a.pitch / 8;
  for (int64_t base = int64_t(blockIdx.x) * (kUnits * 256); base < total; base += int64_t(gridDim.x) * (kUnits * 256)) {
    const int64_t row0 = base / chunks;
    const int c0 = int(base - row0 * chunks);
    Eight<T> v[kUnits];
    int64_t row[kUnits];
    int c[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = c0 + u * 256 + int(threadIdx.x);
      row[u] = row0 + at / chunks;
      c[u] = at % chunks;
      v[u].clear();
      if (row[u] < a.rows) v[u].load(static_cast<const T*>(a.x) + row[u] * a.ld, c[u] * 8, a.cols);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      typename Eight<T>::Tops tops;
      tops.take(v[u]);
      const uint32_t top = max16(tops.all());
      if (row[u] >= a.rows) continue;
      const BlockCoder code(top);
      store_codes(a.q + row[u] * a.pitch + c[u] * 8, code.eight(v[u]));
      const int group = c[u] / 16;
      if (c[u] % 16 == 0 && group * kCodeBlock < a.cols)
        a.scale[row[u] * ((a.cols + kCodeBlock - 1) / kCodeBlock) + group] = code.scale();
    }
  }
}

// Codes of columns, first launch: parts[s][c] <- the maximum of column c over row strip s of x.
// A workgroup takes 256 columns (32 lanes of 8) and 8 rows at a time.  11008 x 4096 bf16 take 19 us
// (4.8 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_quant_cols_max(QuantArgs a) {
  __shared__ uint32_t tops[8][256 + 8];
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int cols = int(a.rows), rows = a.cols;  // of x
  const int strip = (rows + a.part_rows - 1) / a.part_rows;
  const int lo = int(blockIdx.y) * strip, hi = min(rows, lo + strip);
  const int col = int(blockIdx.x) * 256 + lane * 8;
  typename Eight<T>::Tops top;
  for (int r = lo + sub; r < hi; r += 32) {
    Eight<T> v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u].clear();
      if (r + 8 * u < hi) v[u].load(static_cast<const T*>(a.x) + int64_t(r + 8 * u) * a.ld, col, cols);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) top.take(v[u]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) tops[sub][lane * 8 + e] = top.get(e);
  __syncthreads();
  const int c = threadIdx.x;
  uint32_t t = 0;
#pragma unroll
  for (int s = 0; s < 8; ++s) t = max(t, tops[s][c]);
  if (blockIdx.x * 256 + c < cols) a.parts[int64_t(blockIdx.y) * cols + blockIdx.x * 256 + c] = __uint_as_float(t);
}

// Second launch: 128 columns of x by 128 rows to 128 rows of codes by 128, through LDS.  A lane
// has 8 columns and, at a time, 4 consecutive rows: four codes of one column go to LDS as one
// word.  Rows of 33 words: the words of neighbouring lanes lie 8 banks apart.  11008 x 4096 bf16 take
// 25 us (5.4 TB/s), x coming in part from the cache that the first launch filled.
template <typename T>
__global__ __launch_bounds__(256) void k_quant_cols(QuantArgs a) {
  __shared__ uint32_t tile[128 * 33];
  __shared__ uint32_t tops[2][128];
  __shared__ float inverses[128];
  const int cols = int(a.rows), rows = a.cols;  // of x
  const int across = (cols + 127) / 128;
  const int c0 = int(blockIdx.x) % across * 128, r0 = int(blockIdx.x) / across * 128;
  const int lane = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int mine = threadIdx.x & 127, half = threadIdx.x >> 7;
  uint32_t t[kMaxStrips / 2];  // half of the strips' maxima of one column, all asked for at once
#pragma unroll
  for (int s = 0; s < kMaxStrips / 2; ++s)
    t[s] = __float_as_uint(a.parts[int64_t(min(2 * s + half, a.part_rows - 1)) * cols + min(c0 + mine, cols - 1)]);
  Eight<T> v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = r0 + (u >> 2) * 64 + sub * 4 + (u & 3);
    v[u].clear();
    if (r < rows) v[u].load(static_cast<const T*>(a.x) + int64_t(r) * a.ld, c0 + lane * 8, cols);
  }
#pragma unroll
  for (int s = 1; s < kMaxStrips / 2; ++s) t[0] = max(t[0], t[s]);
  tops[half][mine] = t[0];
  __syncthreads();
  // One division a column, not one for each lane that has it.
  if (threadIdx.x < 128) {
    const RowCoder code(max(tops[0][mine], tops[1][mine]));
    inverses[mine] = code.inverse;
    if (r0 == 0 && c0 + mine < cols) a.scale[c0 + mine] = code.scale();
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = lane * 8 + e;
    const RowCoder code(max(tops[0][c], tops[1][c]), inverses[c]);
    uint32_t w[2];
    code.template codes<8, Eight<T>::kShort>(w, [&](int u) { return v[u].get(e); });
    tile[c * 33 + sub] = w[0];
    tile[c * 33 + 16 + sub] = w[1];
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = u * 32 + int(threadIdx.x) / 8, part = int(threadIdx.x) & 7;
    if (c0 + c >= cols) continue;
    const uint32_t* w = tile + c * 33 + part * 4;
    *reinterpret_cast<uint4*>(a.q + int64_t(c0 + c) * a.pitch + r0 + part * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Values of codes: a lane takes 16 bytes of the result, 8 or 4 codes of one row, so that a wave
// writes whole lines.  16384 x 11008 to bf16 take 95 us (5.7 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_dequant(DequantArgs a, int64_t total) {
  constexpr int E = Run<T>::E;
  const int chunks = (a.cols + E - 1) / E;
  for (int64_t base = int64_t(blockIdx.x) * (kUnits * 256); base < total; base += int64_t(gridDim.x) * (kUnits * 256)) {
    const int64_t row0 = base / chunks;
    const int c0 = int(base - row0 * chunks);
    uint32_t q[kUnits][E / 4];
    float s[kUnits];
    int64_t row[kUnits];
    int c[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = c0 + u * 256 + int(threadIdx.x);
      row[u] = row0 + at / chunks;
      c[u] = at % chunks * E;
      if (row[u] < a.rows) {
        const int8_t* p = a.q + row[u] * a.pitch + c[u];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) q[u][i] = reinterpret_cast<const uint32_t*>(p)[i];
        s[u] = a.block ? a.scale[row[u] * ((a.cols + kCodeBlock - 1) / kCodeBlock) + c[u] / kCodeBlock] : a.scale[row[u]];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (row[u] < a.rows) {
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = code_of(q[u][e / 4], e % 4) * s[u];
        Run<T> x;
        x.set(f);
        T* out = static_cast<T*>(a.out) + row[u] * a.ld;
        if (c[u] + E <= a.cols) x.template store<true>(out, c[u], a.cols);
        else x.template store<false>(out, c[u], a.cols);
      }
  }
}

// Rows of bf16 to rows of ldd elements (a multiple of 8), zeros behind their end.
__global__ __launch_bounds__(256) void k_pack_rows(const uint16_t* src, int64_t ld, uint16_t* dst, int64_t ldd,
                                                   int64_t rows, int32_t cols) {
  const int chunks = int(ldd / 8);
  const int64_t total = rows * chunks;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / chunks;
    const int c = int(i - row * chunks);
    Eight<uint16_t> v;
    v.load(src + row * ld, c * 8, cols);
    *reinterpret_cast<uint4*>(dst + row * ldd + c * 8) = v.raw();
  }
}

int grid_of(int64_t n) { return int(std::min<int64_t>(n, 1 << 20)); }

template <typename T>
int quant_rows(const QuantArgs& a, hipStream_t s) {
  // A wave keeps 1024 or 2048 values in registers, 256 lanes 4096 to 16384, no more than the row needs:
  // the registers decide how many rows are in flight.  (16384 bf16 rows of 2048 take 17.7 us with a
  // wave each and 21.6 with 256 lanes, of 4096 then 47 and 39.7; of 11008 100 with room for 12288 and
  // 128 with room for 16384.)
  const dim3 waves(grid_of((a.rows + 3) / 4)), groups(grid_of(a.rows));
  if (a.pitch <= 1024) hipLaunchKernelGGL((k_quant_rows<T, 64, 2>), waves, dim3(256), 0, s, a);
  else if (a.pitch <= 2048) hipLaunchKernelGGL((k_quant_rows<T, 64, 4>), waves, dim3(256), 0, s, a);
  else if (a.pitch <= 4096) hipLaunchKernelGGL((k_quant_rows<T, 256, 2>), groups, dim3(256), 0, s, a);
  else if (a.pitch <= 8192) hipLaunchKernelGGL((k_quant_rows<T, 256, 4>), groups, dim3(256), 0, s, a);
  else if (a.pitch <= 12288) hipLaunchKernelGGL((k_quant_rows<T, 256, 6>), groups, dim3(256), 0, s, a);
  else if (a.pitch <= 16384) hipLaunchKernelGGL((k_quant_rows<T, 256, 8>), groups, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_quant_rows<T, 1024, 4>), groups, dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <typename T>
int quant_cols(const QuantArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_quant_cols_max<T>, dim3(uint32_t((a.rows + 255) / 256), uint32_t(a.part_rows)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t tiles = (a.rows + 127) / 128 * (a.pitch / 128);
  hipLaunchKernelGGL(k_quant_cols<T>, dim3(uint32_t(tiles)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int muon_launch_quant_rows(const QuantArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return bf16 ? quant_rows<uint16_t>(a, s) : quant_rows<float>(a, s);
}

int muon_launch_quant_blocks(const QuantArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t total = a.rows * (a.pitch / 8);
  const dim3 grid(grid_of((total + kUnits * 256 - 1) / (kUnits * 256)));
  if (bf16) hipLaunchKernelGGL(k_quant_blocks<uint16_t>, grid, dim3(256), 0, s, a, total);
  else hipLaunchKernelGGL(k_quant_blocks<float>, grid, dim3(256), 0, s, a, total);
  return hipGetLastError();
}

int muon_launch_quant_cols(const QuantArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return bf16 ? quant_cols<uint16_t>(a, s) : quant_cols<float>(a, s);
}

int muon_launch_dequant(const DequantArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t total = a.rows * (bf16 ? (a.cols + 7) / 8 : (a.cols + 3) / 4);
  const dim3 grid(grid_of((total + kUnits * 256 - 1) / (kUnits * 256)));
  if (bf16) hipLaunchKernelGGL(k_dequant<uint16_t>, grid, dim3(256), 0, s, a, total);
  else hipLaunchKernelGGL(k_dequant<float>, grid, dim3(256), 0, s, a, total);
  return hipGetLastError();
}

int muon_launch_pack_rows(const void* src, int64_t ld, void* dst, int64_t ldd, int64_t rows, int32_t cols, void* stream) {
  const int64_t total = rows * (ldd / 8);
  hipLaunchKernelGGL(k_pack_rows, dim3(grid_of((total + 255) / 256)), dim3(256), 0, static_cast<hipStream_t>(stream),
                     static_cast<const uint16_t*>(src), ld, static_cast<uint16_t*>(dst), ldd, rows, cols);
  return hipGetLastError();
}

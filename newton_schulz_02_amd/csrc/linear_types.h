// Arguments of the kernels of the 8-bit linear operators (muon_linear.h), shared by the host
// and the device code.
#pragma once

#include <cstdint>

namespace muon {

constexpr int kCodeBlock = 128;         // columns of a block scale; codes' rows are padded to it
constexpr int kFewRows = 64;              // most rows of the int8 products' kernel for few rows
constexpr int kMaxStrips = 32;            // row strips of the columns' maxima
constexpr int kMaxIntSum = 131071;      // 128 * 128 * 131071 < 2^31

// Result tiles of the products: 128 x 128 (4 waves, two workgroups per compute unit), 256 x 128 and
// 256 x 256 (8 waves).
enum LinearTile { kTile128 = 0, kTile256x128 = 1, kTile256 = 2 };

struct QuantArgs {
  const void* x;
  int64_t ld;
  int8_t* q;
  float* scale;
  int64_t rows;       // of the codes
  int32_t cols;
  int32_t pitch;
  float* parts;       // transposed: part_rows x (rows) partial maxima
  int32_t part_rows;  // transposed: row strips of x, each with a row of partial maxima
};

struct DequantArgs {
  const int8_t* q;
  const float* scale;
  void* out;
  int64_t ld;
  int64_t rows;
  int32_t cols;
  int32_t pitch;
  int32_t block;
};

struct IntArgs {
  const int8_t* a;       // rows x pitch
  const int8_t* b;       // cols x pitch
  const float* a_scale;
  const float* b_scale;
  const void* x;         // fused: values instead of a and a_scale (NULL where there are no columns)
  int64_t ldx;
  void* out;
  int64_t ldo;
  int32_t rows, cols;    // of out
  int32_t k;             // columns summed over
  int32_t pitch;
  int32_t fused;         // few rows, whose codes the kernel makes itself
  int32_t x_bf16;
  int32_t out_bf16;
};

struct WgradArgs {
  const void* dy;        // tokens x n
  int64_t lddy;
  const int8_t* q;       // tokens x pitch
  const float* scale;    // tokens x groups
  void* out;             // n x k
  int64_t ldo;
  float* parts;          // splits > 1: splits partial results of n x k, joined by a second kernel
  int32_t tokens;
  int32_t n, k;
  int32_t n_read;        // bf16: columns of dy that can be read, a multiple of 8
  int32_t through;       // bf16, 128 x 128 tiles: dy's rows are not 16-byte aligned
  int32_t pitch, groups;
  int32_t splits;        // pieces of the tokens
  int32_t piece;         // tokens of a piece (a multiple of 64)
  int32_t accumulate;
  int32_t out_bf16;
};

}  // namespace muon

// Kernel launchers (defined in the .hip files).  Each returns a hipError_t as int.
int muon_launch_quant_rows(const muon::QuantArgs& a, bool bf16, void* stream);
int muon_launch_quant_blocks(const muon::QuantArgs& a, bool bf16, void* stream);
int muon_launch_quant_cols(const muon::QuantArgs& a, bool bf16, void* stream);
int muon_launch_dequant(const muon::DequantArgs& a, bool bf16, void* stream);
int muon_launch_int8(const muon::IntArgs& a, int tile, void* stream);
int muon_launch_int8_few(const muon::IntArgs& a, void* stream);
// dy's rows, not 16-byte aligned, to rows of ld elements that are.
int muon_launch_pack_rows(const void* src, int64_t ld, void* dst, int64_t ldd, int64_t rows, int32_t cols, void* stream);
int muon_launch_wgrad(const muon::WgradArgs& a, bool dy_bf16, int tile, void* stream);

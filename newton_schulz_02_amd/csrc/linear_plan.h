// Host side of the 8-bit linear operators (muon_linear.h): validation, and how each call is cut
// into launches.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include "../../include/muon_linear.h"
#include "linear_types.h"

namespace muon {

constexpr int64_t kMaxLinear = int64_t(1) << 30;  // rows or columns of an operand

// Memory of a view or of codes: `rows` runs of `run` bytes, `step` bytes from one to the next.
struct Span {
  const char* name;
  uintptr_t lo;
  int64_t rows, run, step;
  uintptr_t hi() const { return lo + uintptr_t((rows - 1) * step + run); }
  bool empty() const { return rows == 0 || run == 0; }
};

// What a call reads and writes, and the workspace that it needs.
struct LinearBuffers {
  Span spans[5];
  int count = 0;
  size_t ws_bytes = 0;
};

// Each fills what its call needs, or returns a status with the reason in *err.

struct QuantPlan {
  QuantArgs args;
  bool bf16, transpose, empty;
  int32_t block;
  LinearBuffers buf;
};
// codes may be NULL: sizes only.
int plan_quantize(const muon_view* x, int32_t transpose, const muon_codes* codes, QuantPlan* p, std::string* err);

struct DequantPlan {
  DequantArgs args;
  bool bf16, empty;
};
int plan_dequantize(const muon_codes* codes, const muon_view* out, DequantPlan* p, std::string* err);

struct IntPlan {
  IntArgs args;
  bool empty;       // no result
  bool few;         // the kernel for at most kFewRows rows
  int tile;         // LinearTile otherwise
  bool quantise;    // muon_int8_linear: a launch before makes the codes of x
  QuantPlan quant;  // with codes at the workspace's start, scales at scale_off
  size_t scale_off;
  LinearBuffers buf;
};
// Either a (codes) or x (values); out may be NULL: sizes only.
int plan_int8(const muon_codes* a, const muon_view* x, const muon_codes* b, const muon_view* out, IntPlan* p,
              std::string* err);

struct WgradPlan {
  WgradArgs args;
  bool bf16, empty;
  int tile;
  bool pack;         // dy is copied to aligned rows first, at the workspace's start
  int64_t pack_ld;
  size_t parts_off;
  LinearBuffers buf;
};
// out may be NULL: sizes only.
int plan_wgrad(const muon_view* dy, const muon_codes* x, const muon_view* out, int32_t accumulate, WgradPlan* p,
               std::string* err);

// MUON_OK, or why a call cannot use this workspace.
int check_linear_workspace(const LinearBuffers& b, const void* workspace, size_t bytes, std::string* err);

}  // namespace muon

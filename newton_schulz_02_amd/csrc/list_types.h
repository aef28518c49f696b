// Types shared by the host side and the kernels of the list operators (muon_grad.h) and of the
// clipped Muon step.
#pragma once

#include <cstdint>

#include "muon_internal.h"

namespace muon {

// Where a clip coefficient comes from; norm null: none (1).
struct ClipArg {
  const float* norm;
  float max_norm;
};

// A decay rate of AdamW's state as the kernels use it: beta = hi + lo, hi being the largest
// float that is not above it, and rest = 1 - beta, rounded once from 64 bits.  One float of beta
// is not enough: 1 - 0.9999f is off by 1.7e-4 of itself, and so would v be, after one step with
// a rounded beta's own difference from 1, after many with the true one.
struct AdamBeta {
  float hi, lo, rest;
};
struct AdamBetas {
  AdamBeta b1, b2;
};

constexpr int64_t kLine = 128;         // gradient chunks start on multiples of this address
constexpr int kTickets = 8;            // groups in which a norm's workgroups count themselves
constexpr int64_t kListTickets = 256;  // a list's workspace: status word, counts, entries
constexpr int64_t kListHead = kListTickets + (kTickets + 1) * kLine;
constexpr int64_t kGradChunk = 32768;  // bytes of one chunk of a gradient list
// Elements of one chunk of an AdamW list: 2048 in runs of 16 per XCD against 1024 in runs of 32
// (which are better than of 16), us: bf16 param and gradient 461 / 489, with 37 x 1031 elements a
// tensor 139 / 150; bf16 with master 1168 / 1186, with fp32 gradients 321 / 312; bf16 with fp32
// gradients 262 / 263; fp32 305 / 290, with bf16 gradients 283 / 271; a ragged mixed list and
// short ones the same.  One size for all: 2048 gains 6 % where it gains, and loses 5 % on fp32.
constexpr int64_t kAdamChunk = 2048;
// Most workgroups (and partial results) of a norm: a few long ones, each 32 KiB of loads ahead.
// us of a 4096-hidden layer in bf16 / of 512 small fp32 matrices: 512 workgroups 61.5 / 200,
// 768 63.4 / 205, 1024 64.1 / 207, 2048 69.8 / 223; 16 KiB chunks with 1024 63.4 / 204; 64 KiB
// with 512 65.7 / 208.
constexpr int kNormParts = 512;

struct GradRec {
  uint64_t ptr;
  int64_t n;
  uint32_t first;  // first chunk
  uint32_t dtype;
};

struct AdamRec {
  uint64_t param, grad, m, v, master;
  int64_t n;
  uint32_t first;  // first chunk
  uint16_t param_bf16, grad_bf16;
  float decay;
  uint32_t reserved;
};

struct GradArgs {
  const GradRec* recs;
  const uint32_t* map;  // tensor of each chunk
  uint32_t chunks;
  double* parts;     // one per workgroup of the norm
  uint32_t* tickets; // counts of the norm's workgroups that are done; 0 between launches
  float* norm;     // output of the norm
  int32_t inf;     // largest magnitude instead of L2
  ClipArg clip;
};

struct AdamListArgs {
  const AdamRec* recs;
  const uint32_t* map;  // tensor of each chunk
  uint32_t chunks;
  ClipArg clip;
  AdamBetas betas;
  float lr, eps, wd;
  float bc1, bc2;
};

}  // namespace muon

// Kernel launchers (kernels_list.hip, kernels_elementwise.hip).  Each returns a hipError_t as int.
int muon_launch_grad_map(const muon::GradRec* recs, int count, uint32_t chunks, uint32_t* map, void* stream);
int muon_launch_adamw_map(const muon::AdamRec* recs, int count, uint32_t chunks, uint32_t* map, void* stream);
int muon_launch_grad_norm(const muon::GradArgs& a, void* stream);
int muon_launch_grad_clip(const muon::GradArgs& a, void* stream);
int muon_launch_adamw_list(const muon::AdamListArgs& a, void* stream);
// muon_launch_adamw with betas in more than fp32 (a.beta1 and a.beta2 are not read).
int muon_launch_adamw(const muon::AdamArgs& a, const muon::AdamBetas& b, void* stream);
// muon_launch_momentum with G scaled by the coefficient of `clip` (its norm is not null).
int muon_launch_momentum_clipped(const muon::MomArgs& a, const muon::ClipArg& clip, int dtype, void* stream);

// Host layout of the list operators (muon_grad.h): the descriptor table of a list of
// tensors, cut into chunks, as the kernels of kernels_list.hip read it.
//
// A list's chunks are numbered through: tensor i owns the chunks [first_i, first_{i+1}), the
// last of each tensor being partial.  Empty tensors have no entry.  Tables are written to the
// caller's workspace once (the *_init calls) and only read afterwards:
//   head (status word, the norm's counts), entries, the map (the entry of each chunk, filled
//   by a kernel), and for a gradient list the norm's partial results.
#pragma once

#include <cstdint>
#include <string>
#include <vector>

#include "../../include/muon_grad.h"
#include "list_types.h"

namespace muon {

constexpr int32_t kMaxList = 1 << 20;              // tensors in one list
constexpr int64_t kMaxListElems = int64_t(1) << 40;  // elements in one list

// A buffer of a list's tensor; no output may overlap another output or any gradient.
struct ListSpan {
  uintptr_t lo, hi;
  int32_t tensor;
  bool output;
};

struct ListTable {
  std::vector<ListSpan> spans;  // in order of address
  std::vector<uint32_t> words;  // head and entries, as uploaded
  uint32_t chunks = 0;
  int32_t entries = 0;          // tensors that are not empty
  int64_t elems = 0;
  double read_bytes = 0.0;      // gradients (all operands of an AdamW list) read once
  double write_bytes = 0.0;     // outputs written once
  size_t map_off = 0;           // bytes from the workspace's start; the norm's partial results follow the map
  size_t ws_bytes = 0;
};

// Validate a list and lay out its table.  MUON_OK, or a status with the reason in *err.
int build_grad_list(const muon_grad* grads, int32_t count, ListTable* t, std::string* err);
int build_adamw_list(const adamw_tensor* tensors, int32_t count, ListTable* t, std::string* err);

// MUON_EALIAS when the list's workspace overlaps one of its buffers.
int check_list_workspace(const ListTable& t, const void* workspace, std::string* err);

// What a muon_grad_list / adamw_list holds.
struct ListHandle {
  uint64_t magic;     // kind of list
  uint64_t workspace;
  uint32_t chunks;
  int32_t device;
  uint64_t map_off;
  uint64_t capture;   // the graph capture the layout was recorded in, 0: none
  double read_bytes, write_bytes;
  uint64_t check;     // over the fields above: an uninitialised or foreign handle is refused
};
constexpr uint64_t kGradListMagic = 0x6d756f6e67726164ull;
constexpr uint64_t kAdamListMagic = 0x6d756f6e6164616dull;

uint64_t handle_check(const ListHandle& h);

// Bytes from the workspace's start to what follows the map of a list's chunks.
inline size_t end_of_map(size_t map_off, uint32_t chunks) {
  return map_off + size_t(round_up(int64_t(chunks) * 4, 256));
}

}  // namespace muon

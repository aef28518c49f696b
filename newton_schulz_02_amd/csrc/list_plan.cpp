// Host validation and layout of the list operators (see list_plan.h).
#include "list_plan.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

namespace muon {

namespace {

int refuse(std::string* err, int status, int32_t i, const char* what) {
  char buf[160];
  snprintf(buf, sizeof buf, "tensor %d: %s", i, what);
  *err = buf;
  return status;
}

// No output may overlap another output or any gradient (which may overlap each other).
int check_spans(std::vector<ListSpan>& spans, std::string* err) {
  std::sort(spans.begin(), spans.end(), [](const ListSpan& a, const ListSpan& b) { return a.lo < b.lo; });
  uintptr_t out_hi = 0, in_hi = 0;
  int32_t out_t = -1, in_t = -1;
  for (const ListSpan& s : spans) {
    const bool hits_out = s.lo < out_hi, hits_in = s.output && s.lo < in_hi;
    if (hits_out || hits_in) {
      char buf[160];
      snprintf(buf, sizeof buf, "tensor %d: buffer overlaps a buffer of tensor %d", s.tensor, hits_out ? out_t : in_t);
      *err = buf;
      return MUON_EALIAS;
    }
    if (s.output) {
      if (s.hi > out_hi) out_hi = s.hi, out_t = s.tensor;
    } else if (s.hi > in_hi) {
      in_hi = s.hi, in_t = s.tensor;
    }
  }
  return MUON_OK;
}

int width(int32_t dtype) { return dtype == MUON_BF16 ? 2 : dtype == MUON_F32 ? 4 : 0; }

template <typename Rec>
void lay_out(const std::vector<Rec>& recs, ListTable* t) {
  static_assert(sizeof(Rec) % 4 == 0, "table entries are uploaded as 32-bit words");
  t->entries = int32_t(recs.size());
  t->words.assign((kListHead + recs.size() * sizeof(Rec)) / 4, 0);
  if (!recs.empty()) std::memcpy(t->words.data() + kListHead / 4, recs.data(), recs.size() * sizeof(Rec));
  t->map_off = size_t(round_up(int64_t(t->words.size()) * 4, 256));
  t->ws_bytes = end_of_map(t->map_off, t->chunks);
}

int check_count(const void* list, int32_t count, std::string* err) {
  if (count < 0 || count > kMaxList) {
    *err = "count outside [0, " + std::to_string(kMaxList) + "]";
    return MUON_EINVAL;
  }
  if (count > 0 && !list) {
    *err = "list is NULL";
    return MUON_EINVAL;
  }
  return MUON_OK;
}

}  // namespace

int build_grad_list(const muon_grad* grads, int32_t count, ListTable* t, std::string* err) {
  int rc = check_count(grads, count, err);
  if (rc != MUON_OK) return rc;
  std::vector<GradRec> recs;
  uint64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    const muon_grad& x = grads[i];
    const int es = width(x.dtype);
    if (!es) return refuse(err, MUON_EINVAL, i, "unknown dtype");
    if (x.reserved != 0) return refuse(err, MUON_EINVAL, i, "reserved field must be 0");
    if (x.n < 0 || x.n > kMaxListElems - t->elems) return refuse(err, MUON_EINVAL, i, "n is negative or too large");
    if (x.n == 0) continue;
    const uintptr_t p = uintptr_t(x.grad);
    if (!p) return refuse(err, MUON_EINVAL, i, "NULL pointer");
    if (p % uintptr_t(es)) return refuse(err, MUON_EINVAL, i, "pointer not aligned to its element size");
    if (uintptr_t(x.n) * uintptr_t(es) > UINTPTR_MAX - p) return refuse(err, MUON_EINVAL, i, "buffer passes the end of memory");
    t->spans.push_back({p, p + uintptr_t(x.n) * uintptr_t(es), i, true});
    recs.push_back({uint64_t(p), x.n, uint32_t(chunks), uint32_t(x.dtype)});
    // Chunks start on line boundaries, the first one at or before the tensor.
    chunks += uint64_t(ceil_div(x.n * es + int64_t(p % uintptr_t(kLine)), kGradChunk));
    t->elems += x.n;
    t->read_bytes += double(x.n) * es;
  }
  t->write_bytes = t->read_bytes;
  if ((rc = check_spans(t->spans, err)) != MUON_OK) return rc;
  t->chunks = uint32_t(chunks);
  lay_out(recs, t);
  t->ws_bytes += kNormParts * sizeof(double);
  return MUON_OK;
}

int build_adamw_list(const adamw_tensor* tensors, int32_t count, ListTable* t, std::string* err) {
  int rc = check_count(tensors, count, err);
  if (rc != MUON_OK) return rc;
  std::vector<AdamRec> recs;
  uint64_t chunks = 0;
  for (int32_t i = 0; i < count; ++i) {
    const adamw_tensor& x = tensors[i];
    const int ep = width(x.param_dtype), eg = width(x.grad_dtype);
    if (!ep || !eg) return refuse(err, MUON_EINVAL, i, "unknown dtype");
    if (x.reserved != 0) return refuse(err, MUON_EINVAL, i, "reserved field must be 0");
    if (!std::isfinite(x.decay)) return refuse(err, MUON_EINVAL, i, "decay is not finite");
    if (x.master && x.param_dtype != MUON_BF16) return refuse(err, MUON_EINVAL, i, "a master belongs to a bf16 param only");
    if (x.n < 0 || x.n > kMaxListElems - t->elems) return refuse(err, MUON_EINVAL, i, "n is negative or too large");
    if (x.n == 0) continue;
    if (!x.param || !x.grad || !x.m || !x.v) return refuse(err, MUON_EINVAL, i, "NULL pointer");
    const struct {
      uintptr_t p;
      int es;
      bool output;
    } bufs[5] = {{uintptr_t(x.param), ep, true},
                 {uintptr_t(x.grad), eg, false},
                 {uintptr_t(x.m), 4, true},
                 {uintptr_t(x.v), 4, true},
                 {uintptr_t(x.master), 4, true}};
    for (const auto& b : bufs) {
      if (!b.p) continue;
      if (b.p % uintptr_t(b.es)) return refuse(err, MUON_EINVAL, i, "pointer not aligned to its element size");
      if (uintptr_t(x.n) * uintptr_t(b.es) > UINTPTR_MAX - b.p) return refuse(err, MUON_EINVAL, i, "buffer passes the end of memory");
      t->spans.push_back({b.p, b.p + uintptr_t(x.n) * uintptr_t(b.es), i, b.output});
      // A master takes the param's place as what is read.
      if (!(x.master && b.p == uintptr_t(x.param))) t->read_bytes += double(x.n) * b.es;
      if (b.output) t->write_bytes += double(x.n) * b.es;
    }
    AdamRec r;
    std::memset(&r, 0, sizeof r);
    r.param = uint64_t(uintptr_t(x.param));
    r.grad = uint64_t(uintptr_t(x.grad));
    r.m = uint64_t(uintptr_t(x.m));
    r.v = uint64_t(uintptr_t(x.v));
    r.master = uint64_t(uintptr_t(x.master));
    r.n = x.n;
    r.first = uint32_t(chunks);
    r.param_bf16 = x.param_dtype == MUON_BF16;
    r.grad_bf16 = x.grad_dtype == MUON_BF16;
    r.decay = x.decay;
    recs.push_back(r);
    // Chunks start where m lies on a line boundary, the first one at or before the tensor.
    chunks += uint64_t(ceil_div(x.n + int64_t(r.m % uint64_t(kLine) / 4), kAdamChunk));
    t->elems += x.n;
  }
  if ((rc = check_spans(t->spans, err)) != MUON_OK) return rc;
  t->chunks = uint32_t(chunks);
  lay_out(recs, t);
  return MUON_OK;
}

int check_list_workspace(const ListTable& t, const void* workspace, std::string* err) {
  const uintptr_t lo = uintptr_t(workspace), hi = lo + t.ws_bytes;
  for (const ListSpan& s : t.spans)
    if (s.lo < hi && lo < s.hi) return refuse(err, MUON_EALIAS, s.tensor, "the workspace overlaps a buffer");
  return MUON_OK;
}

uint64_t handle_check(const ListHandle& h) {
  uint64_t words[sizeof(ListHandle) / 8 - 1], x = 0x9e3779b97f4a7c15ull;
  std::memcpy(words, &h, sizeof words);
  for (uint64_t w : words) {
    x ^= w;
    x *= 0xbf58476d1ce4e5b9ull;
    x ^= x >> 31;
  }
  return x;
}

}  // namespace muon

// Host validation and planning of the 8-bit linear operators (see linear_plan.h).
#include "linear_plan.h"

#include <algorithm>
#include <cstring>
#include <initializer_list>

#include "muon_internal.h"

namespace muon {

namespace {

int refuse(std::string* err, int status, const std::string& what) {
  *err = what;
  return status;
}

int width(int32_t dtype) { return dtype == MUON_BF16 ? 2 : dtype == MUON_F32 ? 4 : 0; }

// Whether two spans share a byte.  Of spans with the same step (rows of one wider buffer) the
// columns are compared; others overlap where their whole ranges do.
bool overlap(const Span& a, const Span& b) {
  if (a.empty() || b.empty() || a.hi() <= b.lo || b.hi() <= a.lo) return false;
  const bool one_row = a.rows == 1 || b.rows == 1;
  const int64_t step = a.rows == 1 ? b.step : a.step;
  if ((!one_row && a.step != b.step) || (a.rows == 1 && b.rows == 1)) return true;
  // Offset of b's columns behind a's, in [0, step).
  const int64_t d = a.lo <= b.lo ? int64_t((b.lo - a.lo) % uintptr_t(step))
                                 : (step - int64_t((a.lo - b.lo) % uintptr_t(step))) % step;
  return d < a.run || step - d < b.run;
}

// No output may overlap another output or an input; *b (may be NULL) keeps them all.
int check_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins, LinearBuffers* b, std::string* err) {
  if (b) {
    b->count = 0;
    for (const Span& s : outs) b->spans[b->count++] = s;
    for (const Span& s : ins) b->spans[b->count++] = s;
  }
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return refuse(err, MUON_EALIAS, std::string(o->name) + " overlaps " + p->name);
    for (const Span& i : ins)
      if (overlap(*o, i)) return refuse(err, MUON_EALIAS, std::string(o->name) + " overlaps " + i.name);
  }
  return MUON_OK;
}

int check_size(const char* name, int64_t rows, int64_t cols, std::string* err) {
  if (rows < 0 || cols < 0 || rows > kMaxLinear || cols > kMaxLinear)
    return refuse(err, MUON_EINVAL, std::string(name) + ": rows and cols must be in [0, 2^30]");
  return MUON_OK;
}

// `rows` runs (at least one) of `run` bytes, `step` bytes from one to the next.
int check_pointer(const char* name, const void* p, uintptr_t align, int64_t rows, int64_t run, int64_t step, std::string* err) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if (!at) return refuse(err, MUON_EINVAL, std::string(name) + ": NULL pointer");
  if (at % align) return refuse(err, MUON_EINVAL, std::string(name) + ": pointer not aligned to " + std::to_string(align) + " bytes");
  // Within the 2^62 bytes that the kernels' 64-bit offsets reach.
  if (uintptr_t(run) > UINTPTR_MAX - at ||
      uintptr_t(rows - 1) > std::min<uintptr_t>(UINTPTR_MAX - at - uintptr_t(run), uintptr_t(1) << 62) / uintptr_t(step))
    return refuse(err, MUON_EINVAL, std::string(name) + ": buffer passes the end of memory");
  return MUON_OK;
}

int check_view(const char* name, const muon_view* v, Span* span, std::string* err) {
  if (!v) return refuse(err, MUON_EINVAL, std::string(name) + " is NULL");
  const int es = width(v->dtype);
  if (!es) return refuse(err, MUON_EINVAL, std::string(name) + ": unknown dtype");
  if (v->reserved != 0) return refuse(err, MUON_EINVAL, std::string(name) + ": reserved field must be 0");
  const int rc = check_size(name, v->rows, v->cols, err);
  if (rc != MUON_OK) return rc;
  *span = {name, reinterpret_cast<uintptr_t>(v->data), v->rows, v->cols * es, v->cols * es};
  if (span->empty()) return MUON_OK;
  if (v->rows > 1) {
    if (v->ld < v->cols || v->ld > (int64_t(1) << 32))
      return refuse(err, MUON_EINVAL, std::string(name) + ": ld must be in [cols, 2^32]");
    span->step = v->ld * es;
  }
  return check_pointer(name, v->data, uintptr_t(es), v->rows, span->run, span->step, err);
}

int64_t groups_of(const muon_codes& c) { return c.block ? ceil_div(c.cols, kCodeBlock) : 1; }

int check_codes(const char* name, const muon_codes* c, int32_t block, Span* q, Span* scale, std::string* err) {
  if (!c) return refuse(err, MUON_EINVAL, std::string(name) + " is NULL");
  if (c->reserved != 0) return refuse(err, MUON_EINVAL, std::string(name) + ": reserved field must be 0");
  if (c->block != 0 && c->block != kCodeBlock) return refuse(err, MUON_EINVAL, std::string(name) + ": block must be 0 or 128");
  if (block >= 0 && c->block != block)
    return refuse(err, MUON_EINVAL, std::string(name) + (block ? ": codes by block are needed" : ": codes by row are needed"));
  int rc = check_size(name, c->rows, c->cols, err);
  if (rc != MUON_OK) return rc;
  const int64_t pitch = MUON_CODES_PITCH(c->cols), groups = groups_of(*c);
  *q = {name, reinterpret_cast<uintptr_t>(c->q), c->rows, pitch, pitch};
  *scale = {name, reinterpret_cast<uintptr_t>(c->scale), c->rows, groups * 4, groups * 4};
  if (!q->empty() && (rc = check_pointer(name, c->q, 16, c->rows, pitch, pitch, err)) != MUON_OK) return rc;
  if (!scale->empty() && (rc = check_pointer(name, c->scale, 4, c->rows, groups * 4, groups * 4, err)) != MUON_OK) return rc;
  return MUON_OK;
}

void set_quant(const muon_view& x, bool transpose, QuantPlan* p) {
  QuantArgs& a = p->args;
  std::memset(&a, 0, sizeof a);
  p->bf16 = x.dtype == MUON_BF16;
  p->transpose = transpose;
  p->block = 0;
  p->buf.ws_bytes = 0;
  a.x = x.data;
  a.ld = x.rows > 1 ? x.ld : x.cols;
  a.rows = transpose ? x.cols : x.rows;
  a.cols = int32_t(transpose ? x.rows : x.cols);
  a.pitch = int32_t(MUON_CODES_PITCH(a.cols));
  p->buf.count = 0;
  p->empty = a.rows == 0;
  if (transpose && a.rows > 0 && a.cols > 0) {
    // Strips of at least 64 rows of x, about 1024 workgroups of 256 columns, and at most kMaxStrips,
    // whose maxima the second launch reads again for each of its tiles.
    const int64_t across = ceil_div(a.rows, 256);
    a.part_rows = int32_t(std::max<int64_t>(1, std::min<int64_t>({ceil_div(a.cols, 64), ceil_div(1024, across), kMaxStrips})));
    p->buf.ws_bytes = size_t(a.rows) * size_t(a.part_rows) * 4;
  }
}

// A launch has fewer than 2^32 lanes.
bool quant_too_large(const QuantPlan& p) {
  return p.transpose && ceil_div(p.args.rows, 128) * (p.args.pitch / 128) > (1 << 23);
}

// Few tiles: the tokens are cut into pieces, whose partial results a second launch joins.  In
// microseconds: a step of 64 tokens takes 0.63 where each workgroup has a compute unit and 0.8 where
// some share one (fp32 dy: 4.5, and two share one with little loss); a join takes 1.7, a tenth for each
// piece and its bytes at 5 TB/s.  (777 tokens, 517 x 1031 results: 17.2 whole, 15.7 in the 3 pieces
// that this chooses; 8192, 768 x 768: 85.1 whole, 24.8 in 6, 24.1 in the 7 that this chooses, 28.3 in 8.)
int32_t wgrad_splits(int64_t tiles, const WgradArgs& a, bool bf16) {
  const double steps = double(ceil_div(a.tokens, 64)), bytes = 8.0 * a.n * a.k;
  auto step = [&](int64_t groups) {
    if (!bf16) return 4.5 * std::max(1.0, double(groups) / 384);
    return groups <= kMaxUnits ? 0.63 : 0.8 * std::max(1.0, double(groups) / (2 * kMaxUnits));
  };
  double best = step(tiles) * steps;
  int32_t splits = 1;
  for (int32_t s = 2; s <= 64 && s <= steps / (bf16 ? 2 : 1) && tiles * s <= 3 * kMaxUnits; ++s) {
    const double t = step(tiles * s) * double(ceil_div(int64_t(steps), s)) + 1.7 + 0.1 * s + s * bytes / 5e6;
    if (t < best) best = t, splits = s;
  }
  return splits;
}

// Which tile: the fewest rounds over the compute units, weighed by what a round takes as a part of a
// round of 256 x 256 tiles (a smaller tile reads more of its operands for each result).  4096
// columns summed over, in tiles of 256 x 256, 256 x 128 and 128 x 128: 4096 x 4096 results take 64, 78 and
// 86 us, 2048 x 4096 take 42, 39 and 42.5, 512 x 4096 37, 24 and 17.3.
int int8_tile(int64_t rows, int64_t cols) {
  const int64_t full = ceil_div(ceil_div(rows, 256) * ceil_div(cols, 256), kMaxUnits);
  const int64_t half = ceil_div(ceil_div(rows, 256) * ceil_div(cols, 128), kMaxUnits);
  const int64_t tiles = ceil_div(rows, 128) * ceil_div(cols, 128);
  const double t256 = 1.0 * full, t256x128 = 0.56 * half;
  const double t128 = tiles <= kMaxUnits ? 0.33 : 0.62 * ceil_div(tiles, 2 * kMaxUnits);
  if (t256 <= t256x128 && t256 <= t128) return kTile256;
  return t256x128 <= t128 ? kTile256x128 : kTile128;
}

}  // namespace

int plan_quantize(const muon_view* x, int32_t transpose, const muon_codes* codes, QuantPlan* p, std::string* err) {
  Span sx, q, scale;
  int rc = check_view("x", x, &sx, err);
  if (rc != MUON_OK) return rc;
  if (transpose != 0 && transpose != 1) return refuse(err, MUON_EINVAL, "transpose must be 0 or 1");
  set_quant(*x, transpose != 0, p);
  if (quant_too_large(*p)) return refuse(err, MUON_EINVAL, "x is too large for codes of its columns");
  if (!codes) return MUON_OK;
  if ((rc = check_codes("codes", codes, transpose ? 0 : -1, &q, &scale, err)) != MUON_OK) return rc;
  if (codes->rows != p->args.rows || codes->cols != p->args.cols)
    return refuse(err, MUON_EINVAL, "codes must be " + std::to_string(p->args.rows) + " x " + std::to_string(p->args.cols));
  if ((rc = check_overlap({q, scale}, {sx}, &p->buf, err)) != MUON_OK) return rc;
  p->args.q = static_cast<int8_t*>(codes->q);
  p->args.scale = codes->scale;
  p->block = codes->block;
  p->empty = scale.empty();
  return MUON_OK;
}

int plan_dequantize(const muon_codes* codes, const muon_view* out, DequantPlan* p, std::string* err) {
  Span q, scale, so;
  int rc = check_codes("codes", codes, -1, &q, &scale, err);
  if (rc != MUON_OK) return rc;
  if ((rc = check_view("out", out, &so, err)) != MUON_OK) return rc;
  if (out->rows != codes->rows || out->cols != codes->cols)
    return refuse(err, MUON_EINVAL, "out must be " + std::to_string(codes->rows) + " x " + std::to_string(codes->cols));
  if ((rc = check_overlap({so}, {q, scale}, nullptr, err)) != MUON_OK) return rc;
  DequantArgs* a = &p->args;
  std::memset(a, 0, sizeof *a);
  a->q = static_cast<const int8_t*>(codes->q);
  a->scale = codes->scale;
  a->out = out->data;
  a->ld = out->rows > 1 ? out->ld : out->cols;
  a->rows = codes->rows;
  a->cols = int32_t(codes->cols);
  a->pitch = int32_t(MUON_CODES_PITCH(codes->cols));
  a->block = codes->block;
  p->bf16 = out->dtype == MUON_BF16;
  p->empty = so.empty();
  return MUON_OK;
}

int plan_int8(const muon_codes* a, const muon_view* x, const muon_codes* b, const muon_view* out, IntPlan* p,
              std::string* err) {
  Span sa, sas, sb, sbs, so;
  int rc = MUON_OK;
  if ((rc = x || !a ? check_view("x", x, &sa, err) : check_codes("a", a, 0, &sa, &sas, err)) != MUON_OK) return rc;
  if (x) sas = {"x", 0, 0, 0, 0};
  if ((rc = check_codes(x ? "w" : "b", b, 0, &sb, &sbs, err)) != MUON_OK) return rc;
  const int64_t rows = x ? x->rows : a->rows, k = x ? x->cols : a->cols;
  if (b->cols != k)
    return refuse(err, MUON_EINVAL, "operands have " + std::to_string(k) + " and " + std::to_string(b->cols) + " columns");
  if (k > kMaxIntSum)
    return refuse(err, MUON_EINVAL, "more than " + std::to_string(kMaxIntSum) + " columns: sums leave 32 bits");
  IntArgs& g = p->args;
  std::memset(&g, 0, sizeof g);
  g.rows = int32_t(rows);
  g.cols = int32_t(b->rows);
  g.k = int32_t(k);
  g.pitch = int32_t(MUON_CODES_PITCH(k));
  g.b = static_cast<const int8_t*>(b->q);
  g.b_scale = b->scale;
  p->empty = g.rows == 0 || g.cols == 0;
  // In the kernel for few rows and in tiles, us: 32 rows of 4096 for 4096 columns 10.6 and 12.8, of 11008 for
  // 4096 25 and 35.5, of 4096 for 11008 19.4 and 16.6; 64 rows 15.2 and 12.8, 36 and 38, 26 and 17.4.
  p->few = g.rows <= kFewRows;
  p->tile = int8_tile(g.rows, g.cols);
  if (p->few ? g.cols > (1 << 26) : ceil_div(g.rows, 128) * ceil_div(g.cols, 128) > (1 << 23))
    return refuse(err, MUON_EINVAL, "the result is too large");
  p->quantise = false;
  p->scale_off = p->buf.ws_bytes = 0;
  if (x) {
    g.x_bf16 = x->dtype == MUON_BF16;
    g.ldx = rows > 1 ? x->ld : x->cols;
    g.x = x->data;
    // Codes made inside the product save a launch (3 us of the host's time), but each of its
    // workgroups of 16 columns reads x: 1 or 2 rows, or 4 MB in all (4 rows of 4096 for 11008 columns,
    // 11 MB, take 18 us that way and 16 in two launches).
    const int64_t codes = int64_t(g.rows) * g.pitch;
    const bool fused = g.rows <= 16 && codes <= 48 * 1024 && (g.rows <= 2 || ceil_div(g.cols, 16) * codes <= (4 << 20));
    p->quantise = !p->empty && !fused;
    g.fused = !p->quantise;
    if (p->quantise) {
      set_quant(*x, false, &p->quant);
      p->scale_off = size_t(round_up(rows * g.pitch, 256));
      p->buf.ws_bytes = p->scale_off + size_t(round_up(rows * 4, 256));
    }
  } else {
    g.a = static_cast<const int8_t*>(a->q);
    g.a_scale = a->scale;
  }
  if (!out) return MUON_OK;
  if ((rc = check_view("out", out, &so, err)) != MUON_OK) return rc;
  if (out->rows != rows || out->cols != b->rows)
    return refuse(err, MUON_EINVAL, "out must be " + std::to_string(rows) + " x " + std::to_string(b->rows));
  if ((rc = check_overlap({so}, {sa, sas, sb, sbs}, &p->buf, err)) != MUON_OK) return rc;
  g.out = out->data;
  g.ldo = rows > 1 ? out->ld : out->cols;
  g.out_bf16 = out->dtype == MUON_BF16;
  return MUON_OK;
}

int plan_wgrad(const muon_view* dy, const muon_codes* x, const muon_view* out, int32_t accumulate, WgradPlan* p,
               std::string* err) {
  Span sd, sq, ss, so;
  int rc = check_view("dy", dy, &sd, err);
  if (rc != MUON_OK) return rc;
  if ((rc = check_codes("x", x, kCodeBlock, &sq, &ss, err)) != MUON_OK) return rc;
  if (dy->rows != x->rows)
    return refuse(err, MUON_EINVAL, "dy has " + std::to_string(dy->rows) + " rows, x " + std::to_string(x->rows));
  WgradArgs& a = p->args;
  std::memset(&a, 0, sizeof a);
  p->bf16 = dy->dtype == MUON_BF16;
  a.dy = dy->data;
  a.lddy = dy->rows > 1 ? dy->ld : dy->cols;
  a.q = static_cast<const int8_t*>(x->q);
  a.scale = x->scale;
  a.tokens = int32_t(dy->rows);
  a.n = int32_t(dy->cols);
  a.k = int32_t(x->cols);
  a.pitch = int32_t(MUON_CODES_PITCH(x->cols));
  a.groups = int32_t(ceil_div(x->cols, kCodeBlock));
  a.n_read = a.n;
  p->empty = a.n == 0 || a.k == 0;
  p->pack = false;
  p->pack_ld = 0;
  p->parts_off = p->buf.ws_bytes = 0;
  p->tile = kTile128;
  a.splits = 1;
  a.piece = std::max(64, int32_t(round_up(a.tokens, 64)));
  if (!p->empty) {
    const int64_t tiles128 = ceil_div(a.n, 128) * ceil_div(a.k, 128), tiles256 = ceil_div(a.n, 256) * ceil_div(a.k, 256);
    if (tiles128 > (1 << 23)) return refuse(err, MUON_EINVAL, "the result is too large");
    // In tiles of 256 x 256 and of 128 x 128, 4096 tokens added to fp32, us: 192 (4096 x 3000 results) 113 and
    // 127, 256 (4096 x 4096) 138 and 167, 384 (6144 x 4096) 223 and 238, 688 (11008 x 4096) 353 and 425.  Just
    // past a round of the compute units the small ones would be faster: 272 (4352 x 4096) 218 and 187.
    if (p->bf16 && tiles256 >= 192) p->tile = kTile256;
    // bf16 rows go to LDS 16 bytes at a time, by 32-bit offsets from the first of 64 tokens.  Others
    // come through registers, in small tiles, or are copied first (517 x 1031 from 777 tokens: 15 us
    // through registers, 20 with the copy).
    constexpr int64_t kMaxStepLd = (1 << 24) - 8;
    if (p->bf16 && (a.n > kMaxStepLd || a.k > kMaxStepLd))
      return refuse(err, MUON_EINVAL, "more than 2^24 - 8 columns of bf16 dy or of x");
    if (p->bf16 && a.tokens > 0 &&
        (reinterpret_cast<uintptr_t>(dy->data) % 16 || a.lddy % 8 || a.n % 8 || a.lddy > kMaxStepLd)) {
      a.through = p->tile == kTile128 && a.n >= 128 && a.lddy <= kMaxStepLd;
      p->pack = !a.through;
    }
    if (p->pack) {
      p->pack_ld = round_up(a.n, 8);
      a.n_read = int32_t(p->pack_ld);
      p->buf.ws_bytes = size_t(round_up(a.tokens * p->pack_ld * 2, 256));
    }
    // Tiles of 256 x 256 keep three quarters of the compute units busy or more, and these draw what power
    // there is: they are not cut (4096 x 3000 results, 16384 tokens: 376 us whole, 430 in 2 pieces).
    if (p->tile != kTile256) a.splits = wgrad_splits(tiles128, a, p->bf16);
    if (a.splits > 1) {
      a.piece = int32_t(round_up(ceil_div(a.tokens, a.splits), 64));
      a.splits = int32_t(ceil_div(a.tokens, a.piece));
    }
    if (a.splits > 1) {
      p->parts_off = p->buf.ws_bytes;
      p->buf.ws_bytes += size_t(a.splits) * size_t(a.n) * size_t(a.k) * 4;
    }
  }
  if (!out) return MUON_OK;
  if ((rc = check_view("out", out, &so, err)) != MUON_OK) return rc;
  if (accumulate != 0 && accumulate != 1) return refuse(err, MUON_EINVAL, "accumulate must be 0 or 1");
  if (out->rows != dy->cols || out->cols != x->cols)
    return refuse(err, MUON_EINVAL, "out must be " + std::to_string(dy->cols) + " x " + std::to_string(x->cols));
  if ((rc = check_overlap({so}, {sd, sq, ss}, &p->buf, err)) != MUON_OK) return rc;
  a.out = out->data;
  a.ldo = out->rows > 1 ? out->ld : out->cols;
  a.out_bf16 = out->dtype == MUON_BF16;
  a.accumulate = accumulate;
  return MUON_OK;
}

int check_linear_workspace(const LinearBuffers& b, const void* workspace, size_t bytes, std::string* err) {
  if (b.ws_bytes == 0) return MUON_OK;
  if (!workspace) return refuse(err, MUON_EINVAL, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return refuse(err, MUON_EINVAL, "workspace is not 256-byte aligned");
  if (bytes < b.ws_bytes)
    return refuse(err, MUON_ENOSPC, "workspace has " + std::to_string(bytes) + " bytes, needs " + std::to_string(b.ws_bytes));
  const Span ws = {"workspace", reinterpret_cast<uintptr_t>(workspace), 1, int64_t(b.ws_bytes), int64_t(b.ws_bytes)};
  for (int i = 0; i < b.count; ++i)
    if (overlap(ws, b.spans[i])) return refuse(err, MUON_EALIAS, std::string("the workspace overlaps ") + b.spans[i].name);
  return MUON_OK;
}

}  // namespace muon

// C ABI entry points of the training operators: validation and launches.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <string>

#include "muon.h"
#include "state.h"
#include "train.h"

namespace {

using namespace muon;

struct Failure {
  muon_status status;
  char msg[200];
};

[[noreturn, gnu::format(printf, 2, 3)]] void refuse(muon_status s, const char *fmt, ...) {
  Failure f{s, {}};
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(f.msg, sizeof f.msg, fmt, ap);
  va_end(ap);
  throw f;
}

// Runs an entry point's body; no exception passes the C boundary.
template <class F>
muon_status entry(F &&body) noexcept {
  State &st = thread_state();
  try {
    body(st);
    st.err.clear();
    return MUON_OK;
  } catch (const Failure &f) {
    try {
      st.err = f.msg;
    } catch (...) {
    }
    return f.status;
  } catch (const std::exception &) {
    return MUON_ERR_HIP;  // host memory
  }
}

void launched(hipError_t e, const char *what) {
  if (e != hipSuccess) refuse(MUON_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
// Pitches for which every offset, in bytes, stays far inside 64 bits.
bool fits(int64_t count, int64_t pitch) { return pitch <= (int64_t(1) << 60) / (count > 1 ? count : 1); }

// A buffer of the call: `rows` runs of `bytes`, `pitch` bytes apart.
struct Span {
  uintptr_t at = 0;
  int64_t rows = 0, bytes = 0, pitch = 0;
  bool written = false;
  const char *name = "";
  uintptr_t end() const { return at + uintptr_t((rows - 1) * pitch + bytes); }
};

// Whether two buffers share a byte. Only asked where their extents meet. With one
// pitch, as the parts of a wide buffer have, the rows' distances are multiples of
// it: the first that brings a's row past the start of b's decides. Else the rows
// of one against the row of the other that each can reach.
bool meet(const Span &a, const Span &b) {
  if (a.rows > 1 && b.rows > 1 && a.pitch == b.pitch) {
    const int64_t d = int64_t(a.at - b.at), over = -a.bytes - d;  // d + k * pitch > -a.bytes
    int64_t k = over / a.pitch - (over % a.pitch < 0 ? 1 : 0) + 1;
    if (k < 1 - b.rows) k = 1 - b.rows;
    return k < a.rows && d + k * a.pitch < b.bytes;
  }
  for (int64_t r = 0; r < a.rows; ++r) {
    const int64_t lo = int64_t(a.at - b.at) + r * a.pitch, hi = lo + a.bytes;  // against b's start
    if (hi <= 0) continue;
    // the last row of b that starts before hi, if it ends after lo
    int64_t q = b.pitch ? (hi - 1) / b.pitch : 0;
    if (q >= b.rows) q = b.rows - 1;
    if (q * b.pitch + b.bytes > lo) return true;
  }
  return false;
}

struct Buffers {
  Span s[16];
  int n = 0;
  void add(const void *p, int64_t rows, int64_t bytes, int64_t pitch, bool written, const char *name) {
    if (!p || rows <= 0 || bytes <= 0) return;
    s[n].at = reinterpret_cast<uintptr_t>(p);
    s[n].rows = rows;
    s[n].bytes = bytes;
    s[n].pitch = rows > 1 ? pitch : bytes;
    s[n].written = written;
    s[n++].name = name;
  }
  // Written buffers meet no other buffer.
  void check() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j) {
        if (!s[i].written && !s[j].written) continue;
        if (s[i].at >= s[j].end() || s[j].at >= s[i].end()) continue;
        const bool small = s[i].rows <= s[j].rows;
        if (meet(small ? s[i] : s[j], small ? s[j] : s[i]))
          refuse(MUON_ERR_ALIAS, "%s and %s overlap", s[j].name, s[i].name);
      }
  }
};

size_t esize(int32_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }

void need(const void *p, const char *name) {
  if (!p) refuse(MUON_ERR_INVALID_ARG, "%s must not be NULL", name);
}

// A matrix operand: dtype, shape, pitch, alignment. Without rows, or as the first
// of none (`none`), it needs no data.
void matrix(const muon_mat *m, const char *name, int64_t max_cols, bool none = false) {
  need(m, name);
  if (m->dtype != MUON_F32 && m->dtype != MUON_BF16) refuse(MUON_ERR_DTYPE, "%s: unknown dtype", name);
  if (m->rows < 0 || m->rows > kMaxIndex || m->cols <= 0 || m->cols > max_cols)
    refuse(MUON_ERR_SHAPE, "%s: rows must lie in [0, 2^31), cols in [1, %lld]", name, (long long)max_cols);
  if (m->ld < m->cols || !fits(m->rows, m->ld)) refuse(MUON_ERR_SHAPE, "%s: ld < cols, or rows * ld > 2^60", name);
  if (m->rows > 0 && !m->data && !none) refuse(MUON_ERR_INVALID_ARG, "%s: NULL data", name);
  if (reinterpret_cast<uintptr_t>(m->data) % esize(m->dtype))
    refuse(MUON_ERR_ALIGN, "%s: data not aligned to its element size", name);
}

void same(const muon_mat *m, const char *name, const muon_mat *as, const char *as_name) {
  if (m->dtype != as->dtype) refuse(MUON_ERR_DTYPE, "%s and %s differ in dtype", name, as_name);
  if (m->rows != as->rows || m->cols != as->cols) refuse(MUON_ERR_SHAPE, "%s and %s differ in shape", name, as_name);
}

void add(Buffers &b, const muon_mat *m, bool written, const char *name) {
  if (m) b.add(m->data, m->rows, m->cols * int64_t(esize(m->dtype)), m->ld * int64_t(esize(m->dtype)), written, name);
}

// A vector of one row per column of x: 1 x cols, any of the two dtypes.
void channel(const muon_mat *m, const char *name, int64_t cols, int32_t *dtype) {
  if (!m) return;
  matrix(m, name, kNormMaxCols);
  if (m->rows != 1 || m->cols != cols) refuse(MUON_ERR_SHAPE, "%s must be 1 x %lld", name, (long long)cols);
  if (*dtype >= 0 && m->dtype != *dtype) refuse(MUON_ERR_DTYPE, "%s: weight, bias and their gradients share one dtype", name);
  *dtype = m->dtype;
}

void aligned4(const void *p, const char *name) {
  if (reinterpret_cast<uintptr_t>(p) % 4) refuse(MUON_ERR_ALIGN, "%s: not aligned to 4 bytes", name);
}

int64_t groups_of(int64_t cols) { return (cols + kCkptGroup - 1) / kCkptGroup; }

CkptView checkpoint(const muon_ckpt *c, const char *name) {
  need(c, name);
  if (c->rows < 0 || c->rows > kMaxIndex || c->cols <= 0 || c->cols > kMaxIndex / 2)
    refuse(MUON_ERR_SHAPE, "%s: rows must lie in [0, 2^31), cols in [1, 2^30)", name);
  if (c->ld_codes < c->cols || c->ld_scales < groups_of(c->cols))
    refuse(MUON_ERR_SHAPE, "%s: ld_codes < cols or ld_scales < ceil(cols / 128)", name);
  if (!fits(c->rows, c->ld_codes) || !fits(c->rows, c->ld_scales))
    refuse(MUON_ERR_SHAPE, "%s: rows * pitch > 2^60", name);
  if (c->rows > 0 && (!c->codes || !c->scales)) refuse(MUON_ERR_INVALID_ARG, "%s: NULL codes or scales", name);
  return CkptView{static_cast<uint8_t *>(c->codes), static_cast<uint8_t *>(c->scales), c->ld_codes, c->ld_scales};
}

void add(Buffers &b, const muon_ckpt *c, bool written) {
  b.add(c->codes, c->rows, c->cols, c->ld_codes, written, "ckpt codes");
  b.add(c->scales, c->rows, groups_of(c->cols), c->ld_scales, written, "ckpt scales");
}

// `bytes` of the thread's workspace, clear of the call's buffers.
char *workspace(const State &st, size_t bytes, Buffers &b) {
  if (!bytes) return nullptr;
  if (!st.ws || st.ws_bytes < bytes)
    refuse(MUON_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu set (muon_set_workspace)", bytes, st.ws_bytes);
  b.add(st.ws, 1, int64_t(bytes), 0, true, "workspace");
  return static_cast<char *>(st.ws);
}

// The weights of the groups: rows x cols of one dtype, stride elements apart.
void weights(Buffers &b, const muon_mat *w, const char *name, int64_t stride, int32_t groups, int32_t dtype, bool written) {
  if (w->rows < 1) refuse(MUON_ERR_SHAPE, "%s: no rows", name);
  if (w->dtype != dtype) refuse(MUON_ERR_DTYPE, "%s: of another dtype than the rows", name);
  const int64_t es = int64_t(esize(dtype)), extent = (w->rows - 1) * w->ld + w->cols;
  if (groups > 1 && stride < extent) refuse(MUON_ERR_SHAPE, "%s: the groups' matrices overlap", name);
  if (groups > 1 && !fits(groups, stride)) refuse(MUON_ERR_SHAPE, "%s: groups * stride > 2^60", name);
  if (groups > 1)
    b.add(w->data, w->ld == w->cols ? groups : 1, (w->ld == w->cols ? extent : (groups - 1) * stride + extent) * es, stride * es,
          written, name);
  else if (groups == 1)
    add(b, w, written, name);
}

// Slots in groups, and the products' sizes.
void slots_of(ProductArgs &a, Buffers &b, int64_t slots, int32_t groups, const int32_t *offsets, const int32_t *rows) {
  if (slots < 0 || slots > kMaxSlots) refuse(MUON_ERR_SHAPE, "slots must lie in [0, 2^31 - 2^22]");
  if (groups < 0 || groups > 65536) refuse(MUON_ERR_INVALID_ARG, "n_groups must lie in [0, 65536]");
  if (groups > 1 && !offsets) refuse(MUON_ERR_INVALID_ARG, "offsets must not be NULL with more than one group");
  aligned4(offsets, "offsets");
  aligned4(rows, "rows");
  b.add(offsets, 1, (int64_t(groups) + 1) * 4, 0, false, "offsets");
  b.add(rows, 1, slots * 4, 0, false, "rows");
  a.slots = slots;
  a.groups = groups;
  a.offsets = offsets;
  a.rows = rows;
}

void sizes(ProductArgs &a, int64_t n, int64_t k) {
  if (n > kMaxIndex / 2 || k > kMaxIndex / 2) refuse(MUON_ERR_SHAPE, "weights: rows and cols must lie below 2^30");
  if (((n + 127) / 128) * (a.slots / 128 + std::min<int64_t>(a.groups, a.slots)) > kMaxIndex)
    refuse(MUON_ERR_SHAPE, "slots * columns too large");
  a.n = int32_t(n);
  a.k = a.x_rows > 0 ? int32_t(k) : 0;  // no row of x: every sum is empty
}

// The workspace of a product, whose kind back, x2 and w2 have been set for, and its check with the call's buffers.
void parts(const State &st, ProductArgs &a, Buffers &b, bool bf16) {
  product_plan(a, bf16);
  a.part = reinterpret_cast<float *>(workspace(st, product_part_bytes(a), b));
  b.check();
}

// What the workspace of a product of these sizes is: weights n x k.
size_t product_workspace(int32_t dtype, int64_t slots, int64_t n, int64_t k, int64_t groups, int32_t backward, bool gated) {
  if (dtype != MUON_F32 && dtype != MUON_BF16) refuse(MUON_ERR_DTYPE, "unknown dtype");
  if (backward != 0 && backward != 1) refuse(MUON_ERR_INVALID_ARG, "backward must be 0 or 1");
  if (groups < 0 || groups > 65536) refuse(MUON_ERR_INVALID_ARG, "groups must lie in [0, 65536]");
  if (n < 1 || k < 1) refuse(MUON_ERR_SHAPE, "n and k must lie in [1, 2^30)");
  ProductArgs a{};
  Buffers b;
  slots_of(a, b, slots, 0, nullptr, nullptr);
  a.groups = int32_t(groups);
  a.x_rows = 1;
  sizes(a, backward ? k : n, backward ? n : k);
  a.back = backward;
  const void *some = &a;  // only whether there is one counts
  a.w2 = gated ? some : nullptr;
  a.x2 = gated && backward ? some : nullptr;
  product_plan(a, dtype == MUON_BF16);
  return product_part_bytes(a);
}

void activation_of(int32_t activation) {
  if (activation != MUON_ACT_SILU && activation != MUON_ACT_GELU)
    refuse(MUON_ERR_INVALID_ARG, "activation must be MUON_ACT_SILU or MUON_ACT_GELU");
}

void expert_product(State &st, const muon_mat *x, const muon_mat *w, int64_t group_stride, int32_t n_groups, int64_t slots,
                    const int32_t *offsets, const int32_t *rows, int32_t gather, int32_t scatter, const muon_mat *y, bool back) {
  matrix(x, "x", kMaxIndex / 2);
  matrix(w, "w", kMaxIndex / 2, n_groups == 0);
  matrix(y, "y", kMaxIndex / 2);
  if (y->dtype != x->dtype) refuse(MUON_ERR_DTYPE, "x and y differ in dtype");
  if (gather < 0) refuse(MUON_ERR_INVALID_ARG, "gather must be >= 0");
  if (scatter != 0 && scatter != 1) refuse(MUON_ERR_INVALID_ARG, "scatter must be 0 or 1");
  ProductArgs a{};
  Buffers b;
  slots_of(a, b, slots, n_groups, offsets, rows);
  if ((gather || scatter) && !rows && slots > 0) refuse(MUON_ERR_INVALID_ARG, "rows must not be NULL with gather or scatter");
  if (!gather && x->rows != slots) refuse(MUON_ERR_SHAPE, "without gather, x has a row for each slot");
  if (!scatter && y->rows != slots) refuse(MUON_ERR_SHAPE, "without scatter, y has a row for each slot");
  if (x->cols != (back ? w->rows : w->cols) || y->cols != (back ? w->cols : w->rows))
    refuse(MUON_ERR_SHAPE, back ? "x's columns are the weights' rows, y's their columns" : "x's columns are the weights' columns, y's their rows");
  a.x_rows = x->rows;
  sizes(a, y->cols, x->cols);
  add(b, x, false, "x");
  weights(b, w, "w", group_stride, n_groups, x->dtype, false);
  add(b, y, true, "y");
  a.back = back;
  parts(st, a, b, x->dtype == MUON_BF16);
  if (n_groups == 0 || slots == 0) return;
  a.x = x->data;
  a.ld_x = x->ld;
  a.w = w->data;
  a.ld_w = w->ld;
  a.w_stride = n_groups > 1 ? group_stride : 0;
  a.gather = gather;
  a.scatter = scatter;
  a.out = y->data;
  a.ld_out = y->ld;
  a.out_rows = y->rows;
  launched(launch_product(a, x->dtype == MUON_BF16, st.stream), "experts' product launch");
}

// What the sum over a token's experts and its backward pass share.
void combine_shape(CombineArgs &a, Buffers &b, int64_t tokens, int64_t cols, int32_t topk, const float *weights,
                   const int32_t *indices, float p, const uint64_t *key) {
  if (topk < 1 || topk > kCombineMaxTopk) refuse(MUON_ERR_INVALID_ARG, "topk must lie in [1, %d]", kCombineMaxTopk);
  if (tokens > kMaxIndex / topk) refuse(MUON_ERR_SHAPE, "tokens * topk must lie below 2^31");
  if (!(p >= 0.f && p < 1.f)) refuse(MUON_ERR_INVALID_ARG, "p must lie in [0, 1)");
  if (p > 0.f) need(key, "key");
  if (reinterpret_cast<uintptr_t>(key) % 8) refuse(MUON_ERR_ALIGN, "key: not aligned to 8 bytes");
  aligned4(weights, "weights");
  aligned4(indices, "indices");
  b.add(weights, 1, tokens * topk * 4, 0, false, "weights");
  b.add(indices, 1, tokens * topk * 4, 0, false, "indices");
  if (p > 0.f) b.add(key, 1, 16, 0, false, "key");
  a.tokens = tokens;
  a.cols = int32_t(cols);
  a.topk = topk;
  a.weights = weights;
  a.indices = indices;
  a.key = p > 0.f ? key : nullptr;
  a.threshold = uint32_t(double(p) * 4294967296.);  // p has 24 bits: below 2^32
  a.scale = float(1. / (1. - double(p)));
}

void combine_forward(State &st, const muon_mat *x, int32_t topk, const float *weights, const int32_t *indices,
                     const muon_mat *residual, float p, const uint64_t *key, const muon_mat *y) {
  matrix(x, "x", kMaxIndex / 2);
  matrix(y, "y", kMaxIndex / 2);
  if (residual) {
    matrix(residual, "residual", kMaxIndex / 2);
    same(residual, "residual", y, "y");
  }
  CombineArgs a{};
  Buffers b;
  combine_shape(a, b, y->rows, y->cols, topk, weights, indices, p, key);
  if (x->dtype != y->dtype) refuse(MUON_ERR_DTYPE, "x and y differ in dtype");
  if (x->rows != y->rows * topk || x->cols != y->cols) refuse(MUON_ERR_SHAPE, "x has topk rows for each row of y");
  add(b, x, false, "x");
  add(b, residual, false, "residual");
  add(b, y, true, "y");
  b.check();
  if (y->rows == 0) return;
  a.x = x->data;
  a.ld_x = x->ld;
  a.res = residual ? residual->data : nullptr;
  a.ld_res = residual ? residual->ld : 0;
  a.out = y->data;
  a.ld_out = y->ld;
  launched(launch_combine_fwd(a, y->dtype == MUON_BF16, st.stream), "combine launch");
}

size_t norm_workspace(int64_t rows, int64_t cols) { return size_t(norm_bwd_blocks(rows, cols)) * 2 * cols * sizeof(float); }

// Offsets of the routing scratch inside the workspace.
struct RouteScratch {
  size_t psum, valid, total;
};
RouteScratch route_scratch(const RouteFwdArgs &a) {
  const size_t table = size_t(a.blocks) * a.experts * 4;
  return {table, 2 * table, a.blocks ? 2 * table + size_t(a.blocks) * 4 : 0};
}

void route_shape(int64_t tokens, int64_t experts, int32_t topk) {
  if (experts < 1 || experts > kRouteMaxExperts)
    refuse(MUON_ERR_SHAPE, "experts must lie in [1, %d]", kRouteMaxExperts);
  if (topk < 1 || topk > kRouteMaxTopk || topk > experts)
    refuse(MUON_ERR_INVALID_ARG, "topk must lie in [1, min(experts, %d)]", kRouteMaxTopk);
  if (tokens < 0 || tokens > kMaxSlots / topk) refuse(MUON_ERR_SHAPE, "tokens * topk must lie in [0, 2^31 - 2^22]");
}

void wgrad_shape(WgradArgs &a, int32_t dtype, int64_t slots, int64_t n, int64_t k, int64_t groups) {
  if (dtype != MUON_F32 && dtype != MUON_BF16) refuse(MUON_ERR_DTYPE, "dy: unknown dtype");
  if (slots < 0 || slots > kMaxSlots || n < 1 || k < 1 || n > kMaxIndex / 2 || k > kMaxIndex / 2)
    refuse(MUON_ERR_SHAPE, "slots must lie in [0, 2^31 - 2^22], n and k in [1, 2^30)");
  if (groups < 0 || groups > 65536) refuse(MUON_ERR_INVALID_ARG, "groups must lie in [0, 65536]");
  if (groups > 0 && ((n + 127) / 128) * ((k + 255) / 256) > kMaxIndex / 512 / groups)
    refuse(MUON_ERR_SHAPE, "groups * n * k too large");
  a.slots = slots;
  a.n = int32_t(n);
  a.k = int32_t(k);
  a.groups = int32_t(groups);
  if (groups > 0) wgrad_plan(a, dtype == MUON_BF16);
}

}  // namespace

extern "C" {

muon_status muon_layernorm_forward(const muon_mat *x, const muon_mat *y, float *mean, float *rstd, const muon_mat *weight,
                                   const muon_mat *bias, float eps, const muon_ckpt *ckpt) {
  return entry([&](State &st) {
    matrix(x, "x", kNormMaxCols);
    matrix(y, "y", kNormMaxCols);
    same(y, "y", x, "x");
    int32_t wt = -1;
    channel(weight, "weight", x->cols, &wt);
    channel(bias, "bias", x->cols, &wt);
    if (!(eps >= 0.f) || !std::isfinite(eps)) refuse(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
    aligned4(mean, "mean");
    aligned4(rstd, "rstd");
    NormFwdArgs a{};
    Buffers b;
    if (ckpt) {
      a.ck = checkpoint(ckpt, "ckpt");
      if (ckpt->rows != x->rows || ckpt->cols != x->cols) refuse(MUON_ERR_SHAPE, "ckpt and x differ in shape");
      add(b, ckpt, true);
    }
    add(b, x, false, "x");
    add(b, y, true, "y");
    add(b, weight, false, "weight");
    add(b, bias, false, "bias");
    b.add(mean, 1, x->rows * 4, 0, true, "mean");
    b.add(rstd, 1, x->rows * 4, 0, true, "rstd");
    b.check();
    if (x->rows == 0) return;
    a.x = x->data;
    a.y = y->data;
    a.w = weight ? weight->data : nullptr;
    a.b = bias ? bias->data : nullptr;
    a.mean = mean;
    a.rstd = rstd;
    a.ld_x = x->ld;
    a.ld_y = y->ld;
    a.rows = x->rows;
    a.cols = int32_t(x->cols);
    a.w_f32 = wt == MUON_F32;
    a.eps = eps;
    a.inv_cols = 1. / double(a.cols);
    launched(launch_norm_fwd(a, x->dtype == MUON_BF16, st.stream), "layer norm launch");
  });
}

muon_status muon_layernorm_workspace_size(int64_t rows, int64_t cols, size_t *bytes) {
  return entry([&](State &) {
    need(bytes, "bytes");
    if (rows < 0 || rows > kMaxIndex || cols < 1 || cols > kNormMaxCols)
      refuse(MUON_ERR_SHAPE, "rows must lie in [0, 2^31), cols in [1, %d]", kNormMaxCols);
    *bytes = norm_workspace(rows, cols);
  });
}

muon_status muon_layernorm_backward(const muon_mat *dy, const muon_mat *x, const float *mean, const float *rstd,
                                    const muon_mat *dx, const muon_mat *weight, const muon_mat *dweight,
                                    const muon_mat *dbias) {
  return entry([&](State &st) {
    matrix(dy, "dy", kNormMaxCols);
    matrix(x, "x", kNormMaxCols);
    matrix(dx, "dx", kNormMaxCols);
    same(x, "x", dy, "dy");
    same(dx, "dx", dy, "dy");
    int32_t wt = -1;
    channel(weight, "weight", x->cols, &wt);
    channel(dweight, "dweight", x->cols, &wt);
    channel(dbias, "dbias", x->cols, &wt);
    if (x->rows > 0) {
      need(mean, "mean");
      need(rstd, "rstd");
    }
    aligned4(mean, "mean");
    aligned4(rstd, "rstd");
    Buffers b;
    add(b, dy, false, "dy");
    add(b, x, false, "x");
    b.add(mean, 1, x->rows * 4, 0, false, "mean");
    b.add(rstd, 1, x->rows * 4, 0, false, "rstd");
    add(b, dx, true, "dx");
    add(b, weight, false, "weight");
    add(b, dweight, true, "dweight");
    add(b, dbias, true, "dbias");
    NormBwdArgs a{};
    a.blocks = norm_bwd_blocks(x->rows, x->cols);
    const bool sums = dweight || dbias;
    // with no rows the sums are empty: the second launch writes zeros
    char *ws = sums && a.blocks ? workspace(st, norm_workspace(x->rows, x->cols), b) : nullptr;
    b.check();
    if (x->rows == 0 && !sums) return;
    a.dy = dy->data;
    a.x = x->data;
    a.w = weight ? weight->data : nullptr;
    a.mean = mean;
    a.rstd = rstd;
    a.dx = dx->data;
    a.dw = dweight ? dweight->data : nullptr;
    a.db = dbias ? dbias->data : nullptr;
    a.part = reinterpret_cast<float *>(ws);
    a.sums = sums;
    a.ld_dy = dy->ld;
    a.ld_x = x->ld;
    a.ld_dx = dx->ld;
    a.rows = x->rows;
    a.cols = int32_t(x->cols);
    a.w_f32 = wt == MUON_F32;
    launched(launch_norm_bwd(a, x->dtype == MUON_BF16, st.stream), "layer norm backward launch");
  });
}

muon_status muon_ckpt_save(const muon_mat *x, const muon_ckpt *ckpt) {
  return entry([&](State &st) {
    matrix(x, "x", kMaxIndex / 2);
    CkptArgs a{};
    a.ck = checkpoint(ckpt, "ckpt");
    if (ckpt->rows != x->rows || ckpt->cols != x->cols) refuse(MUON_ERR_SHAPE, "ckpt and x differ in shape");
    Buffers b;
    add(b, x, false, "x");
    add(b, ckpt, true);
    b.check();
    a.in = x->data;
    a.ld = x->ld;
    a.rows = x->rows;
    a.cols = int32_t(x->cols);
    launched(launch_ckpt_save(a, x->dtype == MUON_BF16, st.stream), "checkpoint save launch");
  });
}

muon_status muon_ckpt_load(const muon_ckpt *ckpt, const muon_mat *out) {
  return entry([&](State &st) {
    matrix(out, "out", kMaxIndex / 2);
    CkptArgs a{};
    a.ck = checkpoint(ckpt, "ckpt");
    if (ckpt->rows != out->rows || ckpt->cols != out->cols) refuse(MUON_ERR_SHAPE, "ckpt and out differ in shape");
    Buffers b;
    add(b, out, true, "out");
    add(b, ckpt, false);
    b.check();
    a.out = out->data;
    a.ld = out->ld;
    a.rows = out->rows;
    a.cols = int32_t(out->cols);
    launched(launch_ckpt_load(a, out->dtype == MUON_BF16, st.stream), "checkpoint load launch");
  });
}

muon_status muon_ckpt_weight_grad_workspace_size(int32_t dtype, int64_t slots, int64_t n, int64_t k, int64_t groups,
                                                 size_t *bytes) {
  return entry([&](State &) {
    need(bytes, "bytes");
    WgradArgs a{};
    wgrad_shape(a, dtype, slots, n, k, groups);
    *bytes = groups > 0 ? wgrad_part_bytes(a) + wgrad_order_bytes(a) : 0;
  });
}

muon_status muon_ckpt_weight_grad(const muon_mat *dy, const muon_ckpt *x, const muon_mat *grads, int64_t group_stride,
                                  int32_t n_groups, const int32_t *offsets, const int32_t *rows,
                                  int32_t rows_per_token) {
  return entry([&](State &st) {
    matrix(dy, "dy", kMaxIndex / 2);
    WgradArgs a{};
    a.x = checkpoint(x, "x");
    matrix(grads, "grads", kMaxIndex / 2, n_groups == 0);
    if (grads->rows < 1) refuse(MUON_ERR_SHAPE, "grads: no rows");
    if (grads->dtype != dy->dtype) refuse(MUON_ERR_DTYPE, "dy and grads differ in dtype");
    if (grads->rows != dy->cols || grads->cols != x->cols) refuse(MUON_ERR_SHAPE, "a gradient is dy's columns x x's columns");
    wgrad_shape(a, dy->dtype, dy->rows, dy->cols, x->cols, n_groups);
    if (n_groups > 1 && group_stride < (grads->rows - 1) * grads->ld + grads->cols)
      refuse(MUON_ERR_SHAPE, "group_stride: gradients overlap");
    if (n_groups > 1 && !fits(n_groups, group_stride)) refuse(MUON_ERR_SHAPE, "group_stride: n_groups * group_stride > 2^60");
    if (n_groups > 1 && !offsets) refuse(MUON_ERR_INVALID_ARG, "offsets must not be NULL with more than one group");
    if (x->ld_codes > kMaxIndex || x->ld_scales > kMaxIndex) refuse(MUON_ERR_SHAPE, "x: pitches must lie below 2^31");
    if (rows_per_token < 1) refuse(MUON_ERR_INVALID_ARG, "rows_per_token must be >= 1");
    if (!rows && dy->rows > x->rows * int64_t(rows_per_token))
      refuse(MUON_ERR_SHAPE, "without rows, dy has at most rows_per_token rows for each row of x");
    aligned4(offsets, "offsets");
    aligned4(rows, "rows");
    Buffers b;
    add(b, dy, false, "dy");
    add(b, x, false);
    const int64_t es = int64_t(esize(grads->dtype));
    const int64_t extent = ((grads->rows - 1) * grads->ld + grads->cols) * es;
    if (grads->ld == grads->cols)
      b.add(grads->data, n_groups, extent, group_stride * es, true, "grads");
    else  // rows of the one matrix, or (several groups) everything from the first byte to the last
      n_groups == 1 ? add(b, grads, true, "grads")
                    : b.add(grads->data, 1, (n_groups - 1) * group_stride * es + extent, 0, true, "grads");
    b.add(offsets, 1, (int64_t(n_groups) + 1) * 4, 0, false, "offsets");
    b.add(rows, 1, dy->rows * 4, 0, false, "rows");
    const size_t parts = n_groups > 0 ? wgrad_part_bytes(a) : 0, order = n_groups > 0 ? wgrad_order_bytes(a) : 0;
    char *ws = workspace(st, parts + order, b);
    b.check();
    if (n_groups == 0) return;
    a.dy = dy->data;
    a.ld_dy = dy->ld;
    a.tokens = x->rows;
    a.offsets = offsets;
    a.rows = rows;
    a.per_token = rows_per_token;
    a.out = grads->data;
    a.ld_out = grads->ld;
    a.stride = group_stride;
    a.part = reinterpret_cast<float *>(ws);
    a.order = order ? reinterpret_cast<int4 *>(ws) : nullptr;
    launched(launch_wgrad(a, dy->dtype == MUON_BF16, st.stream), "weight gradient launch");
  });
}

muon_status muon_route_workspace_size(int64_t tokens, int64_t experts, int32_t topk, size_t *bytes) {
  return entry([&](State &) {
    need(bytes, "bytes");
    route_shape(tokens, experts, topk);
    RouteFwdArgs a{};
    a.tokens = int32_t(tokens);
    a.experts = int32_t(experts);
    a.topk = topk;
    route_plan(a);
    *bytes = route_scratch(a).total;
  });
}

muon_status muon_route_forward(const muon_mat *logits, int32_t topk, int32_t renormalize, float alpha, int32_t *indices,
                               float *weights, int32_t *counts, int32_t *offsets, int32_t *rows, float *loss) {
  return entry([&](State &st) {
    matrix(logits, "logits", kRouteMaxExperts);
    route_shape(logits->rows, logits->cols, topk);
    if (renormalize != 0 && renormalize != 1) refuse(MUON_ERR_INVALID_ARG, "renormalize must be 0 or 1");
    if (!std::isfinite(alpha)) refuse(MUON_ERR_INVALID_ARG, "alpha must be finite");
    if (logits->rows > 0) {
      need(indices, "indices");
      need(weights, "weights");
      need(rows, "rows");
    }
    need(counts, "counts");
    need(offsets, "offsets");
    need(loss, "loss");
    RouteFwdArgs a{};
    a.logits = logits->data;
    a.ld = logits->ld;
    a.tokens = int32_t(logits->rows);
    a.experts = int32_t(logits->cols);
    a.topk = topk;
    a.renorm = renormalize;
    a.alpha = alpha;
    a.indices = indices;
    a.weights = weights;
    a.counts = counts;
    a.offsets = offsets;
    a.rows = rows;
    a.loss = loss;
    route_plan(a);
    const void *outs[6] = {indices, weights, counts, offsets, rows, loss};
    const char *names[6] = {"indices", "weights", "counts", "offsets", "rows", "loss"};
    const int64_t slots = int64_t(a.tokens) * topk, table = int64_t(a.experts) + 1;
    const int64_t len[6] = {slots, slots, table, table, slots, 1};
    Buffers b;
    add(b, logits, false, "logits");
    for (int i = 0; i < 6; ++i) {
      aligned4(outs[i], names[i]);
      b.add(outs[i], 1, len[i] * 4, 0, true, names[i]);
    }
    const RouteScratch sc = route_scratch(a);
    char *ws = workspace(st, sc.total, b);
    b.check();
    if (ws) {
      a.hist = reinterpret_cast<int32_t *>(ws);
      a.psum = reinterpret_cast<float *>(ws + sc.psum);
      a.valid = reinterpret_cast<int32_t *>(ws + sc.valid);
    }
    launched(launch_route_fwd(a, logits->dtype == MUON_BF16, st.stream), "routing launch");
  });
}

muon_status muon_route_backward(const muon_mat *logits, int32_t topk, int32_t renormalize, float alpha,
                                const int32_t *indices, const int32_t *counts, const float *dweights,
                                const float *dloss, const muon_mat *dlogits) {
  return entry([&](State &st) {
    matrix(logits, "logits", kRouteMaxExperts);
    matrix(dlogits, "dlogits", kRouteMaxExperts);
    same(dlogits, "dlogits", logits, "logits");
    route_shape(logits->rows, logits->cols, topk);
    if (renormalize != 0 && renormalize != 1) refuse(MUON_ERR_INVALID_ARG, "renormalize must be 0 or 1");
    if (!std::isfinite(alpha)) refuse(MUON_ERR_INVALID_ARG, "alpha must be finite");
    if (logits->rows > 0) {
      if (dweights) need(indices, "indices");
      need(counts, "counts");
    }
    aligned4(indices, "indices");
    aligned4(counts, "counts");
    aligned4(dweights, "dweights");
    aligned4(dloss, "dloss");
    const int64_t slots = logits->rows * topk;
    Buffers b;
    add(b, logits, false, "logits");
    add(b, dlogits, true, "dlogits");
    b.add(indices, 1, slots * 4, 0, false, "indices");
    b.add(counts, 1, (logits->cols + 1) * 4, 0, false, "counts");
    b.add(dweights, 1, slots * 4, 0, false, "dweights");
    b.add(dloss, 1, 4, 0, false, "dloss");
    b.check();
    RouteBwdArgs a{};
    a.logits = logits->data;
    a.ld = logits->ld;
    a.tokens = int32_t(logits->rows);
    a.experts = int32_t(logits->cols);
    a.topk = topk;
    a.renorm = renormalize;
    a.alpha = alpha;
    a.indices = indices;
    a.counts = counts;
    a.dweights = dweights;
    a.dloss = dloss;
    a.dlogits = dlogits->data;
    a.ld_out = dlogits->ld;
    launched(launch_route_bwd(a, logits->dtype == MUON_BF16, st.stream), "routing backward launch");
  });
}

muon_status muon_gated_forward(const muon_mat *x, const muon_mat *wgate, int64_t gate_stride, const muon_mat *wup,
                               int64_t up_stride, int32_t n_groups, const int32_t *offsets, const int32_t *rows,
                               int32_t rows_per_token, int32_t activation, const muon_mat *h, const muon_mat *gate,
                               const muon_mat *up) {
  return entry([&](State &st) {
    matrix(x, "x", kMaxIndex / 2);
    matrix(wgate, "wgate", kMaxIndex / 2, n_groups == 0);
    matrix(wup, "wup", kMaxIndex / 2, n_groups == 0);
    matrix(h, "h", kMaxIndex / 2);
    const muon_mat *saved[2] = {gate, up};
    const char *names[2] = {"gate", "up"};
    if (h->dtype != x->dtype) refuse(MUON_ERR_DTYPE, "x and h differ in dtype");
    for (int i = 0; i < 2; ++i)
      if (saved[i]) {
        matrix(saved[i], names[i], kMaxIndex / 2);
        same(saved[i], names[i], h, "h");
      }
    same(wup, "wup", wgate, "wgate");
    activation_of(activation);
    if (rows_per_token < 1) refuse(MUON_ERR_INVALID_ARG, "rows_per_token must be >= 1");
    ProductArgs a{};
    Buffers b;
    slots_of(a, b, h->rows, n_groups, offsets, rows);
    if (wgate->cols != x->cols || wgate->rows != h->cols) refuse(MUON_ERR_SHAPE, "weights are h's columns x x's columns");
    if (!rows && h->rows > x->rows * int64_t(rows_per_token))
      refuse(MUON_ERR_SHAPE, "without rows, h has at most rows_per_token rows for each row of x");
    a.x_rows = x->rows;
    sizes(a, h->cols, x->cols);
    add(b, x, false, "x");
    weights(b, wgate, "wgate", gate_stride, n_groups, x->dtype, false);
    weights(b, wup, "wup", up_stride, n_groups, x->dtype, false);
    add(b, h, true, "h");
    add(b, gate, true, "gate");
    add(b, up, true, "up");
    a.w2 = wup->data;
    parts(st, a, b, x->dtype == MUON_BF16);
    if (n_groups == 0 || h->rows == 0) return;
    a.x = x->data;
    a.ld_x = x->ld;
    a.w = wgate->data;
    a.ld_w = wgate->ld;
    a.w_stride = n_groups > 1 ? gate_stride : 0;
    a.ld_w2 = wup->ld;
    a.w2_stride = n_groups > 1 ? up_stride : 0;
    a.gather = rows || rows_per_token > 1 ? rows_per_token : 0;
    a.act = activation;
    a.out = h->data;
    a.ld_out = h->ld;
    a.gate = gate ? gate->data : nullptr;
    a.ld_gate = gate ? gate->ld : 0;
    a.up = up ? up->data : nullptr;
    a.ld_up = up ? up->ld : 0;
    launched(launch_product(a, x->dtype == MUON_BF16, st.stream), "gated block launch");
  });
}

muon_status muon_gated_backward(const muon_mat *dh, const muon_mat *gate, const muon_mat *up, const muon_mat *wgate,
                                int64_t gate_stride, const muon_mat *wup, int64_t up_stride, int32_t n_groups,
                                const int32_t *offsets, const int32_t *rows, int32_t activation, const muon_mat *dgate,
                                const muon_mat *dup, const muon_mat *dx) {
  return entry([&](State &st) {
    const muon_mat *like[5] = {dh, gate, up, dgate, dup};
    const char *names[5] = {"dh", "gate", "up", "dgate", "dup"};
    Buffers b;
    for (int i = 0; i < 5; ++i) {
      matrix(like[i], names[i], kMaxIndex / 2);
      if (i) same(like[i], names[i], dh, "dh");
      add(b, like[i], i >= 3, names[i]);
    }
    activation_of(activation);
    ProductArgs a{};
    slots_of(a, b, dh->rows, n_groups, offsets, rows);
    if (dx) {
      matrix(wgate, "wgate", kMaxIndex / 2, n_groups == 0);
      matrix(wup, "wup", kMaxIndex / 2, n_groups == 0);
      matrix(dx, "dx", kMaxIndex / 2);
      same(wup, "wup", wgate, "wgate");
      if (dx->dtype != dh->dtype) refuse(MUON_ERR_DTYPE, "dh and dx differ in dtype");
      if (wgate->rows != dh->cols || wgate->cols != dx->cols) refuse(MUON_ERR_SHAPE, "weights are dh's columns x dx's columns");
      if (!rows && dh->rows > 0 && dx->rows != dh->rows) refuse(MUON_ERR_SHAPE, "without rows, dx has a row for each slot");
      a.x_rows = dh->rows;
      sizes(a, dx->cols, dh->cols);
      weights(b, wgate, "wgate", gate_stride, n_groups, dh->dtype, false);
      weights(b, wup, "wup", up_stride, n_groups, dh->dtype, false);
      add(b, dx, true, "dx");
      a.back = 1;
      a.x2 = dup->data;
      a.w2 = wup->data;
    }
    const bool bf16 = dh->dtype == MUON_BF16;
    if (dx)
      parts(st, a, b, bf16);
    else
      b.check();
    if (n_groups == 0 || dh->rows == 0) return;
    GatedGradArgs g{};
    g.dh = dh->data;
    g.ld_dh = dh->ld;
    g.gate = gate->data;
    g.ld_gate = gate->ld;
    g.up = up->data;
    g.ld_up = up->ld;
    g.dgate = dgate->data;
    g.ld_dgate = dgate->ld;
    g.dup = dup->data;
    g.ld_dup = dup->ld;
    g.offsets = offsets;
    g.slots = dh->rows;
    g.groups = n_groups;
    g.n = int32_t(dh->cols);
    g.act = activation;
    launched(launch_gated_grad(g, bf16, st.stream), "gated block's gradients launch");
    if (!dx) return;
    a.x = dgate->data;
    a.ld_x = dgate->ld;
    a.ld_x2 = dup->ld;
    a.w = wgate->data;
    a.ld_w = wgate->ld;
    a.w_stride = n_groups > 1 ? gate_stride : 0;
    a.ld_w2 = wup->ld;
    a.w2_stride = n_groups > 1 ? up_stride : 0;
    a.scatter = rows != nullptr;
    a.out = dx->data;
    a.ld_out = dx->ld;
    a.out_rows = dx->rows;
    launched(launch_product(a, bf16, st.stream), "gated block's backward launch");
  });
}

muon_status muon_expert_forward(const muon_mat *x, const muon_mat *w, int64_t group_stride, int32_t n_groups, int64_t slots,
                                const int32_t *offsets, const int32_t *rows, int32_t gather, int32_t scatter,
                                const muon_mat *y) {
  return entry([&](State &st) { expert_product(st, x, w, group_stride, n_groups, slots, offsets, rows, gather, scatter, y, false); });
}

muon_status muon_expert_backward(const muon_mat *dy, const muon_mat *w, int64_t group_stride, int32_t n_groups, int64_t slots,
                                 const int32_t *offsets, const int32_t *rows, int32_t gather, int32_t scatter,
                                 const muon_mat *dx) {
  return entry([&](State &st) { expert_product(st, dy, w, group_stride, n_groups, slots, offsets, rows, gather, scatter, dx, true); });
}

muon_status muon_gated_workspace_size(int32_t dtype, int64_t slots, int64_t n, int64_t k, int64_t groups, int32_t backward,
                                      size_t *bytes) {
  return entry([&](State &) {
    need(bytes, "bytes");
    *bytes = product_workspace(dtype, slots, n, k, groups, backward, true);
  });
}

muon_status muon_expert_workspace_size(int32_t dtype, int64_t slots, int64_t n, int64_t k, int64_t groups, int32_t backward,
                                       size_t *bytes) {
  return entry([&](State &) {
    need(bytes, "bytes");
    *bytes = product_workspace(dtype, slots, n, k, groups, backward, false);
  });
}

muon_status muon_combine_forward(const muon_mat *x, int32_t topk, const float *weights, const int32_t *indices,
                                 const muon_mat *residual, float p, const uint64_t *key, const muon_mat *y) {
  return entry([&](State &st) { combine_forward(st, x, topk, weights, indices, residual, p, key, y); });
}

muon_status muon_combine_workspace_size(int64_t tokens, int32_t topk, size_t *bytes) {
  return entry([&](State &) {
    need(bytes, "bytes");
    if (topk < 1 || topk > kCombineMaxTopk) refuse(MUON_ERR_INVALID_ARG, "topk must lie in [1, %d]", kCombineMaxTopk);
    if (tokens < 0 || tokens > kMaxIndex / topk) refuse(MUON_ERR_SHAPE, "tokens * topk must lie in [0, 2^31)");
    *bytes = size_t(tokens) * size_t(topk) * 4;
  });
}

muon_status muon_combine_backward(const muon_mat *dy, const muon_mat *x, int32_t topk, const float *weights,
                                  const int32_t *indices, const int32_t *rows, float p, const uint64_t *key,
                                  const muon_mat *dx, float *dweights) {
  return entry([&](State &st) {
    matrix(dy, "dy", kMaxIndex / 2);
    matrix(dx, "dx", kMaxIndex / 2);
    CombineArgs a{};
    Buffers b;
    combine_shape(a, b, dy->rows, dy->cols, topk, weights, indices, p, key);
    if (dx->dtype != dy->dtype) refuse(MUON_ERR_DTYPE, "dy and dx differ in dtype");
    if (dx->rows != dy->rows * topk || dx->cols != dy->cols) refuse(MUON_ERR_SHAPE, "dx has topk rows for each row of dy");
    if (dweights) {
      matrix(x, "x", kMaxIndex / 2);
      same(x, "x", dx, "dx");
      add(b, x, false, "x");
    }
    aligned4(rows, "rows");
    aligned4(dweights, "dweights");
    add(b, dy, false, "dy");
    add(b, dx, true, "dx");
    b.add(rows, 1, dx->rows * 4, 0, false, "rows");
    b.add(dweights, 1, dx->rows * 4, 0, true, "dweights");
    char *ws = rows ? workspace(st, size_t(dx->rows) * 4, b) : nullptr;
    b.check();
    if (dy->rows == 0) return;
    a.dy = dy->data;
    a.ld_dy = dy->ld;
    a.x = dweights ? x->data : nullptr;
    a.ld_x = dweights ? x->ld : 0;
    a.out = dx->data;
    a.ld_out = dx->ld;
    a.rows = rows;
    a.places = reinterpret_cast<int32_t *>(ws);
    a.dweights = dweights;
    launched(launch_combine_bwd(a, dy->dtype == MUON_BF16, st.stream), "combine backward launch");
  });
}

muon_status muon_dropout_forward(const muon_mat *x, const muon_mat *residual, float p, const uint64_t *key, const muon_mat *y) {
  return entry([&](State &st) { combine_forward(st, x, 1, nullptr, nullptr, residual, p, key, y); });
}

muon_status muon_dropout_backward(const muon_mat *dy, float p, const uint64_t *key, const muon_mat *dx) {
  return entry([&](State &st) { combine_forward(st, dy, 1, nullptr, nullptr, nullptr, p, key, dx); });
}

}  // extern "C"

// C entry points of the feed-forward operators (residual_norm, linear, glu and
// their gradients): validation, workspace layout and launches. Everything is
// checked on the host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "hc_ffn.h"
#include "hc_internal.h"
#include "hc_plan.h"
#include "hc_status.h"

namespace {

using hc::fail;
using hc::ok;
using hc::Range;

size_t elem_size(int dtype) { return dtype == HCLRMIX_F32 ? 4 : 2; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// A row kernel's grid times its threads stays below 2^32.
constexpr int64_t MAX_ROWS = HCLRMIX_MAX_ROWS;

hclrmix_status check_dtype(int dtype) {
  if (dtype == HCLRMIX_F32 || dtype == HCLRMIX_F16 || dtype == HCLRMIX_BF16) return HCLRMIX_OK;
  return fail(HCLRMIX_ERR_UNSUPPORTED, "unknown dtype %d", dtype);
}

// One tensor of a call: bytes it spans (0: not given).
Range span(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride, size_t es) {
  Range r{name, (uintptr_t)p, (uintptr_t)p};
  if (p && rows > 0) r.hi += ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * es;
  return r;
}

// Element alignment of every tensor, and outputs against everything else.
hclrmix_status check_tensors(std::initializer_list<Range> in, std::initializer_list<Range> out, size_t es) {
  for (const Range& r : in)
    if (r.lo % es) return fail(HCLRMIX_ERR_UNSUPPORTED, "%s must be element-aligned", r.name);
  for (const Range& o : out) {
    if (o.lo % es) return fail(HCLRMIX_ERR_UNSUPPORTED, "%s must be element-aligned", o.name);
    for (const Range& i : in)
      if (overlaps(o, i)) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "%s overlaps %s", o.name, i.name);
    for (const Range& p : out)
      if (&p != &o && overlaps(o, p)) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "%s overlaps %s", o.name, p.name);
  }
  return HCLRMIX_OK;
}

hclrmix_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return HCLRMIX_OK;
  if (!ws || bytes < need) return fail(HCLRMIX_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes, got %zu", need, bytes);
  if ((uintptr_t)ws & 15u) return fail(HCLRMIX_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  return HCLRMIX_OK;
}

hclrmix_status done(hipError_t e) {
  return e == hipSuccess ? ok() : fail(HCLRMIX_ERR_DEVICE, "HIP error: %s", hipGetErrorString(e));
}

bool all16(std::initializer_list<const void*> ps) {
  uintptr_t x = 0;
  for (const void* p : ps) x |= (uintptr_t)p;
  return (x & 15u) == 0;
}

// ------------------------------------------------------------------ norms

hclrmix_status check_norm(const hclrmix_norm_problem* p) {
  if (!p) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "problem must not be NULL");
  if (p->reserved != 0) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "problem.reserved must be 0");
  if (hclrmix_status st = check_dtype(p->dtype)) return st;
  if (p->rows < 0 || p->hidden < 1) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "rows must be >= 0 and hidden >= 1");
  if (p->hidden > HCLRMIX_NORM_MAX_HIDDEN || p->rows > MAX_ROWS)
    return fail(HCLRMIX_ERR_UNSUPPORTED, "at most %d rows of %d elements", (int)MAX_ROWS, HCLRMIX_NORM_MAX_HIDDEN);
  if (p->gate < HCLRMIX_GATE_NONE || p->gate > HCLRMIX_GATE_ELEMENT)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "unknown gate %d", (int)p->gate);
  if (p->gate == HCLRMIX_GATE_ROW ? p->gate_stride < 0 : p->gate_stride != 0)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "gate_stride %lld does not fit the gate", (long long)p->gate_stride);
  if (p->gate_stride > HCLRMIX_PRODUCT_MAX_WIDTH)
    return fail(HCLRMIX_ERR_UNSUPPORTED, "gate_stride above %d", HCLRMIX_PRODUCT_MAX_WIDTH);
  if (p->post_norm != 0 && p->post_norm != 1)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "post_norm must be 0 or 1");
  if (!std::isfinite(p->alpha) || !std::isfinite(p->epsilon) || p->epsilon < 0.0f)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "alpha must be finite and epsilon finite and >= 0");
  return HCLRMIX_OK;
}

hc::NormArgs norm_args(const hclrmix_norm_problem* p) {
  hc::NormArgs a{};
  a.rows = p->rows;
  a.hidden = (int)p->hidden;
  a.gate_kind = p->gate;
  a.gate_stride = p->gate_stride ? p->gate_stride : 1;
  a.post_norm = p->post_norm;
  a.alpha = p->alpha;
  a.eps = p->epsilon;
  return a;
}

Range gate_span(const char* name, const void* gate, const hclrmix_norm_problem* p, size_t es) {
  if (p->gate == HCLRMIX_GATE_ELEMENT) return span(name, gate, p->rows, p->hidden, p->hidden, es);
  return span(name, gate, p->rows, 1, p->gate_stride ? p->gate_stride : 1, es);
}

size_t norm_workspace(const hclrmix_norm_problem* p) {
  return HCLRMIX_COUNTER_BYTES + up256((size_t)hc::norm_backward_most_groups(p->rows, p->hidden) * 2 * (size_t)p->hidden * 4);
}

// ------------------------------------------------------------------ products

struct Strides {
  int64_t x, w, r;
};

hclrmix_status check_product(const hclrmix_product* p, bool linear, Strides* s) {
  if (!p) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "problem must not be NULL");
  if (p->reserved[0] != 0 || p->reserved[1] != 0)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "problem.reserved must be 0");
  if (hclrmix_status st = check_dtype(p->dtype)) return st;
  if (p->rows < 0 || p->in < 1 || p->out < 1)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "rows must be >= 0, in and out >= 1");
  if (p->activation < HCLRMIX_ACT_NONE || p->activation > HCLRMIX_ACT_SIGMOID)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "unknown activation %d", (int)p->activation);
  if (!linear && p->activation == HCLRMIX_ACT_NONE)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "a gated product needs an activation");
  if (p->in > HCLRMIX_PRODUCT_MAX_WIDTH || p->out > HCLRMIX_PRODUCT_MAX_WIDTH || p->rows > MAX_ROWS)
    return fail(HCLRMIX_ERR_UNSUPPORTED, "at most %d rows, in and out at most %d", (int)MAX_ROWS,
                HCLRMIX_PRODUCT_MAX_WIDTH);
  s->x = p->x_stride ? p->x_stride : p->in;
  s->w = p->weight_stride ? p->weight_stride : p->out;
  s->r = p->residual_stride ? p->residual_stride : p->out;
  if (s->x < p->in || s->w < p->out || s->r < p->out)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "a stride is shorter than its row");
  if (s->x > HCLRMIX_PRODUCT_MAX_WIDTH || s->w > HCLRMIX_PRODUCT_MAX_WIDTH || s->r > HCLRMIX_PRODUCT_MAX_WIDTH)
    return fail(HCLRMIX_ERR_UNSUPPORTED, "strides are at most %d", HCLRMIX_PRODUCT_MAX_WIDTH);
  // Tile counts of every product stay inside a launch's grid, and byte counts
  // of every matrix inside 34 bits.
  const int64_t wide = p->out > p->in ? p->out : p->in;
  if (p->rows * wide > (int64_t(1) << 32) || p->in * p->out > (int64_t(1) << 32))
    return fail(HCLRMIX_ERR_UNSUPPORTED, "rows x max(in, out) and in x out are at most 2^32");
  return HCLRMIX_OK;
}

// Workspace: the counters, the split sums of the largest of the call's products,
// and for a backward pass the pre-activation gradients and the column sums.
struct ProductWorkspace {
  size_t scratch, dz0, dz1, sums, bytes;
};

ProductWorkspace forward_workspace(const hclrmix_product* p, bool glu) {
  ProductWorkspace w{};
  w.scratch = HCLRMIX_COUNTER_BYTES;
  w.bytes = w.scratch + up256(hc::product_scratch(p->dtype, p->rows, p->out, p->in, false, glu, 1, 1));
  return w;
}

ProductWorkspace backward_workspace(const hclrmix_product* p, bool glu) {
  ProductWorkspace w{};
  w.scratch = HCLRMIX_COUNTER_BYTES;
  const int two = glu ? 2 : 1;
  const size_t dx = hc::product_scratch(p->dtype, p->rows, p->in, p->out, false, false, two, 1);
  const size_t dw = hc::product_scratch(p->dtype, p->in, p->out, p->rows, true, false, 1, two);
  size_t off = w.scratch + up256(p->rows == 0 ? 0 : dx > dw ? dx : dw);
  const size_t dz = up256((size_t)p->rows * (size_t)p->out * elem_size(p->dtype));
  w.dz0 = off;
  if (glu || p->activation != HCLRMIX_ACT_NONE) off += dz;
  w.dz1 = off;
  if (glu) off += dz;
  w.sums = off;
  off += up256((size_t)hc::grad_groups(p->rows) * two * (size_t)p->out * 4);
  w.bytes = off;
  return w;
}

hclrmix_status size_of(const hclrmix_product* p, size_t* bytes, bool glu, bool backward) {
  Strides s;
  if (hclrmix_status st = check_product(p, !glu, &s)) return st;
  if (!bytes) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  *bytes = (backward ? backward_workspace(p, glu) : forward_workspace(p, glu)).bytes;
  return ok();
}

hc::Product base_product() {
  hc::Product r{};
  r.segments = r.batch = 1;
  r.act = hc::ACT_NONE;
  return r;
}

// dx = dz0 w0^T (+ dz1 w1^T).
hc::Product dx_product(const hclrmix_product* p, const Strides& s, const void* dz0, const void* dz1, const void* w0,
                       const void* w1, void* dx) {
  hc::Product r = base_product();
  r.p[0] = dz0;
  r.p[1] = dz1;
  r.q[0] = w0;
  r.q[1] = w1;
  r.ldp = p->out;
  r.ldq = s.w;
  r.M = p->rows;
  r.N = (int)p->in;
  r.K = (int)p->out;
  r.segments = dz1 ? 2 : 1;
  r.out[0] = dx;
  return r;
}

// dw_b = x^T dz_b.
hc::Product dw_product(const hclrmix_product* p, const Strides& s, const void* x, const void* dz0, const void* dz1,
                       void* dw0, void* dw1) {
  hc::Product r = base_product();
  r.p[0] = x;
  r.p[1] = dz1 ? x : nullptr;
  r.q[0] = dz0;
  r.q[1] = dz1;
  r.ldp = s.x;
  r.ldq = p->out;
  r.M = p->in;
  r.N = (int)p->out;
  r.K = (int)p->rows;
  r.p_trans = r.q_trans = true;
  r.batch = dz1 ? 2 : 1;
  r.out[0] = dw0;
  r.out[1] = dw1;
  return r;
}

}  // namespace

extern "C" {

hclrmix_status hclrmix_residual_norm(const void* y, const void* residual, const void* gate, const void* post_scale,
                                     const void* pre_scale, void* residual_out, void* normed,
                                     const hclrmix_norm_problem* problem, void* stream) {
  if (hclrmix_status st = check_norm(problem)) return st;
  const hclrmix_norm_problem& p = *problem;
  if ((gate != nullptr) != (p.gate != HCLRMIX_GATE_NONE) && p.rows > 0)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "the gate pointer does not match problem.gate");
  if (p.rows == 0) return ok();
  if (!y || !residual_out) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "y and residual_out are required");
  if (pre_scale && !normed) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "pre_scale without normed");
  const size_t es = elem_size(p.dtype);
  const int64_t m = p.rows, h = p.hidden;
  if (hclrmix_status st = check_tensors(
          {span("y", y, m, h, h, es), span("residual", residual, m, h, h, es), gate_span("gate", gate, problem, es),
           span("post_scale", post_scale, 1, h, h, es), span("pre_scale", pre_scale, 1, h, h, es)},
          {span("residual_out", residual_out, m, h, h, es), span("normed", normed, m, h, h, es)}, es))
    return st;
  hc::NormArgs a = norm_args(problem);
  a.y = y;
  a.res = residual;
  a.gate = gate;
  a.post = post_scale;
  a.pre = pre_scale;
  a.res_out = residual_out;
  a.normed = normed;
  const bool aln = h % 8 == 0 && all16({y, residual, p.gate == HCLRMIX_GATE_ELEMENT ? gate : nullptr, post_scale,
                                        pre_scale, residual_out, normed});
  (void)hipGetLastError();
  return done(hc::launch_norm(a, p.dtype, aln, (hipStream_t)stream));
}

hclrmix_status hclrmix_residual_norm_workspace_size(const hclrmix_norm_problem* problem, size_t* bytes) {
  if (hclrmix_status st = check_norm(problem)) return st;
  if (!bytes) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  *bytes = norm_workspace(problem);
  return ok();
}

hclrmix_status hclrmix_residual_norm_backward(const void* y, const void* residual_out, const void* gate,
                                              const void* post_scale, const void* pre_scale,
                                              const void* d_residual_out, const void* d_normed, void* dy,
                                              void* d_residual, void* d_gate, void* d_post_scale, void* d_pre_scale,
                                              void* workspace, size_t workspace_bytes,
                                              const hclrmix_norm_problem* problem, void* stream) {
  if (hclrmix_status st = check_norm(problem)) return st;
  const hclrmix_norm_problem& p = *problem;
  const int64_t m = p.rows, h = p.hidden;
  if ((gate != nullptr) != (p.gate != HCLRMIX_GATE_NONE) && m > 0)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "the gate pointer does not match problem.gate");
  if (d_gate && p.gate == HCLRMIX_GATE_NONE) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "d_gate without a gate");
  if (d_post_scale && !post_scale) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "d_post_scale without post_scale");
  if (d_pre_scale && !pre_scale) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "d_pre_scale without pre_scale");
  if (pre_scale && !d_normed && m > 0) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "pre_scale without d_normed");
  if (!dy && !d_residual && !d_gate && !d_post_scale && !d_pre_scale)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "no gradient is wanted");
  if (m > 0 && (!y || !residual_out)) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "y and residual_out are required");
  const size_t es = elem_size(p.dtype);
  const bool sums = d_post_scale || d_pre_scale;
  const size_t need = sums && m > 0 ? norm_workspace(problem) : 0;
  const Range dg = p.gate == HCLRMIX_GATE_ELEMENT ? span("d_gate", d_gate, m, h, h, es) : span("d_gate", d_gate, m, 1, 1, es);
  if (hclrmix_status st = check_tensors(
          {span("y", y, m, h, h, es), span("residual_out", residual_out, m, h, h, es), gate_span("gate", gate, problem, es),
           span("post_scale", post_scale, 1, h, h, es), span("pre_scale", pre_scale, 1, h, h, es),
           span("d_residual_out", d_residual_out, m, h, h, es), span("d_normed", d_normed, m, h, h, es)},
          {span("dy", dy, m, h, h, es), span("d_residual", d_residual, m, h, h, es), dg,
           span("d_post_scale", d_post_scale, 1, h, h, es), span("d_pre_scale", d_pre_scale, 1, h, h, es),
           Range{"workspace", (uintptr_t)workspace, (uintptr_t)workspace + (workspace ? need : 0)}},
          es))
    return st;
  if (hclrmix_status st = check_workspace(workspace, workspace_bytes, need)) return st;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  if (m == 0) {
    hipError_t e = hipSuccess;
    if (d_post_scale) e = hc::launch_zero(d_post_scale, (size_t)h * es, s);
    if (d_pre_scale && e == hipSuccess) e = hc::launch_zero(d_pre_scale, (size_t)h * es, s);
    return done(e);
  }
  hc::NormArgs a = norm_args(problem);
  a.y = y;
  a.res = residual_out;
  a.gate = gate;
  a.post = post_scale;
  a.pre = pre_scale;
  a.dres = d_residual_out;
  a.dn = d_normed;
  a.dy = dy;
  a.d_residual = d_residual;
  a.d_gate = d_gate;
  a.d_post = d_post_scale;
  a.d_pre = d_pre_scale;
  a.partial = sums ? (float*)((char*)workspace + HCLRMIX_COUNTER_BYTES) : nullptr;
  const bool aln = h % 8 == 0 && all16({y, residual_out, p.gate == HCLRMIX_GATE_ELEMENT ? gate : nullptr,
                                        p.gate == HCLRMIX_GATE_ELEMENT ? d_gate : nullptr, post_scale, pre_scale,
                                        d_residual_out, d_normed, dy, d_residual, d_post_scale, d_pre_scale});
  return done(hc::launch_norm_backward(a, p.dtype, aln, s));
}

hclrmix_status hclrmix_linear(const void* x, const void* weight, const void* bias, const void* residual, void* y,
                              void* preact, void* workspace, size_t workspace_bytes, const hclrmix_product* problem,
                              void* stream) {
  Strides st_;
  if (hclrmix_status st = check_product(problem, true, &st_)) return st;
  const hclrmix_product& p = *problem;
  if (p.rows == 0) return ok();
  if (!x || !weight || !y) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "x, weight and y are required");
  const size_t es = elem_size(p.dtype);
  const ProductWorkspace w = forward_workspace(problem, false);
  if (hclrmix_status st = check_tensors(
          {span("x", x, p.rows, p.in, st_.x, es), span("weight", weight, p.in, p.out, st_.w, es),
           span("bias", bias, 1, p.out, p.out, es), span("residual", residual, p.rows, p.out, st_.r, es)},
          {span("y", y, p.rows, p.out, p.out, es), span("preact", preact, p.rows, p.out, p.out, es),
           Range{"workspace", (uintptr_t)workspace, (uintptr_t)workspace + (workspace ? w.bytes : 0)}},
          es))
    return st;
  if (hclrmix_status st = check_workspace(workspace, workspace_bytes, w.bytes)) return st;
  hc::Product r = base_product();
  r.p[0] = x;
  r.q[0] = weight;
  r.ldp = st_.x;
  r.ldq = st_.w;
  r.ldr = st_.r;
  r.M = p.rows;
  r.N = (int)p.out;
  r.K = (int)p.in;
  r.q_trans = true;
  r.bias[0] = bias;
  r.residual = residual;
  r.out[0] = y;
  r.save[0] = preact;
  r.act = p.activation;
  (void)hipGetLastError();
  return done(hc::launch_product(r, p.dtype, (char*)workspace + w.scratch, (unsigned*)workspace, (hipStream_t)stream));
}

hclrmix_status hclrmix_glu(const void* x, const void* gate_weight, const void* up_weight, const void* gate_bias,
                           const void* up_bias, void* h, void* g_out, void* u_out, void* workspace,
                           size_t workspace_bytes, const hclrmix_product* problem, void* stream) {
  Strides st_;
  if (hclrmix_status st = check_product(problem, false, &st_)) return st;
  const hclrmix_product& p = *problem;
  if (p.residual_stride != 0) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "residual_stride must be 0");
  if ((g_out != nullptr) != (u_out != nullptr))
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "g_out and u_out must be given together");
  if (p.rows == 0) return ok();
  if (!x || !gate_weight || !up_weight || !h)
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "x, gate_weight, up_weight and h are required");
  const size_t es = elem_size(p.dtype);
  const ProductWorkspace w = forward_workspace(problem, true);
  if (hclrmix_status st = check_tensors(
          {span("x", x, p.rows, p.in, st_.x, es), span("gate_weight", gate_weight, p.in, p.out, st_.w, es),
           span("up_weight", up_weight, p.in, p.out, st_.w, es), span("gate_bias", gate_bias, 1, p.out, p.out, es),
           span("up_bias", up_bias, 1, p.out, p.out, es)},
          {span("h", h, p.rows, p.out, p.out, es), span("g_out", g_out, p.rows, p.out, p.out, es),
           span("u_out", u_out, p.rows, p.out, p.out, es),
           Range{"workspace", (uintptr_t)workspace, (uintptr_t)workspace + (workspace ? w.bytes : 0)}},
          es))
    return st;
  if (hclrmix_status st = check_workspace(workspace, workspace_bytes, w.bytes)) return st;
  hc::Product r = base_product();
  r.p[0] = x;
  r.q[0] = gate_weight;
  r.q[1] = up_weight;
  r.ldp = st_.x;
  r.ldq = st_.w;
  r.M = p.rows;
  r.N = (int)p.out;
  r.K = (int)p.in;
  r.q_trans = r.dual = true;
  r.bias[0] = gate_bias;
  r.bias[1] = up_bias;
  r.out[0] = h;
  r.save[0] = g_out;
  r.save[1] = u_out;
  r.act = p.activation;
  (void)hipGetLastError();
  return done(hc::launch_product(r, p.dtype, (char*)workspace + w.scratch, (unsigned*)workspace, (hipStream_t)stream));
}

hclrmix_status hclrmix_linear_backward(const void* x, const void* weight, const void* preact, const void* dy, void* dx,
                                       void* d_weight, void* d_bias, void* workspace, size_t workspace_bytes,
                                       const hclrmix_product* problem, void* stream) {
  Strides st_;
  if (hclrmix_status st = check_product(problem, true, &st_)) return st;
  const hclrmix_product& p = *problem;
  const bool act = p.activation != HCLRMIX_ACT_NONE;
  if (p.residual_stride != 0) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "residual_stride must be 0");
  if (!dx && !d_weight && !d_bias) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "no gradient is wanted");
  if (!act && preact) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "preact without an activation");
  if (p.rows > 0 && (!dy || (act && !preact) || (dx && !weight) || (d_weight && !x)))
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT,
                "dy is required, preact with an activation, weight for dx and x for d_weight");
  const size_t es = elem_size(p.dtype);
  const ProductWorkspace w = backward_workspace(problem, false);
  const int64_t m = p.rows, k = p.in, n = p.out;
  if (hclrmix_status st = check_tensors(
          {span("x", x, m, k, st_.x, es), span("weight", weight, k, n, st_.w, es), span("preact", preact, m, n, n, es),
           span("dy", dy, m, n, n, es)},
          {span("dx", dx, m, k, k, es), span("d_weight", d_weight, k, n, n, es), span("d_bias", d_bias, 1, n, n, es),
           Range{"workspace", (uintptr_t)workspace, (uintptr_t)workspace + (workspace ? w.bytes : 0)}},
          es))
    return st;
  if (hclrmix_status st = check_workspace(workspace, workspace_bytes, m > 0 ? w.bytes : 0)) return st;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  if (m == 0) {
    if (d_weight) e = hc::launch_zero(d_weight, (size_t)k * n * es, s);
    if (d_bias && e == hipSuccess) e = hc::launch_zero(d_bias, (size_t)n * es, s);
    return done(e);
  }
  char* ws = (char*)workspace;
  const bool products = dx || d_weight;
  void* dz = act && products ? ws + w.dz0 : nullptr;
  float* sums = d_bias ? (float*)(ws + w.sums) : nullptr;
  if (dz || sums)
    e = hc::launch_act_grad(dy, preact, nullptr, dz, nullptr, sums, d_bias, nullptr, m, n, p.activation, p.dtype,
                            n % 8 == 0 && all16({dy, preact}), s);
  const void* d = act ? dz : dy;
  if (e == hipSuccess && dx)
    e = hc::launch_product(dx_product(problem, st_, d, nullptr, weight, nullptr, dx), p.dtype, ws + w.scratch, (unsigned*)ws, s);
  if (e == hipSuccess && d_weight)
    e = hc::launch_product(dw_product(problem, st_, x, d, nullptr, d_weight, nullptr), p.dtype, ws + w.scratch, (unsigned*)ws, s);
  return done(e);
}

hclrmix_status hclrmix_glu_backward(const void* x, const void* gate_weight, const void* up_weight, const void* g,
                                    const void* u, const void* dh, void* dx, void* d_gate_weight, void* d_up_weight,
                                    void* d_gate_bias, void* d_up_bias, void* workspace, size_t workspace_bytes,
                                    const hclrmix_product* problem, void* stream) {
  Strides st_;
  if (hclrmix_status st = check_product(problem, false, &st_)) return st;
  const hclrmix_product& p = *problem;
  if (p.residual_stride != 0) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "residual_stride must be 0");
  if ((d_gate_weight != nullptr) != (d_up_weight != nullptr) || (d_gate_bias != nullptr) != (d_up_bias != nullptr))
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "the two weights' gradients come together, and the two biases'");
  if (!dx && !d_gate_weight && !d_gate_bias) return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "no gradient is wanted");
  if (p.rows > 0 && (!g || !u || !dh || (dx && (!gate_weight || !up_weight)) || (d_gate_weight && !x)))
    return fail(HCLRMIX_ERR_INVALID_ARGUMENT, "g, u and dh are required, the weights for dx and x for their gradients");
  const size_t es = elem_size(p.dtype);
  const ProductWorkspace w = backward_workspace(problem, true);
  const int64_t m = p.rows, k = p.in, n = p.out;
  if (hclrmix_status st = check_tensors(
          {span("x", x, m, k, st_.x, es), span("gate_weight", gate_weight, k, n, st_.w, es),
           span("up_weight", up_weight, k, n, st_.w, es), span("g", g, m, n, n, es), span("u", u, m, n, n, es),
           span("dh", dh, m, n, n, es)},
          {span("dx", dx, m, k, k, es), span("d_gate_weight", d_gate_weight, k, n, n, es),
           span("d_up_weight", d_up_weight, k, n, n, es), span("d_gate_bias", d_gate_bias, 1, n, n, es),
           span("d_up_bias", d_up_bias, 1, n, n, es),
           Range{"workspace", (uintptr_t)workspace, (uintptr_t)workspace + (workspace ? w.bytes : 0)}},
          es))
    return st;
  if (hclrmix_status st = check_workspace(workspace, workspace_bytes, m > 0 ? w.bytes : 0)) return st;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  if (m == 0) {
    for (void* q : {d_gate_weight, d_up_weight})
      if (q && e == hipSuccess) e = hc::launch_zero(q, (size_t)k * n * es, s);
    for (void* q : {d_gate_bias, d_up_bias})
      if (q && e == hipSuccess) e = hc::launch_zero(q, (size_t)n * es, s);
    return done(e);
  }
  char* ws = (char*)workspace;
  const bool products = dx || d_gate_weight;
  void* dg = products ? ws + w.dz0 : nullptr;
  void* du = products ? ws + w.dz1 : nullptr;
  float* sums = d_gate_bias ? (float*)(ws + w.sums) : nullptr;
  e = hc::launch_act_grad(dh, g, u, dg, du, sums, d_gate_bias, d_up_bias, m, n, p.activation, p.dtype,
                          n % 8 == 0 && all16({dh, g, u}), s);
  if (e == hipSuccess && dx)
    e = hc::launch_product(dx_product(problem, st_, dg, du, gate_weight, up_weight, dx), p.dtype, ws + w.scratch, (unsigned*)ws, s);
  if (e == hipSuccess && d_gate_weight)
    e = hc::launch_product(dw_product(problem, st_, x, dg, du, d_gate_weight, d_up_weight), p.dtype, ws + w.scratch,
                           (unsigned*)ws, s);
  return done(e);
}

hclrmix_status hclrmix_linear_workspace_size(const hclrmix_product* problem, size_t* bytes) {
  return size_of(problem, bytes, false, false);
}
hclrmix_status hclrmix_linear_backward_workspace_size(const hclrmix_product* problem, size_t* bytes) {
  return size_of(problem, bytes, false, true);
}
hclrmix_status hclrmix_glu_workspace_size(const hclrmix_product* problem, size_t* bytes) {
  return size_of(problem, bytes, true, false);
}
hclrmix_status hclrmix_glu_backward_workspace_size(const hclrmix_product* problem, size_t* bytes) {
  return size_of(problem, bytes, true, true);
}

}  // extern "C"

// C ABI of the operators around dispatch and combine: RMS norm, the experts'
// products, and the backward passes of all of them. Argument checks,
// workspace layout and launches; group offsets and slots come from the plan
// and are checked by the kernels.
#include "ep.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "ep_checks.hpp"
#include "ep_desc.hpp"
#include "ep_kernels.hpp"

namespace {

using ep::check_aligned16;
using ep::check_ptr;
using ep::derive;
using ep::DeviceScope;
using ep::fail;
using ep::fail_hip;

// One buffer of a call: `bytes` from p; name for messages.
struct Span {
  const void* p;
  int64_t bytes;
  const char* name;
};

// Device memory, aligned, large enough; null passes when `optional`.
int check_span(const Span& s, int dev, bool optional = false) {
  if (!s.p && optional) return EP_OK;
  EP_CHECK(check_ptr(s.p, dev, s.name, s.bytes));
  return check_aligned16(s.p, s.name);
}

// No output shares bytes with another buffer of the call.
int check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  const auto meet = [](const Span& a, const Span& b) {
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 &&
           (uintptr_t)a.p < (uintptr_t)b.p + (uint64_t)b.bytes &&
           (uintptr_t)b.p < (uintptr_t)a.p + (uint64_t)a.bytes;
  };
  const auto refuse = [](const Span& a, const Span& b) {
    return fail(EP_ERR_INVALID_ARG,
                (std::string("buffers overlap: ") + a.name + " and " + b.name).c_str());
  };
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    for (auto b = a + 1; b != outs.end(); ++b)
      if (meet(*a, *b)) return refuse(*a, *b);
    for (const Span& b : ins)
      if (meet(*a, b)) return refuse(*a, b);
  }
  return EP_OK;
}

// In-place use of `out` as `in`: the same address, else they must be apart.
const void* unless_same(const void* in, const void* out) { return in == out ? nullptr : in; }

int check_norm(const ep_norm* n) {
  if (!n) return fail(EP_ERR_INVALID_ARG, "null norm");
  if (n->dtype != EP_DTYPE_BF16 && n->dtype != EP_DTYPE_F16)
    return fail(EP_ERR_INVALID_ARG, "norm: dtype must be bf16 or fp16");
  if (n->reserved != 0) return fail(EP_ERR_INVALID_ARG, "norm: reserved must be 0");
  if (n->rows < 0) return fail(EP_ERR_INVALID_ARG, "norm: rows must not be negative");
  if (n->hidden < 8 || n->hidden % 8 != 0)
    return fail(EP_ERR_INVALID_ARG, "norm: hidden must be a positive multiple of 8");
  if (!(n->eps >= 0.0f) || std::isinf(n->eps))
    return fail(EP_ERR_INVALID_ARG, "norm: eps must be finite and not negative");
  if (n->hidden > EP_NORM_MAX_HIDDEN)
    return fail(EP_ERR_UNSUPPORTED, "norm: hidden must be at most EP_NORM_MAX_HIDDEN");
  if (n->rows >= ((int64_t)1 << 31))
    return fail(EP_ERR_UNSUPPORTED, "norm: rows must be < 2^31");
  return EP_OK;
}

int check_product(const ep_product* p) {
  if (!p) return fail(EP_ERR_INVALID_ARG, "null product");
  if (p->dtype != EP_DTYPE_BF16 && p->dtype != EP_DTYPE_E4M3)
    return fail(EP_ERR_INVALID_ARG, "product: dtype must be bf16 or e4m3");
  if (p->act < EP_ACT_NONE || p->act > EP_ACT_SWIGLU)
    return fail(EP_ERR_INVALID_ARG, "product: unknown activation");
  const int unit = p->dtype == EP_DTYPE_E4M3 ? 128 : 8;
  if (p->in < 1 || p->out < 1 || p->in % unit != 0 || p->out % unit != 0)
    return fail(EP_ERR_INVALID_ARG,
                "product: in and out must be positive multiples of 8 (of 128 for e4m3)");
  if (p->dtype != EP_DTYPE_E4M3 && p->w_scale)
    return fail(EP_ERR_INVALID_ARG, "product: scales belong to e4m3 weights only");
  // The kernels take offsets inside a matrix, and inside 256 rows, in 31 bits.
  if ((int64_t)p->in * ep::weight_rows(*p) >= ((int64_t)1 << 30) || p->in >= (1 << 20) ||
      ep::weight_rows(*p) >= (1 << 20))
    return fail(EP_ERR_UNSUPPORTED,
                "product: a matrix must have fewer than 2^30 elements, in and W below 2^20");
  return EP_OK;
}

// Which rows belong to which expert: the plan's, or all of a rank's.
int groups_of(const ep::Dims& d, const void* plan_ws, ep::Groups* g) {
  *g = ep::Groups{nullptr, d.N, d.L, d.cap, d.N * d.cap};
  if (!plan_ws) {
    if (d.E != d.N)
      return fail(EP_ERR_INVALID_ARG, "without a plan n_experts must be n_ranks");
    return EP_OK;
  }
  g->off = ep::plan_ptrs(d, plan_ws).grp_off;
  if (d.NTR < g->most) g->most = d.NTR;
  // Without tokens no plan need have been made, and no row buffer is checked:
  // offsets of any value then name no rows.
  if (g->most == 0) g->cap = 0;
  return EP_OK;
}

int check_plan(const ep::Dims& d, const void* plan_ws, int dev) {
  if (!plan_ws) return EP_OK;
  EP_CHECK(check_ptr(plan_ws, dev, "plan_ws", (int64_t)ep::layout_of(d).bytes));
  return check_aligned16(plan_ws, "plan_ws");
}

int64_t w_elems(const ep::Dims& d, const ep_product& p) {
  return (int64_t)d.E * ep::weight_rows(p) * p.in;
}

}  // namespace

extern "C" {

int ep_rms_norm(const ep_norm* n, const void* x, const void* residual, void* sum, void* y,
                uint8_t* codes, float* scales, hipStream_t stream) {
  EP_CHECK(check_norm(n));
  if (n->rows == 0) return EP_OK;
  if ((residual != nullptr) != (sum != nullptr))
    return fail(EP_ERR_INVALID_ARG, "residual and sum must be given together");
  if ((codes != nullptr) != (scales != nullptr))
    return fail(EP_ERR_INVALID_ARG, "codes and scales must be given together");
  if (!y && !codes) return fail(EP_ERR_INVALID_ARG, "y or codes must be given");
  if (codes && n->hidden % 128 != 0)
    return fail(EP_ERR_INVALID_ARG, "codes need hidden % 128 == 0");
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  const int64_t elems = n->rows * n->hidden;
  const Span sx{x, 2 * elems, "x"}, sr{residual, 2 * elems, "residual"}, ss{sum, 2 * elems, "sum"},
      sy{y, 2 * elems, "y"}, sc{codes, elems, "codes"}, sf{scales, elems / 32, "scales"},
      sw{n->weight, 2 * (int64_t)n->hidden, "weight"};
  EP_CHECK(check_span(sx, scope.device()));
  EP_CHECK(check_span(sw, scope.device()));
  for (const Span& s : {sr, ss, sy, sc, sf}) EP_CHECK(check_span(s, scope.device(), true));
  EP_CHECK(check_apart({ss, sy, sc, sf},
                       {sx, Span{unless_same(residual, sum), 2 * elems, "residual"}, sw}));
  const hipError_t e = ep::launch_rms_norm(*n, x, residual, sum, y, codes, scales, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_rms_norm");
  return EP_OK;
}

size_t ep_rms_norm_grad_bytes(const ep_norm* n) {
  if (check_norm(n) != EP_OK) return 0;
  return (size_t)ep::norm_grad_parts(*n) * n->hidden * 4;
}

int ep_rms_norm_grad(const ep_norm* n, const void* dy, const void* h, const void* dsum, void* dx,
                     float* dweight, void* ws, hipStream_t stream) {
  EP_CHECK(check_norm(n));
  if (!dx && n->rows > 0) return fail(EP_ERR_INVALID_ARG, "null pointer: dx");
  if (n->rows == 0 && !dweight) return EP_OK;
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  const int64_t elems = n->rows * n->hidden;
  const int64_t room = dweight ? (int64_t)ep::norm_grad_parts(*n) * n->hidden * 4 : 0;
  const Span sd{dy, 2 * elems, "dy"}, sh{h, 2 * elems, "h"}, ss{dsum, 2 * elems, "dsum"},
      sx{dx, 2 * elems, "dx"}, sg{dweight, 4 * (int64_t)n->hidden, "dweight"},
      sw{n->weight, 2 * (int64_t)n->hidden, "weight"}, st{ws, room, "ws"};
  if (elems > 0) {
    for (const Span& s : {sd, sh, sx, sw}) EP_CHECK(check_span(s, scope.device()));
    EP_CHECK(check_span(ss, scope.device(), true));
  }
  if (dweight) {
    EP_CHECK(check_span(sg, scope.device()));
    EP_CHECK(check_span(st, scope.device()));
  }
  EP_CHECK(check_apart({sx, sg, st},
                       {sd, sh, sw, Span{unless_same(dsum, dx), 2 * elems, "dsum"}}));
  const hipError_t e = ep::launch_rms_norm_grad(*n, dy, h, dsum, dx, dweight, (float*)ws, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_rms_norm_grad");
  return EP_OK;
}

int ep_expert_product(const ep_desc* d, const ep_product* p, const void* const x[2],
                      const void* plan_ws, const void* residual, void* pre, void* out,
                      hipStream_t stream) {
  ep::Dims dims;
  EP_CHECK(derive(d, &dims));
  EP_CHECK(check_product(p));
  if (!x) return fail(EP_ERR_INVALID_ARG, "null plane array: x");
  const bool fp8 = p->dtype == EP_DTYPE_E4M3;
  if (!fp8 && x[1]) return fail(EP_ERR_INVALID_ARG, "plane 1 must be NULL for bf16: x");
  ep::Groups g;
  EP_CHECK(groups_of(dims, plan_ws, &g));
  if (!ep::line_fits(g, p->out))
    return fail(EP_ERR_UNSUPPORTED, "product: too many tiles of rows by out");
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  const int dev = scope.device();
  EP_CHECK(check_plan(dims, plan_ws, dev));
  if (g.most == 0) return EP_OK;
  const int64_t rows = dims.N * dims.cap, W = ep::weight_rows(*p), we = w_elems(dims, *p);
  const Span s0{x[0], rows * p->in * (fp8 ? 1 : 2), "x"}, s1{x[1], rows * (p->in / 32), "x scales"},
      sw{p->w, we * (fp8 ? 1 : 2), "w"}, sf{p->w_scale, we / 4096, "w_scale"},
      sb{p->bias, 2 * dims.E * W, "bias"}, sr{residual, 2 * rows * p->out, "residual"},
      sp{pre, 2 * rows * W, "pre"}, so{out, 2 * rows * p->out, "out"};
  for (const Span& s : {s0, sw, so}) EP_CHECK(check_span(s, dev));
  for (const Span& s : {sb, sr, sp}) EP_CHECK(check_span(s, dev, true));
  if (fp8) {
    EP_CHECK(check_span(s1, dev));
    EP_CHECK(check_span(sf, dev));
  }
  EP_CHECK(check_apart({so, sp}, {s0, Span{fp8 ? x[1] : nullptr, s1.bytes, "x scales"}, sw, sf, sb,
                                  sr, Span{plan_ws, (int64_t)ep::layout_of(dims).bytes, "plan_ws"}}));
  const hipError_t e = ep::launch_product(*p, g, x, residual, pre, out, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_expert_product");
  return EP_OK;
}

size_t ep_expert_product_grad_bytes(const ep_desc* d, const ep_product* p) {
  ep::Dims dims;
  if (derive(d, &dims) != EP_OK || check_product(p) != EP_OK) return 0;
  return (size_t)ep::product_grad_bytes(*p, dims);
}

int ep_expert_product_grad(const ep_desc* d, const ep_product* p, const uint16_t* dout,
                           const uint16_t* x, const uint16_t* pre, const void* plan_ws, void* ws,
                           uint16_t* dx, uint16_t* dw, float* dbias, hipStream_t stream) {
  ep::Dims dims;
  EP_CHECK(derive(d, &dims));
  EP_CHECK(check_product(p));
  if (p->dtype != EP_DTYPE_BF16)
    return fail(EP_ERR_UNSUPPORTED, "ep_expert_product_grad takes bf16 products");
  const bool empty = dims.N * dims.cap == 0;  // no buffer of rows has an address then
  if (!empty && (pre != nullptr) != (p->act != EP_ACT_NONE))
    return fail(EP_ERR_INVALID_ARG, "pre must be given with an activation, and only then");
  if (!dx && !dw && !dbias)
    return empty ? EP_OK : fail(EP_ERR_INVALID_ARG, "dx, dw or dbias must be given");
  ep::Groups g;
  EP_CHECK(groups_of(dims, plan_ws, &g));
  if (dx && !ep::line_fits(g, p->in))
    return fail(EP_ERR_UNSUPPORTED, "product: too many tiles of rows by in");
  if ((dbias || p->act != EP_ACT_NONE) && !ep::act_grad_fits(g, p->out))
    return fail(EP_ERR_UNSUPPORTED, "product: too many blocks of rows by out for one launch");
  DeviceScope scope(stream);
  if (scope.error() != hipSuccess) return fail_hip(scope.error(), "device");
  const int dev = scope.device();
  EP_CHECK(check_plan(dims, plan_ws, dev));
  const int64_t rows = g.most == 0 ? 0 : dims.N * dims.cap, W = ep::weight_rows(*p);
  const Span sd{dout, 2 * rows * p->out, "dout"}, sx{x, 2 * rows * p->in, "x"},
      sp{pre, 2 * rows * W, "pre"}, sw{p->w, 2 * w_elems(dims, *p), "w"},
      st{ws, ep::product_grad_bytes(*p, dims), "ws"}, s0{dx, 2 * rows * p->in, "dx"},
      s1{dw, 2 * w_elems(dims, *p), "dw"}, s2{dbias, 4 * dims.E * W, "dbias"};
  for (const Span& s : {sd, st}) EP_CHECK(check_span(s, dev));
  for (const Span& s : {sp, s0, s1, s2}) EP_CHECK(check_span(s, dev, true));
  if (dx) EP_CHECK(check_span(sw, dev));
  if (dw) EP_CHECK(check_span(sx, dev));
  EP_CHECK(check_apart({s0, s1, s2, st},
                       {sd, Span{dw ? x : nullptr, sx.bytes, "x"}, sp, sw,
                        Span{plan_ws, (int64_t)ep::layout_of(dims).bytes, "plan_ws"}}));
  const hipError_t e =
      ep::launch_product_grad(*p, dims, g, dout, x, pre, ws, dx, dw, dbias, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_expert_product_grad");
  return EP_OK;
}

int ep_combine_grad(const ep_desc* d, const uint16_t* dout, const uint16_t* y,
                    const float* weights, const void* plan_ws, uint16_t* dy, float* dweights,
                    hipStream_t stream) {
  EP_PROLOGUE(d, stream, plan_ws);
  if (dims.NT == 0) return EP_OK;
  if (!dy && !dweights) return fail(EP_ERR_INVALID_ARG, "dy or dweights must be given");
  const int dev = scope.device();
  const int64_t row = 2 * (int64_t)dims.H, rows = dims.N * dims.cap;
  const Span sd{dout, dims.NT * row, "dout"}, sy{y, rows * row, "y"},
      sw{weights, 4 * dims.NTR, "weights"}, s0{dy, rows * row, "dy"},
      s1{dweights, 4 * dims.NTR, "dweights"},
      sp{plan_ws, (int64_t)ep::layout_of(dims).bytes, "plan_ws"};
  EP_CHECK(check_span(sd, dev));
  if (dy) {
    EP_CHECK(check_span(s0, dev));
    EP_CHECK(check_ptr(weights, dev, "weights", sw.bytes));
  }
  if (dweights) {
    EP_CHECK(check_span(sy, dev));
    EP_CHECK(check_ptr(dweights, dev, "dweights", s1.bytes));
  }
  EP_CHECK(check_apart({s0, s1}, {sd, Span{dweights ? y : nullptr, sy.bytes, "y"},
                                  Span{dy ? weights : nullptr, sw.bytes, "weights"}, sp}));
  const hipError_t e = ep::launch_combine_grad(dims, dout, y, weights, pp, dy, dweights, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_combine_grad");
  return EP_OK;
}

int ep_dispatch_grad(const ep_desc* d, const uint16_t* dgrouped, const uint16_t* add,
                     const void* plan_ws, uint16_t* dx, hipStream_t stream) {
  EP_PROLOGUE(d, stream, plan_ws);
  if (dims.NT == 0) return EP_OK;
  const int dev = scope.device();
  const int64_t row = 2 * (int64_t)dims.H;
  const Span sg{dgrouped, dims.N * dims.cap * row, "dgrouped"}, sa{add, dims.NT * row, "add"},
      sx{dx, dims.NT * row, "dx"}, sp{plan_ws, (int64_t)ep::layout_of(dims).bytes, "plan_ws"};
  EP_CHECK(check_span(sg, dev));
  EP_CHECK(check_span(sa, dev, true));
  EP_CHECK(check_span(sx, dev));
  EP_CHECK(check_apart({sx}, {sg, Span{unless_same(add, dx), sa.bytes, "add"}, sp}));
  const hipError_t e = ep::launch_dispatch_grad(dims, dgrouped, add, pp, dx, stream);
  if (e != hipSuccess) return fail_hip(e, "ep_dispatch_grad");
  return EP_OK;
}

}  // extern "C"

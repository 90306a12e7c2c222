// nodes.cpp -- the norms, the linear layer and the feed-forward layer as autograd
// nodes: checks of arguments, outputs, workspaces, and calls of the C ABI
// (include/swiglu_mlp.h), which does all arithmetic.
//
// In C++ because a small training step is bound by its host code: a node in Python
// runs on the engine's thread, which first has to get the interpreter, with cold
// caches (RMS norm of 33 x 11008 with gradients 86 us as a Python node, 58 as this
// one; layer norm of 777 x 1001 101 and 72).
#include <ATen/DeviceGuard.h>
#include <c10/core/AutogradState.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/extension.h>

#include <cmath>

#include "swiglu_mlp.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using Maybe = std::optional<Tensor>;

// A status of the C ABI.
struct StatusError : std::runtime_error {
  int status;
  const char* where;
  StatusError(int status, const char* where)
      : std::runtime_error(std::string(where) + ": " + swiglu_mlp_status_string(status)), status(status), where(where) {}
};
void check(int status, const char* where) {
  if (status) throw StatusError(status, where);
}

// ---- arguments -------------------------------------------------------------------
int code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SWIGLU_BF16;
    case at::kHalf: return SWIGLU_FP16;
    case at::kFloat: return SWIGLU_FP32;
    default: TORCH_CHECK_TYPE(false, "unsupported dtype ", t.scalar_type(), "; use bfloat16, float16, float32");
  }
}
hipStream_t stream(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }
bool there(const Maybe& t) { return t.has_value() && t->defined(); }
void* ptr(const Tensor& t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; }

// All tensors share x's type and device, which is a GPU.
void same(const Tensor& x, std::initializer_list<const Tensor*> others) {
  for (const Tensor* t : others)
    TORCH_CHECK_VALUE(!t || (t->scalar_type() == x.scalar_type() && t->device() == x.device()),
                      "all tensors must share dtype and device");
  TORCH_CHECK_VALUE(x.is_cuda(), "tensors must be on a GPU (cuda/HIP device)");
  code(x);
}
const Tensor* opt(const Maybe& t) { return there(t) ? &*t : nullptr; }

void norm_args(const Tensor& x, const Tensor& w, const Maybe& b, double eps, bool rms) {
  TORCH_CHECK_VALUE(x.dim() == 2 && w.dim() == 1 && w.size(0) == x.size(1) && x.size(1) > 0,
                    "expected X[T,D] and weight[D]: X", x.sizes(), " weight", w.sizes());
  TORCH_CHECK_VALUE(!rms || !there(b), "RMS norm has no bias");
  TORCH_CHECK_VALUE(!there(b) || b->sizes() == w.sizes(), "bias must be [D]: ", b->sizes());
  TORCH_CHECK_VALUE(eps >= 0 && eps < INFINITY, "eps must be a number from 0 up: got ", eps);
  same(x, {&w, opt(b)});
}
void linear_args(const Tensor& x, const Tensor& w, const Maybe& b, const Maybe& r) {
  TORCH_CHECK_VALUE(x.dim() == 2 && w.dim() == 2 && x.size(1) == w.size(1),
                    "shape mismatch (expected X[T,K], W[N,K]): X", x.sizes(), " W", w.sizes());
  TORCH_CHECK_VALUE(!there(b) || (b->dim() == 1 && b->size(0) == w.size(0)), "bias must be [N] = [", w.size(0), "]: ",
                    b->sizes());
  TORCH_CHECK_VALUE(!there(r) || (r->dim() == 2 && r->size(0) == x.size(0) && r->size(1) == w.size(0)),
                    "residual must be [T, N] = [", x.size(0), ", ", w.size(0), "]: ", r->sizes());
  same(x, {&w, opt(b), opt(r)});
}

// Contiguous, and without a negation that torch has put off (the imaginary part of a
// conjugate is such a view).
Tensor flat(const Tensor& t) {
  if (t.is_neg()) return t.resolve_neg().contiguous();
  return t.is_contiguous() ? t : t.contiguous();
}
// Contiguous and at an address that the matrix kernels take (a gradient may be a
// view that starts anywhere).
Tensor flat16(const Tensor& t) {
  Tensor f = flat(t);
  return (uintptr_t)f.data_ptr() % 16 ? f.clone() : f;
}
Tensor flat(const Maybe& t) { return there(t) ? flat(*t) : Tensor(); }
Tensor flat16(const Maybe& t) { return there(t) ? flat16(*t) : Tensor(); }

Tensor workspace(size_t bytes, const Tensor& like) {
  return bytes ? at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)) : Tensor();
}

// ---- calls (arguments checked, flat, on the current device) -------------------------
struct Normed {
  Tensor y, stats;
};
Normed norm_forward(const Tensor& x, const Tensor& w, const Tensor& b, double eps, bool rms, bool stats) {
  Normed r{at::empty_like(x), {}};
  if (stats) r.stats = at::empty({rms ? 1 : 2, x.size(0)}, x.options().dtype(at::kFloat));
  check(swiglu_mlp_norm_fwd(ptr(x), ptr(w), ptr(b), ptr(r.y), (float*)ptr(r.stats), x.size(0), x.size(1), (float)eps, rms,
                            code(x), stream(x)),
        "swiglu_mlp_norm_fwd");
  return r;
}
struct NormGrads {
  Tensor x, w, b;
};
NormGrads norm_backward(const Tensor& dy, const Tensor& x, const Tensor& w, const Tensor& stats, const Tensor& dres, bool rms,
                        bool bias) {
  NormGrads g{at::empty_like(x), at::empty_like(w), bias ? at::empty_like(w) : Tensor()};
  const size_t need = swiglu_mlp_norm_bwd_workspace_bytes(x.size(0), x.size(1), rms, code(x));
  const Tensor ws = workspace(need, x);
  check(swiglu_mlp_norm_bwd(ptr(dy), ptr(x), ptr(w), (const float*)ptr(stats), ptr(dres), ptr(g.x), ptr(g.w), ptr(g.b),
                            ptr(ws), need, x.size(0), x.size(1), rms, code(x), stream(x)),
        "swiglu_mlp_norm_bwd");
  return g;
}
struct Projected {
  Tensor y, z;
};
Projected linear_forward(const Tensor& x, const Tensor& w, const Tensor& b, const Tensor& r, int64_t act, bool keep) {
  const int64_t T = x.size(0), N = w.size(0), K = x.size(1);
  Projected o{at::empty({T, N}, x.options()), {}};
  if (keep && act) o.z = at::empty_like(o.y);
  const size_t need = swiglu_mlp_linear_workspace_bytes(T, N, K, code(x));
  const Tensor ws = workspace(need, x);
  check(swiglu_mlp_linear_fwd(ptr(x), ptr(w), ptr(b), ptr(r), ptr(o.y), ptr(o.z), ptr(ws), need, T, N, K, (int)act, code(x),
                              stream(x)),
        "swiglu_mlp_linear_fwd");
  return o;
}
struct LinearGrads {
  Tensor x, w, b;
};
// x is read for dw, w for dx: what is not wanted may be undefined. K: x's columns.
LinearGrads linear_backward(const Tensor& dy, const Tensor& x, const Tensor& w, const Tensor& z, int64_t K, int64_t act, bool dx,
                            bool dw, bool db) {
  const int64_t T = dy.size(0), N = dy.size(1);
  LinearGrads g;
  if (!dx && !dw && !db) return g;
  if (dx) g.x = at::empty({T, K}, dy.options());
  if (dw) g.w = at::empty({N, K}, dy.options());
  if (db) g.b = at::empty({N}, dy.options());
  const size_t need = swiglu_mlp_linear_bwd_workspace_bytes(T, N, K, (int)act, code(dy));
  const Tensor ws = workspace(need, dy);
  check(swiglu_mlp_linear_bwd(ptr(dy), ptr(x), ptr(w), ptr(z), ptr(g.x), ptr(g.w), ptr(g.b), ptr(ws), need, T, N, K, (int)act,
                              code(dy), stream(dy)),
        "swiglu_mlp_linear_bwd");
  return g;
}

// ---- nodes ----------------------------------------------------------------------
// What the nodes keep beside tensors; whether an input's gradient is wanted is
// asked by its place among the tensors that are there.
struct Needs {
  AutogradContext* ctx;
  size_t at = 0;
  bool next(bool is_there) { return is_there && ctx->needs_input_grad(at++); }
};
void no_second() { TORCH_CHECK(!at::GradMode::is_enabled(), "create_graph=True (double backward) is not supported"); }
int64_t kept(AutogradContext* ctx, const char* key) { return ctx->saved_data[key].toInt(); }

// Only what a wanted gradient reads is kept: a frozen weight's input is free to go, or to
// be changed in place.
Tensor kept_if(bool wanted, const Tensor& t) { return wanted ? t : Tensor(); }
bool wants(const Tensor& t) { return t.requires_grad(); }
bool wants(const Maybe& t) { return there(t) && t->requires_grad(); }

struct Norm : torch::autograd::Function<Norm> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x_, const Tensor& w_, const Maybe& b_, double eps, bool rms) {
    const at::DeviceGuard guard(x_.device());
    const Tensor x = flat(x_), w = flat(w_);
    const Normed r = norm_forward(x, w, flat(b_), eps, rms, true);
    ctx->save_for_backward({x, w, r.stats});
    ctx->saved_data["form"] = (int64_t)(rms + 2 * there(b_));
    return r.y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list dy) {
    no_second();
    const auto s = ctx->get_saved_variables();
    const int64_t form = kept(ctx, "form");
    const at::DeviceGuard guard(s[0].device());
    const NormGrads g = norm_backward(flat(dy[0]), s[0], s[1], s[2], Tensor(), form & 1, form & 2);
    return {g.x, g.w, g.b, Tensor(), Tensor()};
  }
};

struct Linear : torch::autograd::Function<Linear> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x_, const Tensor& w_, const Maybe& b_, const Maybe& r_,
                        int64_t act) {
    const at::DeviceGuard guard(x_.device());
    const Tensor x = flat16(x_), w = flat16(w_);
    const bool dz = wants(x_) || wants(w_) || wants(b_);
    const Projected o = linear_forward(x, w, flat16(b_), flat16(r_), act, dz);
    ctx->save_for_backward({kept_if(wants(w_), x), kept_if(wants(x_), w), o.z});
    ctx->saved_data["act"] = act;
    ctx->saved_data["K"] = x.size(1);
    ctx->saved_data["form"] = (int64_t)(there(b_) + 2 * there(r_));
    return o.y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list dy) {
    no_second();
    const auto s = ctx->get_saved_variables();
    const int64_t form = kept(ctx, "form");
    Needs needs{ctx};
    const bool dx = needs.next(true), dw = needs.next(true), db = needs.next(form & 1), dr = needs.next(form & 2);
    const at::DeviceGuard guard(dy[0].device());
    const LinearGrads g = linear_backward(flat16(dy[0]), s[0], s[1], s[2], kept(ctx, "K"), kept(ctx, "act"), dx, dw, db);
    return {g.x, g.w, g.b, dr ? dy[0] : Tensor(), Tensor()};
  }
};

// The layer as one node: its backward hands the stream's gradient to the norm's
// backward, which adds it to its own, instead of leaving a sum of two tensors.
struct FeedForward : torch::autograd::Function<FeedForward> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x_, const Tensor& nw_, const Maybe& nb_, const Tensor& w1_,
                        const Maybe& b1_, const Tensor& w2_, const Maybe& b2_, int64_t act, double eps, bool rms) {
    const at::DeviceGuard guard(x_.device());
    const Tensor x = flat16(x_), nw = flat(nw_), w1 = flat16(w1_), w2 = flat16(w2_);
    const bool norm = wants(x_) || wants(nw_) || wants(nb_), inner = norm || wants(w1_) || wants(b1_);
    const Normed n = norm_forward(x, nw, flat(nb_), eps, rms, norm);
    const Projected a = linear_forward(n.y, w1, flat16(b1_), Tensor(), act, inner);
    const Projected y = linear_forward(a.y, w2, flat16(b2_), x, SWIGLU_ACT_NONE, false);
    ctx->save_for_backward({kept_if(norm, x), kept_if(norm, nw), kept_if(norm, w1), kept_if(inner, w2), kept_if(wants(w1_), n.y), n.stats,
                            kept_if(wants(w2_), a.y), a.z});
    ctx->saved_data["act"] = act;
    ctx->saved_data["H"] = w1.size(0);
    ctx->saved_data["form"] = (int64_t)(rms + 2 * there(nb_) + 4 * there(b1_) + 8 * there(b2_));
    return y.y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list dy_) {
    no_second();
    const auto s = ctx->get_saved_variables();
    const Tensor &x = s[0], &nw = s[1], &w1 = s[2], &w2 = s[3], &n = s[4], &stats = s[5], &a = s[6], &z = s[7];
    const int64_t form = kept(ctx, "form");
    Needs needs{ctx};
    const bool dx = needs.next(true), dnw = needs.next(true), dnb = needs.next(form & 2), dw1 = needs.next(true),
               db1 = needs.next(form & 4), dw2 = needs.next(true), db2 = needs.next(form & 8);
    const bool norm = dx || dnw || dnb, inner = norm || dw1 || db1;
    const at::DeviceGuard guard(dy_[0].device());
    const Tensor dy = flat16(dy_[0]);
    LinearGrads g2 = linear_backward(dy, a, w2, Tensor(), kept(ctx, "H"), SWIGLU_ACT_NONE, inner, dw2, db2), g1;
    NormGrads g0;
    if (inner) {
      g1 = linear_backward(g2.x, n, w1, z, dy.size(1), kept(ctx, "act"), norm, dw1, db1);
      g2.x = Tensor();  // (its memory serves what follows)
      if (norm) g0 = norm_backward(g1.x, x, nw, stats, dy, form & 1, form & 2);
    }
    return {g0.x, g0.w, g0.b, g1.w, g1.b, g2.w, g2.b, Tensor(), Tensor(), Tensor()};
  }
};

// ---- entries ----------------------------------------------------------------------
// The kernels' work is seen by no tracer and by no forward-mode derivative: refused,
// where a traced call would be left out of the graph and its output be whatever the
// memory holds, and a derivative be zero.
void check_transforms(std::initializer_list<const Tensor*> ts) {
  using Modes = c10::impl::TorchDispatchModeTLS;
  TORCH_CHECK(!torch::jit::tracer::isTracing() &&
                  !(Modes::any_modes_set() && Modes::get_mode(c10::impl::TorchDispatchModeKey::PROXY).has_value()),
              "this operator cannot be traced (torch.jit.trace, make_fx): its kernels would be left out of the graph");
  if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
  for (const Tensor* t : ts)
    TORCH_CHECK(!t || !t->_fw_grad(0).defined(), "this operator has no forward-mode derivative, and an input has a tangent");
}
bool wants_grad(std::initializer_list<const Tensor*> ts) {
  if (!at::GradMode::is_enabled()) return false;
  for (const Tensor* t : ts)
    if (t && t->requires_grad()) return true;
  return false;
}
// A leaf's accumulation node belongs to the stream it was made on and lives as long as a
// graph that uses it. Where that is the default stream, a captured backward would
// make the default stream wait for the capture, which is an error that ends the
// capture in the engine's threads: refused here instead. In the forward, although only a
// backward would leave the capture, since other operators' nodes of the same step may
// reach such a leaf before these nodes are asked; a forward without a backward belongs under
// torch.no_grad, which nothing refuses.
void check_capture(std::initializer_list<const Tensor*> ts) {
  const Tensor& x = **ts.begin();
  hipStream_t s = stream(x);
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  if (!s || hipStreamIsCapturing(s, &status) != hipSuccess || status == hipStreamCaptureStatusNone) return;
  for (const Tensor* t : ts) {
    if (!t || !t->requires_grad() || !t->is_leaf()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    const auto made_on = node ? node->stream() : std::nullopt;
    TORCH_CHECK(!made_on || made_on->id() != 0,
                "an autograd graph of the same leaves, built on the default stream, is alive: its accumulation would leave "
                "this capture; delete it (its loss and outputs) or build it on a side stream; capture a forward without a backward under "
                "torch.no_grad()");
  }
}
// x [..., D] as rows
Tensor rows(const Tensor& x) {
  if (x.dim() == 2) return x;
  TORCH_CHECK_VALUE(x.dim() > 0 && x.size(-1) > 0, "expected X[..., D] with a last axis of one element at least: ", x.sizes());
  return x.reshape({-1, x.size(-1)});
}

Tensor norm(const Tensor& x_, const Tensor& w, const Maybe& b, double eps, bool rms) {
  check_transforms({&x_, &w, opt(b)});
  const Tensor x = rows(x_);
  norm_args(x, w, b, eps, rms);
  Tensor y;
  if (wants_grad({&x, &w, opt(b)})) {
    check_capture({&x_, &w, opt(b)});
    y = Norm::apply(x, w, b, eps, rms);
  } else {
    const at::DeviceGuard guard(x.device());
    y = norm_forward(flat(x), flat(w), flat(b), eps, rms, false).y;
  }
  return x_.dim() == 2 ? y : y.reshape(x_.sizes());
}

Tensor linear(const Tensor& x_, const Tensor& w, const Maybe& b, const Maybe& r_, int64_t act) {
  check_transforms({&x_, &w, opt(b), opt(r_)});
  TORCH_CHECK_VALUE(x_.dim() > 0 && w.dim() == 2, "expected X[..., K] and W[N, K]");
  auto shape = x_.sizes().vec();
  shape.back() = w.size(0);
  TORCH_CHECK_VALUE(!there(r_) || r_->sizes() == shape, "residual must be ", shape, ": ", r_->sizes());
  const Tensor x = rows(x_);
  const Maybe r = there(r_) && r_->dim() != 2 ? Maybe(r_->reshape({x.size(0), w.size(0)})) : r_;
  linear_args(x, w, b, r);
  Tensor y;
  if (wants_grad({&x, &w, opt(b), opt(r)})) {
    check_capture({&x_, &w, opt(b), opt(r_)});
    y = Linear::apply(x, w, b, r, act);
  } else {
    const at::DeviceGuard guard(x.device());
    y = linear_forward(flat16(x), flat16(w), flat16(b), flat16(r), act, false).y;
  }
  return x_.dim() == 2 ? y : y.reshape(shape);
}

Tensor feed_forward(const Tensor& x_, const Tensor& nw, const Maybe& nb, const Tensor& w1, const Maybe& b1, const Tensor& w2,
                    const Maybe& b2, int64_t act, double eps, bool rms) {
  check_transforms({&x_, &nw, opt(nb), &w1, opt(b1), &w2, opt(b2)});
  const Tensor x = rows(x_);
  norm_args(x, nw, nb, eps, rms);
  linear_args(x, w1, b1, Maybe());
  TORCH_CHECK_VALUE(w2.dim() == 2 && w2.size(0) == x.size(1) && w2.size(1) == w1.size(0),
                    "expected w1[H,D] and w2[D,H]: w1", w1.sizes(), " w2", w2.sizes());
  TORCH_CHECK_VALUE(!there(b2) || (b2->dim() == 1 && b2->size(0) == x.size(1)), "b2 must be [D]: ", b2->sizes());
  same(x, {&w2, opt(b2)});
  Tensor y;
  if (wants_grad({&x, &nw, opt(nb), &w1, opt(b1), &w2, opt(b2)})) {
    check_capture({&x_, &nw, opt(nb), &w1, opt(b1), &w2, opt(b2)});
    y = FeedForward::apply(x, nw, nb, w1, b1, w2, b2, act, eps, rms);
  } else {
    const at::DeviceGuard guard(x.device());
    const Tensor xf = flat16(x);
    const Tensor n = norm_forward(xf, flat(nw), flat(nb), eps, rms, false).y;
    const Tensor a = linear_forward(n, flat16(w1), flat16(b1), Tensor(), act, false).y;
    y = linear_forward(a, flat16(w2), flat16(b2), xf, SWIGLU_ACT_NONE, false).y;
  }
  return x_.dim() == 2 ? y : y.reshape(x_.sizes());
}

// f without the interpreter's lock; a status becomes the package's exception.
template <class R, class... A>
auto entry(R (*f)(A...)) {
  return torch::wrap_pybind_function([f](A... a) -> R {
    try {
      py::gil_scoped_release release;
      return f(a...);
    } catch (const StatusError& e) {
      const py::object type = py::module_::import("backward_gate_up_amd._lib").attr("SwiGLUError");
      const py::object error = type(e.status, e.where);
      PyErr_SetObject(type.ptr(), error.ptr());
      throw py::error_already_set();
    }
  });
}

}  // namespace

PYBIND11_MODULE(_nodes, m) {
  m.def("norm", entry(&norm));
  m.def("linear", entry(&linear));
  m.def("feed_forward", entry(&feed_forward));
}

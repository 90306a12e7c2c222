// dense.hip -- the C ABI of the norms and of the linear layer (include/swiglu_mlp.h):
// argument checks, size queries and the dispatch to the per-dtype drivers.
#include "checks.hpp"
#include "linear.hpp"

namespace swiglu {

// the drivers are compiled in their own translation units (dense_instantiate.hip)
#define SWIGLU_DECLARE_DENSE(E)                                                        \
  namespace norm {                                                                     \
  extern template int run_fwd<E>(const Args&, bool, hipStream_t);                      \
  extern template int run_bwd<E>(const Args&, bool, void*, void*, hipStream_t);        \
  }                                                                                    \
  namespace lin {                                                                      \
  extern template int run_fwd<E>(const Fwd&);                                          \
  extern template int run_bwd<E>(const Bwd&);                                          \
  }
SWIGLU_DECLARE_DENSE(Bf16)
SWIGLU_DECLARE_DENSE(Fp16)
SWIGLU_DECLARE_DENSE(Fp32)
#undef SWIGLU_DECLARE_DENSE

// Like check_ptrs, for buffers whose rows may start at any element.
static int check_elements(const Range* r, int n, size_t align) {
  for (int i = 0; i < n; ++i)
    if (r[i].n > 0 && !r[i].p) return SWIGLU_ERR_NULL;
  for (int i = 0; i < n; ++i)
    if ((uintptr_t)r[i].p % align) return SWIGLU_ERR_ALIGN;
  return SWIGLU_OK;
}
static int check_apart(const Range* out, int n_out, const Range* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return SWIGLU_ERR_ALIAS;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(out[i], out[j])) return SWIGLU_ERR_ALIAS;
  }
  return SWIGLU_OK;
}
static int check_norm(int64_t T, int64_t D, float eps, int rms) {
  if (T < 0 || T > 0x7fffffffLL || D <= 0 || D > SWIGLU_NORM_MAX_D) return SWIGLU_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > 3.4e38f || rms < 0 || rms > 1) return SWIGLU_ERR_ARG;
  return SWIGLU_OK;
}
static Range optional(const void* p, size_t n) { return {p, p ? n : 0}; }

}  // namespace swiglu

using namespace swiglu;

extern "C" {

size_t swiglu_mlp_norm_stats_bytes(int64_t T, int rms) {
  return T < 0 || T > 0x7fffffffLL ? 0 : (size_t)T * (rms ? 1 : 2) * 4;
}

size_t swiglu_mlp_norm_bwd_workspace_bytes(int64_t T, int64_t D, int rms, int dtype) {
  const size_t e = elt_bytes(dtype);
  if (!e || check_norm(T, D, 0.f, rms)) return 0;
  return norm::bwd_bytes(T, D, rms != 0, e);
}

int swiglu_mlp_norm_fwd(const void* X, const void* weight, const void* bias, void* Y, float* stats, int64_t T, int64_t D,
                        float eps, int rms, int dtype, hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  int rc = check_norm(T, D, eps, rms);
  if (rc) return rc;
  if (rms && bias) return SWIGLU_ERR_ARG;
  const size_t td = (size_t)T * D * e;
  const Range in[] = {{X, td}, {weight, (size_t)D * e}, optional(bias, (size_t)D * e)};
  const Range out[] = {{Y, td}, optional(stats, swiglu_mlp_norm_stats_bytes(T, rms))};
  if ((rc = check_elements(in, 3, e)) || (rc = check_elements(out, 1, e)) || (rc = check_elements(out + 1, 1, 4))) return rc;
  if ((rc = check_apart(out, 2, in, 3)) || (rc = check_device())) return rc;
  if (T == 0) return SWIGLU_OK;
  norm::Args a{};
  a.x = (const char*)X;
  a.w = (const char*)weight;
  a.b = (const char*)bias;
  a.y = (char*)Y;
  a.stats = stats;
  a.T = T;
  a.D = (int)D;
  a.eps = eps;
  a.inv_d = 1.0f / (float)D;
  switch (dtype) {
    case SWIGLU_BF16: return norm::run_fwd<Bf16>(a, rms != 0, stream);
    case SWIGLU_FP16: return norm::run_fwd<Fp16>(a, rms != 0, stream);
    default: return norm::run_fwd<Fp32>(a, rms != 0, stream);
  }
}

int swiglu_mlp_norm_bwd(const void* dY, const void* X, const void* weight, const float* stats, const void* dres, void* dX,
                        void* dweight, void* dbias, void* workspace, size_t workspace_bytes, int64_t T, int64_t D, int rms,
                        int dtype, hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  int rc = check_norm(T, D, 0.f, rms);
  if (rc) return rc;
  if (rms && dbias) return SWIGLU_ERR_ARG;
  const size_t td = (size_t)T * D * e, d = (size_t)D * e, need = swiglu_mlp_norm_bwd_workspace_bytes(T, D, rms, dtype);
  const Range in[] = {{dY, td}, {X, td}, {weight, d}, optional(dres, td), {stats, swiglu_mlp_norm_stats_bytes(T, rms)}};
  const Range out[] = {{dX, td}, {dweight, d}, optional(dbias, d), {workspace, need}};
  if ((rc = check_elements(in, 4, e)) || (rc = check_elements(in + 4, 1, 4)) || (rc = check_elements(out, 3, e))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_apart(out, 4, in, 5)) || (rc = check_device())) return rc;
  norm::Args a{};
  a.x = (const char*)X;
  a.w = (const char*)weight;
  a.y = (char*)dX;
  a.stats = (float*)stats;
  a.dy = (const char*)dY;
  a.dres = (const char*)dres;
  a.partial = (float*)workspace;
  a.T = T;
  a.D = (int)D;
  a.inv_d = 1.0f / (float)D;
  switch (dtype) {
    case SWIGLU_BF16: return norm::run_bwd<Bf16>(a, rms != 0, dweight, dbias, stream);
    case SWIGLU_FP16: return norm::run_bwd<Fp16>(a, rms != 0, dweight, dbias, stream);
    default: return norm::run_bwd<Fp32>(a, rms != 0, dweight, dbias, stream);
  }
}

size_t swiglu_mlp_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype) {
  const size_t e = elt_bytes(dtype);
  if (!e || check_shape(T, N, K, e)) return 0;
  return lin::fwd_bytes(T, N, K, e);
}

int swiglu_mlp_linear_fwd(const void* X, const void* W, const void* bias, const void* residual, void* Y, void* Z,
                          void* workspace, size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int act, int dtype,
                          hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  if (act < 0 || act >= SWIGLU_NUM_ACTS) return SWIGLU_ERR_ARG;
  int rc = check_shape(T, N, K, e);
  if (rc) return rc;
  const size_t tn = (size_t)T * N * e, need = lin::fwd_bytes(T, N, K, e);
  const Range in[] = {{X, (size_t)T * K * e}, {W, (size_t)N * K * e}, optional(bias, (size_t)N * e), optional(residual, tn)};
  const Range out[] = {{Y, tn}, optional(Z, tn), {workspace, need}};
  if ((rc = check_ptrs(in, 4)) || (rc = check_ptrs(out, 2))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_apart(out, 3, in, 4)) || (rc = check_device())) return rc;
  if (T == 0) return SWIGLU_OK;
  const lin::Fwd c{X, W, bias, residual, Y, Z, (char*)workspace, T, N, K, act, stream};
  switch (dtype) {
    case SWIGLU_BF16: return lin::run_fwd<Bf16>(c);
    case SWIGLU_FP16: return lin::run_fwd<Fp16>(c);
    default: return lin::run_fwd<Fp32>(c);
  }
}

size_t swiglu_mlp_linear_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K, int act, int dtype) {
  const size_t e = elt_bytes(dtype);
  if (!e || act < 0 || act >= SWIGLU_NUM_ACTS || check_shape(T, N, K, e)) return 0;
  return lin::bwd_plan(T, N, K, e, act != SWIGLU_ACT_NONE).total;
}

int swiglu_mlp_linear_bwd(const void* dY, const void* X, const void* W, const void* Z, void* dX, void* dW, void* dbias,
                          void* workspace, size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int act, int dtype,
                          hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  if (act < 0 || act >= SWIGLU_NUM_ACTS) return SWIGLU_ERR_ARG;
  int rc = check_shape(T, N, K, e);
  if (rc) return rc;
  const size_t tn = (size_t)T * N * e, tk = (size_t)T * K * e, nk = (size_t)N * K * e;
  const size_t need = swiglu_mlp_linear_bwd_workspace_bytes(T, N, K, act, dtype);
  const Range in[] = {{dY, tn}, {X, X || dW ? tk : 0}, {W, W || dX ? nk : 0}, {Z, act == SWIGLU_ACT_NONE ? 0 : tn}};
  const Range out[] = {optional(dX, tk), optional(dW, nk), optional(dbias, (size_t)N * e), {workspace, need}};
  if ((rc = check_ptrs(in, 4)) || (rc = check_ptrs(out, 3))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_apart(out, 4, in, 4)) || (rc = check_device())) return rc;
  const lin::Bwd c{dY, X, W, Z, dX, dW, dbias, (char*)workspace, T, N, K, act, stream};
  switch (dtype) {
    case SWIGLU_BF16: return lin::run_bwd<Bf16>(c);
    case SWIGLU_FP16: return lin::run_bwd<Fp16>(c);
    default: return lin::run_bwd<Fp32>(c);
  }
}

int swiglu_mlp_linear_plan(int64_t T, int64_t N, int64_t K, int dtype, int dw, int dx, swiglu_linear_plan_t* plan) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  if (!plan) return SWIGLU_ERR_NULL;
  const int rc = check_shape(T, N, K, e);
  if (rc) return rc;
  *plan = swiglu_linear_plan_t{};
  if (!dw && !dx) {
    const bool few = T <= lin::kFewT;
    const lin::Product p = few ? lin::Product{} : lin::fwd_plan(T, N, K, e);
    plan->fwd_engine = few ? 0 : 1 + p.tile;
    plan->fwd_parts = few ? lin::few_splits(T, N, K, e) : p.splits;
    return SWIGLU_OK;
  }
  const lin::Grads g = lin::bwd_plan(T, N, K, e, true).grads[(dw ? 1 : 0) + (dx ? 2 : 0)];
  if (dw) plan->dw_engine = 1 + g.w.tile, plan->dw_parts = g.w.splits;
  if (dx) plan->dx_engine = 1 + g.x.tile, plan->dx_parts = g.x.splits;
  plan->together = g.together;
  return SWIGLU_OK;
}

}  // extern "C"

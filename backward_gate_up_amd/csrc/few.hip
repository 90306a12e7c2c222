// few.hip -- the C ABI of the few-token serving operators: the router, the
// mixture of experts and the products with 4-bit weights (include/swiglu_mlp.h).
#include "checks.hpp"
#include "route.hpp"
#include "w4.hpp"

namespace swiglu {

// the drivers are compiled in their own translation units (few_instantiate.hip)
namespace few {
#define SWIGLU_DECLARE_FEW(E, FMT)                     \
  extern template int run_block<E, FMT>(const Call&);  \
  extern template int run_linear<E, FMT>(const Call&);
SWIGLU_DECLARE_FEW(Bf16, 32)
SWIGLU_DECLARE_FEW(Bf16, 64)
SWIGLU_DECLARE_FEW(Bf16, 128)
SWIGLU_DECLARE_FEW(Fp16, 32)
SWIGLU_DECLARE_FEW(Fp16, 64)
SWIGLU_DECLARE_FEW(Fp16, 128)
#undef SWIGLU_DECLARE_FEW
extern template int run_block<Bf16, 0>(const Call&);
extern template int run_block<Fp16, 0>(const Call&);
extern template int run_block<Fp32, 0>(const Call&);
}  // namespace few
namespace route {
extern template int run_route<Bf16>(Args, hipStream_t);
extern template int run_route<Fp16>(Args, hipStream_t);
extern template int run_route<Fp32>(Args, hipStream_t);
}  // namespace route

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// The kernels address a chunk's up to 64 * 32 rows of either width with 32-bit
// byte offsets.
static bool ld_ok(int64_t v) { return v > 0 && (v & 7) == 0 && v <= SWIGLU_FEW_MAX_D; }

static int check_few(int64_t T, int64_t E, int64_t k) {
  if (T < 0 || T > SWIGLU_FEW_MAX_T) return SWIGLU_ERR_SHAPE;
  if (E < 1 || E > few::kMaxExperts || k < 1 || k > few::kMaxTopK || k > E) return SWIGLU_ERR_SHAPE;
  return SWIGLU_OK;
}

static int check_group(int64_t N, int64_t K, int group) {
  if (group != 32 && group != 64 && group != 128) return SWIGLU_ERR_SHAPE;
  if (!ld_ok(N) || !ld_ok(K) || K % group) return SWIGLU_ERR_SHAPE;
  return SWIGLU_OK;
}
static int check_w4(const swiglu_w4_t* w) {
  if (!w) return SWIGLU_ERR_NULL;
  if (w->experts < 1 || w->experts > few::kMaxExperts) return SWIGLU_ERR_SHAPE;
  return check_group(w->N, w->K, w->group);
}

static Range w4_range(const swiglu_w4_t* w) {
  return {w->data, w4::layout(w->experts, w->N, w->K, w->group, w->has_zeros != 0).total};
}
static few::Weight w4_weight(const swiglu_w4_t* w) {
  return {(const char*)w->data, w4::layout(w->experts, w->N, w->K, w->group, w->has_zeros != 0).expert};
}
static few::Weight row_weight(const void* w, int64_t N, int64_t K, size_t e) {
  return {(const char*)w, (int64_t)(N * K * e)};
}

static int run_block_for(int dtype, int group, const few::Call& c) {
  using namespace few;
  if (group == 0) {
    if (dtype == SWIGLU_BF16) return run_block<Bf16, 0>(c);
    if (dtype == SWIGLU_FP16) return run_block<Fp16, 0>(c);
    return run_block<Fp32, 0>(c);
  }
  if (dtype == SWIGLU_BF16)
    return group == 32 ? run_block<Bf16, 32>(c) : group == 64 ? run_block<Bf16, 64>(c) : run_block<Bf16, 128>(c);
  return group == 32 ? run_block<Fp16, 32>(c) : group == 64 ? run_block<Fp16, 64>(c) : run_block<Fp16, 128>(c);
}
static int run_linear_for(int dtype, int group, const few::Call& c) {
  using namespace few;
  if (dtype == SWIGLU_BF16)
    return group == 32 ? run_linear<Bf16, 32>(c) : group == 64 ? run_linear<Bf16, 64>(c) : run_linear<Bf16, 128>(c);
  return group == 32 ? run_linear<Fp16, 32>(c) : group == 64 ? run_linear<Fp16, 64>(c) : run_linear<Fp16, 128>(c);
}

// Weights and ids of the router are read and written one word at a time.
static int check_words(const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    if (r[i].n > 0 && !r[i].p) return SWIGLU_ERR_NULL;
  for (int i = 0; i < n; ++i)
    if ((uintptr_t)r[i].p & 3) return SWIGLU_ERR_ALIGN;
  return SWIGLU_OK;
}

// Outputs may overlap neither an input nor one another.
static int check_alias(const Range* out, int no, const Range* in, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlap(out[i], in[j])) return SWIGLU_ERR_ALIAS;
    for (int j = i + 1; j < no; ++j)
      if (overlap(out[i], out[j])) return SWIGLU_ERR_ALIAS;
  }
  return SWIGLU_OK;
}

static int run_route_for(int dtype, const route::Args& r, hipStream_t stream) {
  if (dtype == SWIGLU_BF16) return route::run_route<Bf16>(r, stream);
  if (dtype == SWIGLU_FP16) return route::run_route<Fp16>(r, stream);
  return route::run_route<Fp32>(r, stream);
}

// A mixture's workspace: the block's, which is free while the router runs and
// holds its workspace, then the router's weights and ids.
struct MoePlan {
  size_t wts, ids, total;
};
static MoePlan moe_plan(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k, bool w4, size_t e) {
  const size_t p = (size_t)T * k;
  MoePlan m;
  m.wts = few::block_plan(few::shape_of(T, k, E, true, w4, e), T, D, H, k, e).total;
  const size_t r = up256(route::route_bytes(T, D, E, e));
  if (m.wts < r) m.wts = r;
  m.ids = m.wts + up256(p * 4);
  m.total = m.ids + up256(p * 4);
  return m;
}

// The experts' part of a mixture, rows or 4-bit. Wr: NULL, or the router's
// weight [E, D], with which the choices are computed into the workspace first.
static int moe_call(const void* X, const void* Wr, const float* weights, const int32_t* ids, const Range (&w)[3],
                    few::Call& c, void* Y, void* ws, size_t ws_bytes, int64_t T, int64_t k, int renorm, int dtype,
                    int group, hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  const MoePlan m = moe_plan(T, c.D, c.H, c.E, k, group != 0, e);
  const size_t p4 = (size_t)T * k * 4;
  const bool routed = Wr != nullptr;
  const Range in[] = {{X, (size_t)T * c.D * e}, w[0], w[1], w[2], {Wr, routed ? (size_t)c.E * c.D * e : 0},
                      {weights, routed ? 0 : p4}, {ids, routed ? 0 : p4}};
  const Range out[] = {{Y, (size_t)T * c.D * e}, {ws, m.total}};
  int rc;
  if ((rc = check_ptrs(in, 5)) || (rc = check_ptrs(out, 1)) || (rc = check_words(in + 5, 2))) return rc;
  if (m.total > 0 && (!ws || ws_bytes < m.total)) return SWIGLU_ERR_WORKSPACE;
  if (ws && !aligned16(ws)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_alias(out, 2, in, 7))) return rc;
  if ((rc = check_device())) return rc;
  if (T == 0) return SWIGLU_OK;
  c.x = (const char*)X;
  c.y = (char*)Y;
  c.ws = (char*)ws;
  c.T = T;
  c.k = (int)k;
  c.stream = stream;
  c.wts = weights;
  c.ids = ids;
  if (routed) {
    float* rw = (float*)((char*)ws + m.wts);
    int* ri = (int*)((char*)ws + m.ids);
    const route::Args r{(const char*)X, (const char*)Wr, rw, ri, (int)T, (int)c.D, c.E, (int)k, renorm != 0, (float*)ws, 1, 0};
    if ((rc = run_route_for(dtype, r, stream))) return rc;
    c.wts = rw;
    c.ids = ri;
  }
  return run_block_for(dtype, group, c);
}

static int moe_rows(const void* X, const void* Wr, bool routed, const float* weights, const int32_t* ids,
                    const void* Wg, const void* Wu, const void* Wd, void* Y, void* ws, size_t ws_bytes, int64_t T,
                    int64_t D, int64_t H, int64_t E, int64_t k, int renorm, int dtype, hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  if (!ld_ok(D) || !ld_ok(H)) return SWIGLU_ERR_SHAPE;
  int rc = check_few(T, E, k);
  if (rc) return rc;
  if (routed && !Wr) return SWIGLU_ERR_NULL;
  const size_t n = (size_t)E * D * H * e;
  few::Call c{};
  c.wg = row_weight(Wg, H, D, e);
  c.wu = row_weight(Wu, H, D, e);
  c.wd = row_weight(Wd, D, H, e);
  c.D = D;
  c.H = H;
  c.E = (int)E;
  const Range w[3] = {{Wg, n}, {Wu, n}, {Wd, n}};
  return moe_call(X, routed ? Wr : nullptr, weights, ids, w, c, Y, ws, ws_bytes, T, k, renorm, dtype, 0, stream);
}

static int moe_w4(const void* X, const void* Wr, bool routed, const float* weights, const int32_t* ids,
                  const swiglu_w4_t* wg, const swiglu_w4_t* wu, const swiglu_w4_t* wd, void* Y, void* ws,
                  size_t ws_bytes, int64_t T, int64_t k, int renorm, int dtype, hipStream_t stream) {
  if (elt_bytes(dtype) != 2) return SWIGLU_ERR_DTYPE;
  int rc;
  if ((rc = check_w4(wg)) || (rc = check_w4(wu)) || (rc = check_w4(wd))) return rc;
  if (wu->N != wg->N || wu->K != wg->K || wd->N != wg->K || wd->K != wg->N || wu->experts != wg->experts ||
      wd->experts != wg->experts || wu->group != wg->group || wd->group != wg->group || !wu->has_zeros != !wg->has_zeros ||
      !wd->has_zeros != !wg->has_zeros)
    return SWIGLU_ERR_SHAPE;
  if ((rc = check_few(T, wg->experts, k))) return rc;
  if (routed && !Wr) return SWIGLU_ERR_NULL;
  few::Call c{};
  c.wg = w4_weight(wg);
  c.wu = w4_weight(wu);
  c.wd = w4_weight(wd);
  c.D = wg->K;
  c.H = wg->N;
  c.E = wg->experts;
  c.zeros = wg->has_zeros != 0;
  const Range w[3] = {w4_range(wg), w4_range(wu), w4_range(wd)};
  return moe_call(X, routed ? Wr : nullptr, weights, ids, w, c, Y, ws, ws_bytes, T, k, renorm, dtype, wg->group,
                  stream);
}

static dim3 blocks_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return dim3((unsigned)(b < 16384 ? b : 16384));
}

}  // namespace swiglu

using namespace swiglu;

extern "C" {

size_t swiglu_mlp_moe_route_workspace_bytes(int64_t T, int64_t D, int64_t E, int dtype) {
  const size_t e = elt_bytes(dtype);
  if (!e || !ld_ok(D) || check_few(T, E, 1)) return 0;
  return route::route_bytes(T, D, E, e);
}

int swiglu_mlp_moe_route(const void* X, const void* Wr, float* weights, int32_t* ids, void* workspace,
                         size_t workspace_bytes, int64_t T, int64_t D, int64_t E, int64_t k, int renorm, int dtype,
                         hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (!e) return SWIGLU_ERR_DTYPE;
  if (!ld_ok(D)) return SWIGLU_ERR_SHAPE;
  int rc = check_few(T, E, k);
  if (rc) return rc;
  const size_t need = route::route_bytes(T, D, E, e);
  const Range in[] = {{X, (size_t)T * D * e}, {Wr, (size_t)E * D * e}};
  const Range out[] = {{weights, (size_t)T * k * 4}, {ids, (size_t)T * k * 4}, {workspace, need}};
  if ((rc = check_ptrs(in, 2)) || (rc = check_words(out, 2))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_alias(out, 3, in, 2))) return rc;
  if ((rc = check_device())) return rc;
  const route::Args r{(const char*)X, (const char*)Wr, weights, (int*)ids, (int)T, (int)D, (int)E, (int)k, renorm != 0,
                      (float*)workspace, 1, 0};
  return run_route_for(dtype, r, stream);
}

size_t swiglu_mlp_moe_workspace_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k, int dtype) {
  const size_t e = elt_bytes(dtype);
  if (!e || T <= 0 || !ld_ok(D) || !ld_ok(H) || check_few(T, E, k)) return 0;
  // the larger of the two weight formats' plans
  const size_t rows = moe_plan(T, D, H, E, k, false, e).total, w4 = moe_plan(T, D, H, E, k, true, e).total;
  return rows > w4 ? rows : w4;
}

int swiglu_mlp_moe_experts(const void* X, const float* weights, const int32_t* ids, const void* Wg, const void* Wu,
                           const void* Wd, void* Y, void* workspace, size_t workspace_bytes, int64_t T, int64_t D,
                           int64_t H, int64_t E, int64_t k, int dtype, hipStream_t stream) {
  return moe_rows(X, nullptr, false, weights, ids, Wg, Wu, Wd, Y, workspace, workspace_bytes, T, D, H, E, k, 0, dtype,
                  stream);
}

int swiglu_mlp_moe_infer(const void* X, const void* Wr, const void* Wg, const void* Wu, const void* Wd, void* Y,
                         void* workspace, size_t workspace_bytes, int64_t T, int64_t D, int64_t H, int64_t E,
                         int64_t k, int renorm, int dtype, hipStream_t stream) {
  return moe_rows(X, Wr, true, nullptr, nullptr, Wg, Wu, Wd, Y, workspace, workspace_bytes, T, D, H, E, k, renorm,
                  dtype, stream);
}

int swiglu_mlp_moe_experts_w4(const void* X, const float* weights, const int32_t* ids, const swiglu_w4_t* Wg,
                              const swiglu_w4_t* Wu, const swiglu_w4_t* Wd, void* Y, void* workspace,
                              size_t workspace_bytes, int64_t T, int64_t k, int dtype, hipStream_t stream) {
  return moe_w4(X, nullptr, false, weights, ids, Wg, Wu, Wd, Y, workspace, workspace_bytes, T, k, 0, dtype, stream);
}

int swiglu_mlp_moe_infer_w4(const void* X, const void* Wr, const swiglu_w4_t* Wg, const swiglu_w4_t* Wu,
                            const swiglu_w4_t* Wd, void* Y, void* workspace, size_t workspace_bytes, int64_t T,
                            int64_t k, int renorm, int dtype, hipStream_t stream) {
  return moe_w4(X, Wr, true, nullptr, nullptr, Wg, Wu, Wd, Y, workspace, workspace_bytes, T, k, renorm, dtype, stream);
}

size_t swiglu_mlp_w4_bytes(int64_t experts, int64_t N, int64_t K, int group, int has_zeros) {
  if (experts < 1 || experts > few::kMaxExperts || check_group(N, K, group)) return 0;
  return w4::layout(experts, N, K, group, has_zeros != 0).total;
}

int swiglu_mlp_w4_quantize(const void* W, void* codes, void* scales, void* zeros, int64_t experts, int64_t N,
                           int64_t K, int group, int dtype, hipStream_t stream) {
  if (elt_bytes(dtype) != 2) return SWIGLU_ERR_DTYPE;
  if (experts < 1 || experts > few::kMaxExperts) return SWIGLU_ERR_SHAPE;
  int rc = check_group(N, K, group);
  if (rc) return rc;
  const size_t n = (size_t)(experts * N * K), ng = n / group;
  const Range in[] = {{W, n * 2}};
  const Range out[] = {{codes, n / 2}, {scales, ng * 2}, {zeros, zeros ? ng : 0}};
  if ((rc = check_ptrs(in, 1)) || (rc = check_ptrs(out, 3)) || (rc = check_alias(out, 3, in, 1))) return rc;
  if ((rc = check_device())) return rc;
  const int64_t n8 = (int64_t)(n / 8);
  if (dtype == SWIGLU_BF16)
    hipLaunchKernelGGL((w4::w4_quantize<Bf16>), blocks_for(n8), dim3(256), 0, stream, (const __bf16*)W, n8, group,
                       (uint32_t*)codes, (__bf16*)scales, (uint8_t*)zeros);
  else
    hipLaunchKernelGGL((w4::w4_quantize<Fp16>), blocks_for(n8), dim3(256), 0, stream, (const _Float16*)W, n8, group,
                       (uint32_t*)codes, (_Float16*)scales, (uint8_t*)zeros);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

int swiglu_mlp_w4_pack(const void* codes, const void* scales, const void* zeros, void* data, int64_t experts,
                       int64_t N, int64_t K, int group, hipStream_t stream) {
  if (experts < 1 || experts > few::kMaxExperts) return SWIGLU_ERR_SHAPE;
  int rc = check_group(N, K, group);
  if (rc) return rc;
  const w4::Layout l = w4::layout(experts, N, K, group, zeros != nullptr);
  const size_t n = (size_t)(experts * N * K), ng = n / group;
  const Range in[] = {{codes, n / 2}, {scales, ng * 2}, {zeros, zeros ? ng : 0}};
  const Range out[] = {{data, l.total}};
  if ((rc = check_ptrs(in, 3)) || (rc = check_ptrs(out, 1)) || (rc = check_alias(out, 1, in, 3))) return rc;
  if ((rc = check_device())) return rc;
  hipLaunchKernelGGL(w4::w4_pack, blocks_for(experts * l.recs * 64), dim3(256), 0, stream, (const uint8_t*)codes,
                     (const uint16_t*)scales, (const uint8_t*)zeros, (char*)data, l, experts, (int)N, (int)K, group);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

int swiglu_mlp_w4_dequantize(const swiglu_w4_t* w, void* W, int dtype, hipStream_t stream) {
  if (elt_bytes(dtype) != 2) return SWIGLU_ERR_DTYPE;
  int rc = check_w4(w);
  if (rc) return rc;
  const w4::Layout l = w4::layout(w->experts, w->N, w->K, w->group, w->has_zeros != 0);
  const Range in[] = {w4_range(w)};
  const Range out[] = {{W, (size_t)(w->experts * w->N * w->K) * 2}};
  if ((rc = check_ptrs(in, 1)) || (rc = check_ptrs(out, 1)) || (rc = check_alias(out, 1, in, 1))) return rc;
  if ((rc = check_device())) return rc;
  const dim3 b = blocks_for(w->experts * w->N * (w->K / 8));
  if (dtype == SWIGLU_BF16)
    hipLaunchKernelGGL((w4::w4_unpack<Bf16>), b, dim3(256), 0, stream, (const char*)w->data, l, w->has_zeros,
                       w->experts, (int)w->N, (int)w->K, w->group, (__bf16*)W);
  else
    hipLaunchKernelGGL((w4::w4_unpack<Fp16>), b, dim3(256), 0, stream, (const char*)w->data, l, w->has_zeros,
                       w->experts, (int)w->N, (int)w->K, w->group, (_Float16*)W);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

size_t swiglu_mlp_w4_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype) {
  if (elt_bytes(dtype) != 2 || T <= 0 || T > SWIGLU_FEW_MAX_T || !ld_ok(N) || !ld_ok(K)) return 0;
  return few::linear_bytes(T, N, K);
}

int swiglu_mlp_w4_linear(const void* X, const swiglu_w4_t* w, void* Y, void* workspace, size_t workspace_bytes,
                         int64_t T, int dtype, hipStream_t stream) {
  if (elt_bytes(dtype) != 2) return SWIGLU_ERR_DTYPE;
  int rc = check_w4(w);
  if (rc) return rc;
  if (w->experts != 1 || T < 0 || T > SWIGLU_FEW_MAX_T) return SWIGLU_ERR_SHAPE;
  const size_t need = T ? few::linear_bytes(T, w->N, w->K) : 0;
  const Range in[] = {{X, (size_t)T * w->K * 2}, w4_range(w)};
  const Range out[] = {{Y, (size_t)T * w->N * 2}, {workspace, need}};
  if ((rc = check_ptrs(in, 2)) || (rc = check_ptrs(out, 1))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_alias(out, 2, in, 2))) return rc;
  if ((rc = check_device())) return rc;
  if (T == 0) return SWIGLU_OK;
  few::Call c{};
  c.wd = w4_weight(w);
  c.y = (char*)Y;
  c.ws = (char*)workspace;
  c.T = T;
  c.x = (const char*)X;
  c.D = w->N;
  c.H = w->K;
  c.k = 1;
  c.E = 1;
  c.zeros = w->has_zeros != 0;
  c.stream = stream;
  return run_linear_for(dtype, w->group, c);
}

size_t swiglu_mlp_w4_infer_workspace_bytes(int64_t T, int64_t D, int64_t H, int dtype) {
  const size_t e = elt_bytes(dtype);
  if (e != 2 || T <= 0 || T > SWIGLU_FEW_MAX_T || !ld_ok(D) || !ld_ok(H)) return 0;
  return few::block_plan(few::shape_of(T, 1, 1, false, true, 2), T, D, H, 1, e).total;
}

int swiglu_mlp_w4_infer(const void* X, const swiglu_w4_t* wg, const swiglu_w4_t* wu, const swiglu_w4_t* wd, void* Y,
                        void* workspace, size_t workspace_bytes, int64_t T, int dtype, hipStream_t stream) {
  const size_t e = elt_bytes(dtype);
  if (e != 2) return SWIGLU_ERR_DTYPE;
  int rc;
  if ((rc = check_w4(wg)) || (rc = check_w4(wu)) || (rc = check_w4(wd))) return rc;
  if (wu->N != wg->N || wu->K != wg->K || wd->N != wg->K || wd->K != wg->N || wg->experts != 1 || wu->experts != 1 ||
      wd->experts != 1 || wu->group != wg->group || wd->group != wg->group || !wu->has_zeros != !wg->has_zeros ||
      !wd->has_zeros != !wg->has_zeros || T < 0 || T > SWIGLU_FEW_MAX_T)
    return SWIGLU_ERR_SHAPE;
  const size_t td = (size_t)T * wg->K * e;
  const size_t need = few::block_plan(few::shape_of(T, 1, 1, false, true, 2), T, wg->K, wg->N, 1, e).total;
  const Range in[] = {{X, td}, w4_range(wg), w4_range(wu), w4_range(wd)};
  const Range out[] = {{Y, td}, {workspace, need}};
  if ((rc = check_ptrs(in, 4)) || (rc = check_ptrs(out, 1))) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return SWIGLU_ERR_ALIGN;
  if ((rc = check_alias(out, 2, in, 4))) return rc;
  if ((rc = check_device())) return rc;
  if (T == 0) return SWIGLU_OK;
  few::Call c{};
  c.x = (const char*)X;
  c.wg = w4_weight(wg);
  c.wu = w4_weight(wu);
  c.wd = w4_weight(wd);
  c.ws = (char*)workspace;
  c.y = (char*)Y;
  c.T = T;
  c.D = wg->K;
  c.H = wg->N;
  c.k = 1;
  c.E = 1;
  c.zeros = wg->has_zeros != 0;
  c.stream = stream;
  return run_block_for(dtype, wg->group, c);
}

}  // extern "C"

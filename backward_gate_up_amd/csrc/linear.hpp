// linear.hpp -- the linear layer with an epilogue, forward and backward, gfx950.
//
//   forward   z = x W^T + b, y = act(z) + res           x [T, K], W [N, K] (nn.Linear layout)
//   backward  dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum over tokens of dz, dres = dy
//
// The products run on the engines of the SwiGLU block: for many tokens the ring
// of direct-to-LDS loads (16 bits) or the register-staged tiles (fp32, and where
// ring tiles would be too few), for at most 64 tokens a stream of the weight
// through LDS rings (few.hpp's), bound by reading it. Bias, activation and
// residual are applied to the fp32 sums, and y is rounded once. For training the
// sums with their bias are kept besides, rounded to the storage type: the
// backward differentiates at those.
//
// dz is a pass over dy and z of its own, bound by memory, which also forms db's
// sums from the unrounded values. It is rounded to the storage type, which is
// what the matrix instructions take: an error of its own beside that of the
// rounding of dx and dW, 1.4 times theirs alone.
#pragma once
#include "few.hpp"
#include "norm.hpp"

namespace swiglu {
namespace lin {

// ---- few tokens ------------------------------------------------------------------
// Tokens up to which the weight is streamed through LDS rings.
constexpr int kFewT = 64;

struct FewArgs {
  few::Args f;       // x, w0, T, K, N, once
  KArgs e;           // the epilogue: c0, ldc, bias, res, z, act
  int splits;        // workgroups per tile along K
  float* partial;    // splits > 1: [splits][T][N]
};

// y of at most XR tokens. A tile is 16 SH columns. NW / SH groups of waves take
// equal parts of K, and grid y further ones; a group's waves share the token rows
// of one ring (SH > 1) and split the tile's columns. A workgroup walks over tiles,
// its rings running on from one to the next. The groups' sums of a tile meet in
// LDS and are added in order; those of several workgroups (splits > 1) are left
// for lin_join.
template <class E, int XR, int NW, int SH, int RING>
__global__ void __launch_bounds__(NW * 64, (NW == 4 ? 2 : 1)) lin_few(const FewArgs a) {
  constexpr int KG = NW / SH, COLS = 16 * SH;
  using S = few::RowStream<E, 1, XR, SH, RING / KG>;
  constexpr int MT = S::MT;
  const few::Args& g = a.f;
  __shared__ __attribute__((aligned(1024))) char lds[RING];
  __shared__ __attribute__((aligned(16))) float red[NW * MT * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / SH, share = wave % SH;
  const int tiles = (g.N + COLS - 1) / COLS;
  int tile = __builtin_amdgcn_readfirstlane((int)((int64_t)tiles * blockIdx.x / gridDim.x));
  const int last = __builtin_amdgcn_readfirstlane((int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x));
  if (tile >= last) return;
  S st;
  st.init(g, g.x, (uint32_t)g.T * (uint32_t)g.K * E::kBytes, share, lane);
#pragma unroll
  for (int j = 0; j < S::XD; ++j) {
    const int i = st.x_row(j, lane);
    st.token_row(j, i < g.T ? (uint32_t)i * (uint32_t)(g.K * E::kBytes) : kOOB, lane);
  }
  // the group's stages of K: as many for each, those past the end load zeros
  const int stages = S::stages(g.K), parts = a.splits * KG, part = blockIdx.y * KG + group;
  const int per = __builtin_amdgcn_readfirstlane((stages + parts - 1) / parts);
  const int s0 = part * per, s1 = min(stages, s0 + per);
  int get_tile = tile, get_s = s0;
  auto set_weights = [&] { st.weight(0, g.w0, 0, get_tile * COLS + 16 * share, g.N); };
  auto issue = [&](uint32_t slot) {
    st.issue(slot, get_s, get_tile < last && get_s < s1, lane);
    if (++get_s < s0 + per || get_tile >= last) return;
    get_s = s0;
    if (++get_tile < last) set_weights();
  };
  set_weights();
  few::Ring<S, SH> r;
  r.start(lds + group * (RING / KG), issue);
  for (; tile < last; ++tile) {
    f32x4_t acc[1][MT] = {};
#pragma unroll 1
    for (int s = 0; s < per; ++s) r.step(st, acc, lane, issue);
    ring::lds_barrier();  // the last tile's sums have been read
#pragma unroll
    for (int m = 0; m < MT; ++m) *(f32x4_t*)(red + ((wave * MT + m) * 64 + lane) * 4) = acc[0][m];
    ring::lds_barrier();
    // thread -> (token, column): lane l of a block holds column l % 16, tokens 4 (l / 16) + j
    const int rows = min(16 * MT, g.T);
    for (int i = threadIdx.x; i < rows * COLS; i += NW * 64) {
      const int row = i / COLS, col = i % COLS, n = tile * COLS + col;
      if (n >= g.N) continue;
      const int at = ((row >> 4) * 64 + ((row & 15) >> 2) * 16 + (col & 15)) * 4 + (row & 3);
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) v += red[(k * SH + col / 16) * MT * 256 + at];
      const int64_t to = (int64_t)row * g.N + n;
      if (a.splits > 1) {
        a.partial[(int64_t)blockIdx.y * g.T * g.N + to] = v;
        continue;
      }
      using T_ = typename E::elem;
      if (a.e.bias) v += E::to_f32(((const T_*)a.e.bias)[n]);
      if (a.e.z) ((T_*)a.e.z)[to] = E::from_f32(v);
      f32x4_t y{v, 0.f, 0.f, 0.f};
      act4<E::kBytes == 4>(a.e.act, y);
      v = y[0];
      if (a.e.res) v += E::to_f32(((const T_*)a.e.res)[to]);
      ((T_*)a.e.c0)[to] = E::from_f32(v);
    }
  }
  ring::wait_vmcnt<0>();  // no load may land in LDS after the workgroup's end
}

// The epilogue on the sums of the splits' parts, four columns of a token per thread.
template <class E>
__global__ void __launch_bounds__(256) lin_join(const KArgs g, const float* partial, int splits, int64_t quads) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  f32x4_t v{};
  for (int s0 = 0; s0 < splits; s0 += 4) {
    f32x4_t b[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) b[s] = s0 + s < splits ? ((const f32x4_t*)partial)[(s0 + s) * quads + i] : f32x4_t{};
#pragma unroll
    for (int s = 0; s < 4; ++s) v += b[s];
  }
  const int q = g.N / 4;
  linear_store<E>(g, (int)(i / q), (int)(i % q) * 4, v);
}

// ---- dz --------------------------------------------------------------------------
// dz = dy act'(z) and, per strip of rows, the column sums of the unrounded values.
// A lane's piece of 16 bytes of columns; the four waves take every fourth row of
// the strip.
struct DzArgs {
  const char* dy;
  const char* z;    // nullptr: no activation, only the sums
  char* dz;
  float* partial;   // [gridDim.y][N], nullptr: no sums
  int64_t T;
  int N, act;
};
template <class E, int ACT>
__device__ __forceinline__ void dz_rows(const DzArgs& g, int at, int64_t t0, int64_t t1, float (&sum)[16 / E::kBytes]) {
  using P = norm::Piece<E>;
  constexpr int V = P::V;
  const int64_t rowb = (int64_t)g.N * E::kBytes;
#pragma unroll 4
  for (int64_t t = t0; t < t1; t += 4) {
    P dy, z, dz;
    dy.template load<true>(g.dy + t * rowb, at, g.N);
    if constexpr (ACT != SWIGLU_ACT_NONE) z.template load<true>(g.z + t * rowb, at, g.N);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = dy.get(i);
      if constexpr (ACT != SWIGLU_ACT_NONE) {
        v *= act_slope<E::kBytes == 4, ACT>(z.get(i));
        dz.put(i, E::from_f32(v));
      }
      sum[i] += v;
    }
    if constexpr (ACT != SWIGLU_ACT_NONE) dz.template store<true>(g.dz + t * rowb, at, g.N);
  }
}
template <class E>
__global__ void __launch_bounds__(256) lin_dz(const DzArgs g) {
  constexpr int V = 16 / E::kBytes;
  __shared__ float red[4][V][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = (blockIdx.x * 64 + lane) * V;
  const int64_t t0 = g.T * blockIdx.y / gridDim.y + wave, t1 = g.T * (blockIdx.y + 1) / gridDim.y;
  float sum[V] = {};
  if (at < g.N) {
    if (!g.z) dz_rows<E, SWIGLU_ACT_NONE>(g, at, t0, t1, sum);
    else if (g.act == SWIGLU_ACT_RELU) dz_rows<E, SWIGLU_ACT_RELU>(g, at, t0, t1, sum);
    else if (g.act == SWIGLU_ACT_GELU) dz_rows<E, SWIGLU_ACT_GELU>(g, at, t0, t1, sum);
    else if (g.act == SWIGLU_ACT_GELU_TANH) dz_rows<E, SWIGLU_ACT_GELU_TANH>(g, at, t0, t1, sum);
    else dz_rows<E, SWIGLU_ACT_SILU>(g, at, t0, t1, sum);
  }
  if (!g.partial) return;
#pragma unroll
  for (int i = 0; i < V; ++i) red[wave][i][lane] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * V; i += 256) {
    const int n = blockIdx.x * 64 * V + i, l = i / V, e = i % V;
    if (n < g.N) g.partial[(int64_t)blockIdx.y * g.N + n] = ((red[0][e][l] + red[1][e][l]) + red[2][e][l]) + red[3][e][l];
  }
}
static inline int dz_strips(int64_t T, int64_t N, size_t e) {
  const int64_t cols = (N * (int64_t)e + 1023) / 1024;  // workgroups per strip
  int64_t s = (8 * dev_ncu() + cols - 1) / cols;
  const int64_t most = (T + 15) / 16;  // four rows per wave at least
  if (s > most) s = most;
  return s < 1 ? 1 : s > 256 ? 256 : (int)s;
}

// ---- plans -------------------------------------------------------------------------
struct Fwd {
  const void *x, *w, *bias, *res;
  void *y, *z;
  char* ws;
  int64_t T, N, K;
  int act;
  hipStream_t stream;
};
struct Bwd {
  const void *dy, *x, *w, *z;
  void *dx, *dw, *db;
  char* ws;
  int64_t T, N, K;
  int act;
  hipStream_t stream;
};

// At most 16 tokens: one workgroup of many waves per CU where there are few tiles
// of 16 columns, else two of four. More: tiles of 64 columns, K split over
// workgroups until every CU has one, each part 6 stages at least.
static inline int few_splits(int64_t T, int64_t N, int64_t K, size_t e) {
  if (T <= 16) return 1;
  const int64_t tiles = (N + 63) / 64, most = (K * (int64_t)e + 127) / 128 / 12;
  int64_t s = dev_ncu() / tiles;
  if (s > most) s = most;
  return s < 2 ? 1 : s > 16 ? 16 : (int)s;
}
static inline size_t fwd_bytes(int64_t T, int64_t N, int64_t K, size_t e) {
  if (T <= 0 || T > kFewT) return 0;
  const int s = few_splits(T, N, K, e);
  return s > 1 ? (size_t)s * T * N * 4 : 0;
}

// Backward workspace: dz, then the column sums' parts or (they come one after the
// other) the weight gradient's parts, each 256-byte aligned.
static inline bool ring_dw(int64_t T, size_t e) { return e == 2 && T > 512; }
struct BwdPlan {
  size_t sums, total;
  int strips;
};
static inline BwdPlan bwd_plan(int64_t T, int64_t N, int64_t K, size_t e, bool act) {
  BwdPlan p{};
  p.strips = dz_strips(T, N, e);
  p.sums = act ? align256((size_t)T * N * e) : 0;
  size_t parts = (size_t)p.strips * N * 4;
  if (ring_dw(T, e)) {
    const WgradPlan w = wgrad_plan(cdiv(N, 256) * cdiv(K, 256), T, dev_ncu(), wgrad_bk<STAGE_LINEAR_DW>());
    const size_t b = (size_t)w.n_split * w.ksplit * 65536 * 4;
    if (b > parts) parts = b;
  }
  p.total = p.sums + align256(parts);
  return p;
}

static inline KArgs fwd_args(const Fwd& c) {
  KArgs a{};
  a.a0 = opnd(c.x, c.K, c.T, c.K);
  a.b0 = opnd(c.w, c.K, c.N, c.K);
  a.c0 = (char*)c.y;
  a.ldc = c.N;
  a.M = (int)c.T;
  a.N = (int)c.N;
  a.bias = (const char*)c.bias;
  a.res = (const char*)c.res;
  a.z = (char*)c.z;
  a.act = c.act;
  return a;
}

// ---- many tokens, 16 bits: the ring, its activation fixed at compile time -----------
template <class E, int ACT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) lin_ring(const KArgs g) {
  SWIGLU_RING_LDS(true)
  ring5_tile<E, KC, KC, LINEAR, ACT>(g, R, blockIdx.x, 0);
}
template <class E, int ACT>
int launch_lin_ring(KArgs a, hipStream_t s) {
  a.group_m = 2;
  StageScope scope(STAGE_LINEAR, s);
  hipLaunchKernelGGL((lin_ring<E, ACT>), dim3(a.tiles_m * a.tiles_n), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}
#define SWIGLU_LIN_RING_DECL(PREFIX, E)                                       \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_NONE>(KArgs, hipStream_t);      \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_RELU>(KArgs, hipStream_t);      \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_GELU>(KArgs, hipStream_t);      \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_GELU_TANH>(KArgs, hipStream_t); \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_SILU>(KArgs, hipStream_t);

template <class E, int XR, int NW, int SH, int RING>
static int launch_few(const FewArgs& a, int grid, hipStream_t s) {
  StageScope scope(STAGE_LINEAR, s);
  hipLaunchKernelGGL((lin_few<E, XR, NW, SH, RING>), dim3(grid, a.splits), dim3(NW * 64), 0, s, a);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}
template <class E, int XR>
static int few_own(const FewArgs& a, hipStream_t s) {
  const int tiles = cdiv(a.f.N, 16), ncu = dev_ncu();
  if (tiles <= ncu) return launch_few<E, XR, 16, 1, 131072>(a, tiles, s);
  const int fit = 2 * ncu;
  return launch_few<E, XR, 4, 1, 65536>(a, tiles < fit ? tiles : fit, s);
}

// Tiles of 64 rows: the widest that still gives every CU one.
template <class E, int AL, int BL, int KIND, int STAGE>
static int launch_rows64(KArgs a, hipStream_t s) {
  a.tiles_m = cdiv(a.M, 64);
  if (a.tiles_m * cdiv(a.N, 256) >= dev_ncu()) {
    a.tiles_n = cdiv(a.N, 256);
    return launch<E, 64, 256, AL, BL, KIND, STAGE>(a, 1, s);
  }
  if (a.tiles_m * cdiv(a.N, 128) >= dev_ncu()) {
    a.tiles_n = cdiv(a.N, 128);
    return launch<E, 64, 128, AL, BL, KIND, STAGE>(a, 1, s);
  }
  a.tiles_n = cdiv(a.N, 64);
  return launch<E, 64, 64, AL, BL, KIND, STAGE>(a, 1, s);
}

template <class E>
int run_fwd(const Fwd& c) {
  KArgs a = fwd_args(c);
  if (c.T <= kFewT) {
    FewArgs f{};
    f.f.x = (const char*)c.x;
    f.f.w0 = few::Weight{(const char*)c.w, 0};
    f.f.T = (int)c.T;
    f.f.N = (int)c.N;
    f.f.K = (int)c.K;
    f.f.once = c.K * E::kBytes % 128 == 0;
    f.e = a;
    f.splits = few_splits(c.T, c.N, c.K, E::kBytes);
    f.partial = (float*)c.ws;
    if (c.T <= 8) return few_own<E, 8>(f, c.stream);
    if (c.T <= 16) return few_own<E, 16>(f, c.stream);
    const int rc = launch_few<E, 64, 8, 4, 122880>(f, cdiv(c.N, 64), c.stream);
    if (rc || f.splits == 1) return rc;
    StageScope scope(STAGE_LINEAR, c.stream);
    const int64_t quads = c.T * c.N / 4;
    hipLaunchKernelGGL((lin_join<E>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, c.stream, a,
                       (const float*)f.partial, f.splits, quads);
    return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
  }
  if constexpr (E::kBytes == 2) {
    a.tiles_m = cdiv(c.T, 256);
    a.tiles_n = cdiv(c.N, 256);
    // (64-row tiles where those fit one round on the CUs, as in the SwiGLU block)
    if (c.T > 512 && cdiv(c.T, 64) * a.tiles_n > dev_ncu()) {
      switch (c.act) {
        case SWIGLU_ACT_RELU: return launch_lin_ring<E, SWIGLU_ACT_RELU>(a, c.stream);
        case SWIGLU_ACT_GELU: return launch_lin_ring<E, SWIGLU_ACT_GELU>(a, c.stream);
        case SWIGLU_ACT_GELU_TANH: return launch_lin_ring<E, SWIGLU_ACT_GELU_TANH>(a, c.stream);
        case SWIGLU_ACT_SILU: return launch_lin_ring<E, SWIGLU_ACT_SILU>(a, c.stream);
        default: return launch_lin_ring<E, SWIGLU_ACT_NONE>(a, c.stream);
      }
    }
  }
  return launch_rows64<E, KC, KC, LINEAR, STAGE_LINEAR>(a, c.stream);
}

template <class E>
int run_bwd(const Bwd& c) {
  const BwdPlan p = bwd_plan(c.T, c.N, c.K, E::kBytes, c.act != SWIGLU_ACT_NONE);
  const char* dz = (const char*)c.dy;
  float* parts = (float*)(c.ws + p.sums);
  const bool act = c.act != SWIGLU_ACT_NONE;
  if (c.db || (act && (c.dx || c.dw))) {
    StageScope scope(STAGE_LINEAR_DZ, c.stream);
    DzArgs d{(const char*)c.dy, act ? (const char*)c.z : nullptr, act ? c.ws : nullptr, c.db ? parts : nullptr,
             c.T, (int)c.N, c.act};
    if (act) dz = c.ws;
    hipLaunchKernelGGL((lin_dz<E>), dim3((unsigned)((c.N * E::kBytes + 1023) / 1024), p.strips), dim3(256), 0, c.stream, d);
    if (hipGetLastError() != hipSuccess) return SWIGLU_ERR_LAUNCH;
    if (c.db) {
      const int rc = norm::launch_sum_parts<E>(parts, p.strips, 1, c.N, c.db, nullptr, c.stream);
      if (rc) return rc;
    }
  }
  if (c.dw) {
    KArgs a{};  // dW [N, K]: rows dz^T, columns x, summed over tokens
    a.a0 = opnd(dz, c.N, c.N, c.T);
    a.b0 = opnd(c.x, c.K, c.K, c.T);
    a.c0 = (char*)c.dw;
    a.ldc = c.K;
    a.M = (int)c.N;
    a.N = (int)c.K;
    int rc = SWIGLU_OK;
    bool done = false;
    if constexpr (E::kBytes == 2) {
      if (ring_dw(c.T, E::kBytes)) {
        a.tiles_m = cdiv(a.M, 256);
        a.tiles_n = cdiv(a.N, 256);
        rc = launch_ring_wgrad<E, MC, MC, STAGE_LINEAR_DW>(a, 1, parts, c.stream);
        done = true;
      }
    }
    if (!done) rc = launch_rows64<E, MC, MC, PLAIN, STAGE_LINEAR_DW>(a, c.stream);
    if (rc) return rc;
  }
  if (c.dx) {
    KArgs a{};  // dx [T, K]: rows dz, columns of W, summed over N
    a.a0 = opnd(dz, c.N, c.T, c.N);
    a.b0 = opnd(c.w, c.K, c.K, c.N);
    a.c0 = (char*)c.dx;
    a.ldc = c.K;
    a.M = (int)c.T;
    a.N = (int)c.K;
    if constexpr (E::kBytes == 2) {
      a.tiles_m = cdiv(c.T, 256);
      a.tiles_n = cdiv(c.K, 256);
      if (c.T > 512 && cdiv(c.T, 64) * a.tiles_n > dev_ncu())
        return launch_ring<E, KC, MC, PLAIN, STAGE_LINEAR_DX>(a, 1, c.stream);
    }
    return launch_rows64<E, KC, MC, PLAIN, STAGE_LINEAR_DX>(a, c.stream);
  }
  return SWIGLU_OK;
}

}  // namespace lin
}  // namespace swiglu

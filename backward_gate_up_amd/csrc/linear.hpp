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
// for lin_join. Bound by reading the weight: T = 1, N = 11008, K = 4096, bf16 18.8 us,
// 4.8 TB/s from HBM (a 2 GiB copy 4.9); T = 33, N = 4096, K = 11008, fp16 20.3 us in
// four parts of K, and 4.0 to join them.
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

// The epilogue on the sums of parts, 16 bytes of a row's outputs per thread, for one
// or two products (na and nb such pieces).
template <class E>
__global__ void __launch_bounds__(256) lin_join(const KArgs a, const KArgs b, int64_t na, int64_t nb) {
  constexpr int V = 16 / E::kBytes;
  const int64_t blocks = (na + 255) / 256;
  const bool second = blockIdx.x >= blocks;
  const KArgs& g = second ? b : a;
  const int64_t pieces = second ? nb : na, i = (blockIdx.x - (second ? blocks : 0)) * 256 + threadIdx.x;
  if (i >= pieces) return;
  float z[V] = {};
  const f32x4_t* at = (const f32x4_t*)(g.P + i * V);
  for (int s0 = 0; s0 < g.ksplit; s0 += 4) {
    f32x4_t p[4][V / 4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int q = 0; q < V / 4; ++q) p[s][q] = s0 + s < g.ksplit ? at[(s0 + s) * (pieces * V / 4) + q] : f32x4_t{};
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int e = 0; e < V; ++e) z[e] += p[s][e / 4][e % 4];
  }
  const int q = g.N / V;
  linear_store<E>(g, (int)(i / q), (int)(i % q) * V, z);
}

// ---- dz --------------------------------------------------------------------------
// dz = dy act'(z) and, per strip of rows, the column sums of the unrounded values.
// A lane's piece of 16 bytes of columns; the four waves take every fourth row of
// the strip. Bound by memory: 16384 x 11008 bf16, gelu, 225 us, 4.8 TB/s.
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
// The same with all rows in one workgroup of sixteen waves per 128 bytes of columns,
// which writes db itself: up to kDzRows rows one launch less is worth more than
// the strips. A thread has at most four rows, one after another and the next one's
// loads ahead: with the rows unrolled the code is four times as long, and a
// launch this short waits for its instructions (T = 300, N = 712, fp16 9.8 -> 6.1
// us).
constexpr int kDzRows = 512;
template <class E, int ACT>
__device__ __forceinline__ void dz_few_rows(const DzArgs& g, int at, int first, float (&sum)[16 / E::kBytes]) {
  using P = norm::Piece<E>;
  constexpr int V = P::V;
  const int64_t rowb = (int64_t)g.N * E::kBytes;
  P dy, z;
  auto load = [&](int64_t row) {
    if (row >= g.T) return;
    dy.template load<true>(g.dy + row * rowb, at, g.N);
    if constexpr (ACT != SWIGLU_ACT_NONE) z.template load<true>(g.z + row * rowb, at, g.N);
  };
  load(first);
#pragma unroll 1
  for (int64_t row = first; row < g.T; row += 128) {
    const P d = dy, y = z;
    load(row + 128);
    P dz;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = d.get(i);
      if constexpr (ACT != SWIGLU_ACT_NONE) {
        v *= act_slope<E::kBytes == 4, ACT>(y.get(i));
        dz.put(i, E::from_f32(v));
      }
      sum[i] += v;
    }
    if constexpr (ACT != SWIGLU_ACT_NONE) dz.template store<true>(g.dz + row * rowb, at, g.N);
  }
}
template <class E>
__global__ void __launch_bounds__(1024) lin_dz_few(const DzArgs g, char* db) {
  constexpr int V = 16 / E::kBytes, C = 8 * V;  // columns
  __shared__ float red[128][C + 1];
  const int lane = threadIdx.x & 7, row = threadIdx.x >> 3;
  const int at = (blockIdx.x * 8 + lane) * V;
  float sum[V] = {};
  if (at < g.N) {
    if (!g.z) dz_few_rows<E, SWIGLU_ACT_NONE>(g, at, row, sum);
    else if (g.act == SWIGLU_ACT_RELU) dz_few_rows<E, SWIGLU_ACT_RELU>(g, at, row, sum);
    else if (g.act == SWIGLU_ACT_GELU) dz_few_rows<E, SWIGLU_ACT_GELU>(g, at, row, sum);
    else if (g.act == SWIGLU_ACT_GELU_TANH) dz_few_rows<E, SWIGLU_ACT_GELU_TANH>(g, at, row, sum);
    else dz_few_rows<E, SWIGLU_ACT_SILU>(g, at, row, sum);
  }
  if (!db) return;
#pragma unroll
  for (int i = 0; i < V; ++i) red[row][lane * V + i] = sum[i];
  __syncthreads();
  // eight rows' sums per thread, then the sixteen of a column
  const int c = threadIdx.x % C, p = threadIdx.x / C, n = blockIdx.x * C + c;
  float v = 0.f;
  if (p < 16) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v += red[p * 8 + r][c];
  }
  __syncthreads();
  if (p < 16) red[p][c] = v;
  __syncthreads();
  if (p == 0 && n < g.N) {
    v = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) v += red[r][c];
    ((typename E::elem*)db)[n] = E::from_f32(v);
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

// How a product [M, N] over K runs: on register-staged tiles, several workgroups
// per CU, or (16 bits) on the ring of 256 x 256 tiles, one per CU, which is the
// fastest where there are enough of them; with K split where there are too few
// tiles for the CUs, the parts being joined by a second launch. The ring's tiles
// are split where at least two parts of each find a CU (128 tiles of K = 5632 110 ->
// 90 us); to split the tiles of a last, partly filled round is slower, whose CUs
// clock higher instead (688 tiles of K = 16384 1098 us, the last 176 in four parts
// 1169).
//
// Chosen by the time of a model in us: r tiles that a CU runs at once (at most
// `most`) take fix r + K max(lat, thr r), parts of K a launch and a pass over them
// more. The figures were fitted to the times of 7 thousand products of random
// sizes (65 to 16384 by 256 to 11008, all three layouts), each on several tiles in 1
// to 16 parts. With the tiles' loads two stages ahead they are 5 to 15 % long for
// them, which changes no choice by much: what is chosen takes 1.5 % longer than the
// best of what was timed in the geometric mean over nine thousand others, and with
// figures fitted again 0.3 % less. 235 of those are more than 15 % behind, 41 more
// than 25: 49 with a short K and a large output, where the ring is taken for tiles up
// to 46 % faster (ring_us has no term for its outputs, which no other tile of a CU
// covers; 15773 x 10712 over 368 317 us, 128 x 128 tiles 218); 52 with a long K and a
// narrow output, where it is not (below 64 of its tiles it is left out; 4403 x 712 over
// 8536 103 us, the ring in four parts 73); else products of tiles of 10 to 30 us.
// fp32 has only 64 x 64: wider ones were behind at every
// size but the largest, by 3 % there (M = N = 2000, K = 8000 503 against 487 us).
// What the choice is worth (us, unsplit 64 x 64 / 128 x 128 / best split; bf16): 256
// x 1024, K = 8192 62 / 88 / 17.5; 4096 x 2048, K = 5632 154 / 105 / 97 (ring); 4096
// x 5632, K = 2048 164 / 118, ring 96.
enum { T64 = 0, T64x128 = 1, T128 = 2, TRING = 3 };
struct Product {
  int tile, splits, kchunk;  // kchunk: K values per part (ring: stages)
  double us;
};
struct TileCost {
  int bm, bn, most;
  double lat, thr, fix;
  // a CU's share of r tiles over a K
  double us(double r, double k) const {
    const double rounds = (double)(int64_t)(r / most), rest = r - rounds * most;
    auto one = [&](double n) { return n > 0 ? (lat > thr * n ? lat : thr * n) : 0.0; };
    return fix * r + k * (rounds * one(most) + one(rest));
  }
};
static inline TileCost tile_cost(int tile, size_t e) {
  if (e == 4) return {64, 64, 4, 19.1e-3, 16.0e-3, 0.72};
  if (tile == T64) return {64, 64, 4, 6.4e-3, 4.0e-3, 0.38};
  if (tile == T64x128) return {64, 128, 2, 8.7e-3, 5.8e-3, 1.2};
  return {128, 128, 2, 10.9e-3, 8.1e-3, 2.2};
}
// n ring tiles over k, one per CU at a time. The clock falls under the power limit as
// the CUs fill and with the length of the tiles (a full round of K = 2048 47.5 us,
// 4096 93, 11008 249, 16384 366; a quarter of one of K = 8425 134).
static inline double ring_us(int64_t n, double k, int ncu) {
  const double fix = 13.4, least = 12.5e-3, full = 17.0e-3 + 4.5e-7 * (k < 1e4 ? k : 1e4);
  const double rest = (double)(n % ncu) / ncu;
  return (double)(n / ncu) * (fix + k * full) + (rest > 0 ? fix + k * (least + rest * (full - least)) : 0);
}
// Writing and reading fp32 parts, and the launch that joins them.
static inline double join_us(double values) { return 5.0 + values * 1.0e-6; }
static Product plan_product(int64_t M, int64_t N, int64_t K, size_t e) {
  const int ncu = dev_ncu(), bk = e == 4 ? 32 : 64, nk = K > 0 ? cdiv(K, bk) : 1;
  Product best{};
  best.us = 1e30;
  for (int tile = T64; tile <= (e == 4 ? T64 : T128); ++tile) {
    const TileCost c = tile_cost(tile, e);
    const int64_t n = (int64_t)cdiv(M, c.bm) * cdiv(N, c.bn);
    for (int s = 1; s <= 16 && (s == 1 || (nk / s >= 4 && n * s <= 8 * ncu)); ++s) {
      const int per = cdiv(nk, s), parts = cdiv(nk, per);
      if (parts != s) continue;
      const double us = c.us((double)((n * s + ncu - 1) / ncu), (double)per * bk) + (s > 1 ? join_us((double)s * M * N) : 0);
      if (us < best.us) best = {tile, s, per * bk, us};
    }
  }
  if (e == 4) return best;
  const int64_t nt = (int64_t)cdiv(M, 256) * cdiv(N, 256);
  if (4 * nt < ncu) return best;
  for (int s = 1; s <= 4 && (s == 1 || (nt * s <= ncu && nk / s >= 8)); ++s) {
    const int per = cdiv(nk, s), parts = cdiv(nk, per);
    if (parts != s) continue;
    const double us = ring_us(nt * s, (double)per * bk, ncu) + (s > 1 ? join_us((double)nt * s * 65536) : 0);
    if (us < best.us) best = {TRING, s, per, us};
  }
  return best;
}
static inline size_t product_bytes(const Product& p, int64_t M, int64_t N) {
  if (p.splits == 1) return 0;
  return (size_t)p.splits * 4 * (p.tile == TRING ? (size_t)cdiv(M, 256) * cdiv(N, 256) * 65536 : (size_t)M * N);
}
// The backward's two products, dW [N, K] over T and dx [T, K] over N. Both in one
// launch, so that the short tiles of one fill the CUs that the other's last round
// leaves: on the ring, or on 64 x 64 tiles, where it also saves a launch, the longer
// tiles first either way; or each on its own as above. T = 4096, N = 2048, K = 5632,
// bf16, 176 ring tiles over 4096 and 352 over 2048: 157 us, apart 91 and 95; over
// four thousand random sizes 0.80 of the time of the two apart.
struct Grads {
  bool together, ring;
  Product w, x;
};
static Grads plan_grads(int64_t T, int64_t N, int64_t K, size_t e, bool dw, bool dx) {
  Grads g{};
  if (dw) g.w = plan_product(N, K, T, e);
  if (dx) g.x = plan_product(T, K, N, e);
  if (!dw || !dx || T == 0) return g;
  // (a launch; fp32 always both in one, 1.5 % shorter over 160 sizes, 15 % at best and 3 %
  // longer at worst, where the model's choice left half of that)
  double best = e == 4 ? 1e30 : g.w.us + g.x.us + 4.7;
  const int ncu = dev_ncu();
  {
    // 64 x 64 tiles together, whole or in as many parts as give two per CU
    const TileCost c = tile_cost(T64, e);
    const int bk = e == 4 ? 32 : 64;
    auto split = [&](int64_t M, int64_t n_cols, int64_t len, bool parts) {
      const int nk = cdiv(len, bk);
      const int64_t n = (int64_t)cdiv(M, 64) * cdiv(n_cols, 64);
      Product p{T64, 1, nk * bk, 0};
      for (int s = 2; parts && s <= 16 && nk / s >= 4 && n * s <= 2 * ncu; ++s) {
        const int per = cdiv(nk, s);
        if (cdiv(nk, per) == s) p = {T64, s, per * bk, 0};
      }
      return p;
    };
    const double nw = (double)cdiv(N, 64) * cdiv(K, 64), nx = (double)cdiv(T, 64) * cdiv(K, 64);
    const double load = c.thr * (nw * T + nx * N) / ncu + c.fix * (nw + nx) / ncu;
    for (int parts = 0; parts < 2; ++parts) {
      const Product w = split(N, K, T, parts), x = split(T, K, N, parts);
      const double lat = c.lat * (w.kchunk > x.kchunk ? w.kchunk : x.kchunk);
      const double v = (w.splits > 1 ? (double)w.splits * N * K : 0) + (x.splits > 1 ? (double)x.splits * T * K : 0);
      // (neither the work nor the longest tile alone: the short tiles wait for the long ones' CUs)
      const double us = 1.1 * (load > lat ? load + 0.5 * lat : lat + 0.5 * load) + (v > 0 ? join_us(v) : 0);
      if (us < best) {
        best = us;
        g = {true, false, w, x};
      }
    }
  }
  if (e == 2) {
    const int64_t nw = (int64_t)cdiv(N, 256) * cdiv(K, 256), nx = (int64_t)cdiv(T, 256) * cdiv(K, 256);
    // a tiles of length l first, then b of length s
    const int64_t a = T >= N ? nw : nx, b = T >= N ? nx : nw;
    const double l = ring_us(ncu, T >= N ? T : N, ncu), s = ring_us(ncu, T >= N ? N : T, ncu);
    // (all CUs busy until the last tiles, which start half a short one late)
    const double work = (a * l + b * s) / ncu + 0.5 * s, longest = (double)((a + ncu - 1) / ncu) * l;
    const double us = work > longest ? work : longest;
    // (the two together run 3 to 5 % slower than each alone at its best: their panels share L2)
    if (nw + nx >= ncu && 1.05 * us < best) {
      best = us;
      g = {true, true, Product{TRING, 1, 0, 0}, Product{TRING, 1, 0, 0}};
    }
  }
  return g;
}

// Plans by their sizes: a model calls with the same few, and a plan takes about as
// long as a launch.
template <class P>
struct Plans {
  struct Key {
    int64_t T = -1, N = 0, K = 0, form = 0;
    bool operator==(const Key& o) const { return T == o.T && N == o.N && K == o.K && form == o.form; }
  };
  static constexpr int kSlots = 64;
  Key key[kSlots];
  P plan[kSlots];
  template <class Make>
  const P& get(int64_t T, int64_t N, int64_t K, int64_t form, Make&& make) {
    Key k;
    k.T = T;
    k.N = N;
    k.K = K;
    k.form = form * 4096 + dev_ncu();
    const int i = (int)(((uint64_t)(T * 31 + N * 7 + K * 3 + form) * 0x9E3779B97F4A7C15ull) >> 58);
    if (!(key[i] == k)) {
      plan[i] = make();
      key[i] = k;
    }
    return plan[i];
  }
};
static inline Product fwd_plan(int64_t T, int64_t N, int64_t K, size_t e) {
  static thread_local Plans<Product> plans;
  return plans.get(T, N, K, (int64_t)e, [&] { return plan_product(T, N, K, e); });
}
static inline size_t fwd_bytes(int64_t T, int64_t N, int64_t K, size_t e) {
  if (T <= 0) return 0;
  if (T > kFewT) return product_bytes(fwd_plan(T, N, K, e), T, N);
  const int s = few_splits(T, N, K, e);
  return s > 1 ? (size_t)s * T * N * 4 : 0;
}

// Backward workspace: dz, then the column sums' parts or (they come one after the
// other) the products' parts, each 256-byte aligned. grads: by what is wanted, 1
// dW, 2 dx, 3 both.
struct BwdPlan {
  size_t parts, total;
  int strips;
  Grads grads[4];
};
static BwdPlan make_bwd_plan(int64_t T, int64_t N, int64_t K, size_t e, bool act) {
  BwdPlan p{};
  p.strips = T <= kDzRows ? 0 : dz_strips(T, N, e);
  p.parts = act ? align256((size_t)T * N * e) : 0;
  size_t most = (size_t)p.strips * N * 4;
  for (int wants = 1; wants <= 3; ++wants) {
    const Grads g = p.grads[wants] = plan_grads(T, N, K, e, wants & 1, wants & 2);
    const size_t w = wants & 1 ? align256(product_bytes(g.w, N, K)) : 0;
    const size_t b = w + (wants & 2 ? product_bytes(g.x, T, K) : 0);
    if (b > most) most = b;
  }
  p.total = p.parts + align256(most);
  return p;
}
static inline BwdPlan bwd_plan(int64_t T, int64_t N, int64_t K, size_t e, bool act) {
  static thread_local Plans<BwdPlan> plans;
  return plans.get(T, N, K, (int64_t)e * 2 + act, [&] { return make_bwd_plan(T, N, K, e, act); });
}

// ---- launches ------------------------------------------------------------------------
// A product on register-staged tiles: LINEAR's epilogue, or its parts. fp32, T = 1000, N
// = 2816, K = 1024, gelu: 62 to 65 us, 92 TFLOP/s on 2.75 tiles per CU; 1024 x 4096 x 4096
// 249 us, 138 (the library's 8192^3 152). fp16, T = 300, N = 712, K = 1000 11 us: latency.
template <class E, int BM, int BN, int AL, int BL, int STAGE>
__global__ void __launch_bounds__(256, (BM == 64 && BN == 64 ? 3 : 2)) lin_tile(const KArgs g) {
  __shared__ __attribute__((aligned(16))) char smem[Geometry<E, BM, BN, AL, BL>::LDS];
  const int nt = g.tiles_m * g.tiles_n, b = blockIdx.x;
  gemm_tile<E, BM, BN, AL, BL, LINEAR>(g, smem, b % nt, b / nt);
}
// dW and dx on 64 x 64 tiles, the longer ones first.
template <class E>
__global__ void __launch_bounds__(256, 3) lin_tile_grads(const KArgs w, const KArgs x, int x_first) {
  constexpr int LW = Geometry<E, 64, 64, MC, MC>::LDS, LX = Geometry<E, 64, 64, KC, MC>::LDS;
  __shared__ __attribute__((aligned(16))) char smem[LW > LX ? LW : LX];
  const int nw = w.tiles_m * w.tiles_n, nx = x.tiles_m * x.tiles_n, b = blockIdx.x;
  const int bw = b - (x_first ? nx * x.ksplit : 0), bx = b - (x_first ? 0 : nw * w.ksplit);
  if (x_first ? bw >= 0 : bx < 0) gemm_tile<E, 64, 64, MC, MC, LINEAR>(w, smem, bw % nw, bw / nw);
  else gemm_tile<E, 64, 64, KC, MC, LINEAR>(x, smem, bx % nx, bx / nx);
}

// The ring, whole tiles with the epilogue. T = 16384, N = 11008, K = 4096, bf16, gelu
// with z kept: 1164 us, 1270 TFLOP/s (dW 1090 and dx 955 us, 1356 and 1547; a plain
// 8192^3 product of the library 1365).
template <class E, int ACT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) lin_ring(const KArgs g) {
  SWIGLU_RING_LDS(true)
  ring5_tile<E, KC, KC, LINEAR, ACT>(g, R, blockIdx.x, 0);
}
// Parts of its tiles, workgroup i being part i % ksplit of tile i / ksplit. (A kernel
// that ended in either the epilogue or a part's sums spilled accumulators: 1210 us
// became 1314.)
template <class E>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) lin_ring_parts(const KArgs g) {
  SWIGLU_RING_LDS(true)
  const int i = blockIdx.x;
  ring5_tile<E, KC, KC, PLAIN>(g, R, i / g.ksplit, 0, i % g.ksplit, i);
}
// dx, whole tiles or parts. (The host pass of the compiler refuses to instantiate
// this tile from two kernels.)
template <class E>
__device__ __forceinline__ void dx_tile(const KArgs& g, char* const (&R)[5], int item, int ks, int piece) {
  ring5_tile<E, KC, MC, PLAIN>(g, R, item, 0, ks, piece);
}
template <class E>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) lin_ring_dx(const KArgs g) {
  SWIGLU_RING_LDS(true)
  const int i = blockIdx.x;
  dx_tile<E>(g, R, i / g.ksplit, i % g.ksplit, g.ksplit > 1 ? i : -1);
}
template <class E>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) lin_ring_dw(const KArgs g) {
  SWIGLU_RING_LDS(true)
  const int i = blockIdx.x;
  ring5_tile<E, MC, MC, PLAIN>(g, R, i / g.ksplit, 0, i % g.ksplit, g.ksplit > 1 ? i : -1);
}
// Joins the parts of the ring's tiles (16 bits): eight columns of a row per thread.
template <class E>
__global__ void __launch_bounds__(256) lin_join_tiles(const KArgs g) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i >> 13), r = (int)(i >> 5) & 255, c = ((int)i & 31) * 8;
  int tm, tn;
  tile_coords(t, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
  const int m = tm * 256 + r, n = tn * 256 + c;
  if (m >= g.M || n >= g.N) return;
  const float* p = g.P + (int64_t)t * g.ksplit * 65536 + r * 256 + c;
  float z[8] = {};
  for (int s = 0; s < g.ksplit; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += p[(int64_t)s * 65536 + e];
  linear_store<E>(g, m, n, z);
}
// dW and dx on the ring, the longer tiles first.
template <class E>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
lin_ring_grads(const KArgs w, const KArgs x, int first) {
  SWIGLU_RING_LDS(true)
  const int nw = w.tiles_m * w.tiles_n, nx = x.tiles_m * x.tiles_n, b = blockIdx.x;
  if (first ? b >= nx : b < nw) ring5_tile<E, MC, MC, PLAIN>(w, R, first ? b - nx : b, 0);
  else dx_tile<E>(x, R, first ? b : b - nw, 0, -1);
}

static inline int status() { return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH; }

static inline dim3 ring_grid(const KArgs& a) { return dim3(a.tiles_m * a.tiles_n * a.ksplit); }
template <class E, int ACT>
int launch_lin_ring(const KArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lin_ring<E, ACT>), ring_grid(a), dim3(256), 0, s, a);
  return status();
}
template <class E>
int launch_lin_ring_parts(const KArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lin_ring_parts<E>), ring_grid(a), dim3(256), 0, s, a);
  return status();
}
template <class E>
static int launch_ring_dx(const KArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lin_ring_dx<E>), ring_grid(a), dim3(256), 0, s, a);
  return status();
}
template <class E>
static int launch_ring_dw(const KArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lin_ring_dw<E>), ring_grid(a), dim3(256), 0, s, a);
  return status();
}
#define SWIGLU_LIN_RING_DECL(PREFIX, E)                                             \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_NONE>(const KArgs&, hipStream_t);      \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_RELU>(const KArgs&, hipStream_t);      \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_GELU>(const KArgs&, hipStream_t);      \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_GELU_TANH>(const KArgs&, hipStream_t); \
  PREFIX template int launch_lin_ring<E, SWIGLU_ACT_SILU>(const KArgs&, hipStream_t);      \
  PREFIX template int launch_lin_ring_parts<E>(const KArgs&, hipStream_t);

template <class E, int XR, int NW, int SH, int RING>
static int launch_few(const FewArgs& a, int grid, hipStream_t s) {
  StageScope scope(STAGE_LINEAR, s);
  hipLaunchKernelGGL((lin_few<E, XR, NW, SH, RING>), dim3(grid, a.splits), dim3(NW * 64), 0, s, a);
  return status();
}
template <class E, int XR>
static int few_own(const FewArgs& a, hipStream_t s) {
  const int tiles = cdiv(a.f.N, 16), ncu = dev_ncu();
  if (tiles <= ncu) return launch_few<E, XR, 16, 1, 131072>(a, tiles, s);
  const int fit = 2 * ncu;
  return launch_few<E, XR, 4, 1, 65536>(a, tiles < fit ? tiles : fit, s);
}
// The parts of up to two products joined in one launch.
template <class E>
static int launch_join(const KArgs& a, const KArgs& b, hipStream_t s) {
  constexpr int V = 16 / E::kBytes;
  const int64_t qa = a.ksplit > 1 ? (int64_t)a.M * a.N / V : 0, qb = b.ksplit > 1 ? (int64_t)b.M * b.N / V : 0;
  if (qa + qb == 0) return SWIGLU_OK;
  hipLaunchKernelGGL((lin_join<E>), dim3((unsigned)((qa + 255) / 256 + (qb + 255) / 256)), dim3(256), 0, s, a, b, qa, qb);
  return status();
}

template <class E, int AL, int BL, int STAGE, int BM, int BN>
static int launch_tiles(KArgs a, hipStream_t s) {
  a.tiles_m = cdiv(a.M, BM);
  a.tiles_n = cdiv(a.N, BN);
  if (a.tiles_m * a.tiles_n == 0) return SWIGLU_OK;
  hipLaunchKernelGGL((lin_tile<E, BM, BN, AL, BL, STAGE>), dim3(a.tiles_m * a.tiles_n * a.ksplit), dim3(256), 0, s, a);
  const int rc = status();
  return rc ? rc : launch_join<E>(a, KArgs{}, s);
}
// A product as planned; on the ring `whole` launches it, or `parts` its parts.
using RingLaunch = int (*)(const KArgs&, hipStream_t);
template <class E, int AL, int BL, int STAGE>
static int run_product(KArgs a, const Product& p, float* sums, hipStream_t s, RingLaunch whole, RingLaunch parts) {
  a.planes = 1;
  a.ksplit = p.splits;
  a.kchunk = p.kchunk;
  a.P = sums;
  if constexpr (E::kBytes == 2) {
    if (p.tile == TRING) {
      a.tiles_m = cdiv(a.M, 256);
      a.tiles_n = cdiv(a.N, 256);
      a.group_m = AL == MC ? 4 : BL == MC ? 1 : 2;
      if (p.splits == 1) return whole(a, s);
      const int rc = parts(a, s);
      if (rc) return rc;
      hipLaunchKernelGGL((lin_join_tiles<E>), dim3(a.tiles_m * a.tiles_n * 32), dim3(256), 0, s, a);
      return status();
    }
    if (p.tile == T64x128) return launch_tiles<E, AL, BL, STAGE, 64, 128>(a, s);
    if (p.tile == T128) return launch_tiles<E, AL, BL, STAGE, 128, 128>(a, s);
  }
  return launch_tiles<E, AL, BL, STAGE, 64, 64>(a, s);
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
    a.P = f.partial;
    a.ksplit = f.splits;
    return launch_join<E>(a, KArgs{}, c.stream);
  }
  RingLaunch whole = nullptr, parts = nullptr;
  if constexpr (E::kBytes == 2) {
    parts = &launch_lin_ring_parts<E>;
    whole = c.act == SWIGLU_ACT_RELU        ? &launch_lin_ring<E, SWIGLU_ACT_RELU>
            : c.act == SWIGLU_ACT_GELU      ? &launch_lin_ring<E, SWIGLU_ACT_GELU>
            : c.act == SWIGLU_ACT_GELU_TANH ? &launch_lin_ring<E, SWIGLU_ACT_GELU_TANH>
            : c.act == SWIGLU_ACT_SILU      ? &launch_lin_ring<E, SWIGLU_ACT_SILU>
                                            : &launch_lin_ring<E, SWIGLU_ACT_NONE>;
  }
  StageScope scope(STAGE_LINEAR, c.stream);
  return run_product<E, KC, KC, STAGE_LINEAR>(a, fwd_plan(c.T, c.N, c.K, E::kBytes), (float*)c.ws, c.stream, whole, parts);
}

template <class E>
int run_bwd(const Bwd& c) {
  const bool act = c.act != SWIGLU_ACT_NONE;
  const BwdPlan p = bwd_plan(c.T, c.N, c.K, E::kBytes, act);
  const char* dz = (const char*)c.dy;
  float* parts = (float*)(c.ws + p.parts);
  hipStream_t s = c.stream;
  if (c.db || (act && (c.dx || c.dw))) {
    StageScope scope(STAGE_LINEAR_DZ, s);
    const char* z = act ? (const char*)c.z : nullptr;
    if (act) dz = c.ws;
    if (p.strips == 0) {
      const DzArgs d{(const char*)c.dy, z, c.ws, nullptr, c.T, (int)c.N, c.act};
      hipLaunchKernelGGL((lin_dz_few<E>), dim3((unsigned)((c.N * E::kBytes + 127) / 128)), dim3(1024), 0, s, d, (char*)c.db);
      if (status()) return SWIGLU_ERR_LAUNCH;
    } else {
      const DzArgs d{(const char*)c.dy, z, c.ws, c.db ? parts : nullptr, c.T, (int)c.N, c.act};
      hipLaunchKernelGGL((lin_dz<E>), dim3((unsigned)((c.N * E::kBytes + 1023) / 1024), p.strips), dim3(256), 0, s, d);
      if (status()) return SWIGLU_ERR_LAUNCH;
      if (c.db) {
        const int rc = norm::launch_sum_parts<E>(parts, p.strips, 1, c.N, c.db, nullptr, s);
        if (rc) return rc;
      }
    }
  }
  if (!c.dw && !c.dx) return SWIGLU_OK;
  KArgs w{}, x{};
  w.a0 = opnd(dz, c.N, c.N, c.T);  // dW [N, K]: rows dz^T, columns x, summed over tokens
  w.b0 = opnd(c.x, c.K, c.K, c.T);
  w.c0 = (char*)c.dw;
  w.ldc = c.K;
  w.M = (int)c.N;
  w.N = (int)c.K;
  x.a0 = opnd(dz, c.N, c.T, c.N);  // dx [T, K]: rows dz, columns of W, summed over N
  x.b0 = opnd(c.w, c.K, c.K, c.N);
  x.c0 = (char*)c.dx;
  x.ldc = c.K;
  x.M = (int)c.T;
  x.N = (int)c.K;
  const Grads& g = p.grads[(c.dw ? 1 : 0) + (c.dx ? 2 : 0)];
  float* x_parts = (float*)((char*)parts + (c.dw ? align256(product_bytes(g.w, c.N, c.K)) : 0));
  if (g.together) {
    StageScope scope(STAGE_LINEAR_DW, s);
    if constexpr (E::kBytes == 2) {
      if (g.ring) {
        w.tiles_m = cdiv(w.M, 256);
        x.tiles_m = cdiv(x.M, 256);
        w.tiles_n = x.tiles_n = cdiv(w.N, 256);
        w.group_m = 4;
        x.group_m = 1;
        hipLaunchKernelGGL((lin_ring_grads<E>), dim3((w.tiles_m + x.tiles_m) * w.tiles_n), dim3(256), 0, s, w, x,
                           c.T >= c.N ? 0 : 1);
        return status();
      }
    }
    w.tiles_m = cdiv(w.M, 64);
    x.tiles_m = cdiv(x.M, 64);
    w.tiles_n = x.tiles_n = cdiv(w.N, 64);
    w.ksplit = g.w.splits;
    w.kchunk = g.w.kchunk;
    w.P = parts;
    x.ksplit = g.x.splits;
    x.kchunk = g.x.kchunk;
    x.P = x_parts;
    const int n = w.tiles_n * (w.tiles_m * w.ksplit + x.tiles_m * x.ksplit);
    hipLaunchKernelGGL((lin_tile_grads<E>), dim3(n), dim3(256), 0, s, w, x, x.kchunk > w.kchunk);
    const int rc = status();
    return rc ? rc : launch_join<E>(w, x, s);
  }
  RingLaunch dw_ring = nullptr, dx_ring = nullptr;
  if constexpr (E::kBytes == 2) {
    dw_ring = &launch_ring_dw<E>;
    dx_ring = &launch_ring_dx<E>;
  }
  if (c.dw) {
    StageScope scope(STAGE_LINEAR_DW, s);
    const int rc = run_product<E, MC, MC, STAGE_LINEAR_DW>(w, g.w, parts, s, dw_ring, dw_ring);
    if (rc) return rc;
  }
  if (c.dx) {
    StageScope scope(STAGE_LINEAR_DX, s);
    return run_product<E, KC, MC, STAGE_LINEAR_DX>(x, g.x, x_parts, s, dx_ring, dx_ring);
  }
  return SWIGLU_OK;
}

}  // namespace lin
}  // namespace swiglu

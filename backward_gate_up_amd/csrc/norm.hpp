// norm.hpp -- layer norm and RMS norm over the last axis, forward and backward, gfx950.
//
//   forward   n = (x - mean) rstd, y = n w + b      rstd = 1 / sqrt(mean (x - mean)^2 + eps)
//   backward  g = dy w
//             dx = rstd (g - mean(g) - n mean(g n)) (+ dres)
//             dw = sum over rows of dy n, db = sum over rows of dy
//   RMS norm: mean = 0 throughout and no mean(g) term.
//
// What bounds it: memory. The forward reads x and writes y, the backward reads
// x and dy and writes dx, each element once: a row is held in registers (as its
// 16-byte pieces, widened where they are used) while its sums are formed, so the
// variance is that of the differences from the mean and not a difference of two
// large sums. All sums are fp32.
//
// The mean is formed twice: the row's sum times 1 / D is off by the sum's roundings
// and by that of 1 / D, an error of |mean| and not of the spread, which rstd
// multiplies by up to 1 / sqrt(eps) (a constant row of 1000 with D = 1000 gave n =
// -0.019). The pass that sums the squares of x - mean also sums x - mean itself;
// its mean is what the first was off by, and its square comes off the variance. So a
// constant row's mean is exact, and any row's off by its own rounding and by roundings
// of the spread.
//
// Split: W waves hold a row, NC pieces of 16 bytes per lane: one wave up to 4
// KiB, four up to 16 KiB, sixteen up to 32 KiB; wider rows are walked three times
// (they come from L2 after the first). A group of waves walks rows with the
// stride of the grid, keeps w and b, and asks for the next row before it works
// on the one it has.
//
// Measured (bf16): forward of 16384 x 4096 53 us and of 65536 x 1024 54 us, 5.1 and
// 5.0 TB/s, the rate of a copy; RMS 50 and 52. Where a call writes the last one's y
// again, of which the 256 MB cache holds a part, 46, 48, 45 and 48. Their backward 90 us
// (4.5 TB/s, two sums per row between loads and stores) and, RMS of 65536 x 1024, 81 us
// (5.0 TB/s), the join of the weight's gradient 5 us. fp32, 16384 x 4096, 104 and 160
// us (5.2 and 5.0 TB/s). 16 rows of 2048 3.3 us, a launch and two latencies.
//
// The weight's gradient is summed in the same pass over x and dy: each lane owns
// its columns for all rows of its group, so its sums are registers. They are
// joined within the workgroup in LDS, across workgroups through one fp32 row
// per workgroup and a second launch, in a fixed order: no atomics, the same
// bits every time.
//
// Rows need not be aligned: pieces are loaded at the alignment of an element,
// which global memory takes at full rate where they do not cross a line, and a
// row's last piece, where it is a part of one, element by element.
#pragma once
#include "kernels.hpp"

namespace swiglu {
namespace norm {

struct Args {
  const char* x;
  const char* w;
  const char* b;      // forward: may be nullptr
  char* y;            // forward: y; backward: dx
  float* stats;       // [2][T] mean, rstd (RMS: [T] rstd); forward: may be nullptr
  const char* dy;     // backward
  const char* dres;   // backward: added to dx, may be nullptr
  float* partial;     // backward: [workgroups][V][D], V = 2 (RMS: 1)
  int64_t T;
  int D;
  float eps, inv_d;
};

// ---- pieces of a row ----------------------------------------------------------
typedef u32x4_t __attribute__((aligned(2))) u32x4_at2_t;
typedef u32x4_t __attribute__((aligned(4))) u32x4_at4_t;

template <class E>
struct Piece {
  static constexpr int V = 16 / E::kBytes;  // elements
  using any_u32x4_t = std::conditional_t<E::kBytes == 4, u32x4_at4_t, u32x4_at2_t>;
  u32x4_t v;

  // elements [at, at + V) of a row of D; zeros past its end. EVEN: D is a
  // multiple of V, so a piece is inside or outside.
  template <bool EVEN = false>
  __device__ __forceinline__ void load(const char* row, int at, int D) {
    if (EVEN ? at < D : at + V <= D) {
      v = *(const any_u32x4_t*)(row + (int64_t)at * E::kBytes);
    } else {
      v = u32x4_t{};
      if (!EVEN && at < D) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at + i < D) put(i, ((const typename E::elem*)row)[at + i]);
      }
    }
  }
  template <bool EVEN = false>
  __device__ __forceinline__ void store(char* row, int at, int D) const {
    if (EVEN ? at < D : at + V <= D) {
      *(any_u32x4_t*)(row + (int64_t)at * E::kBytes) = v;
    } else if (!EVEN && at < D) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at + i < D) ((typename E::elem*)row)[at + i] = elem(i);
    }
  }
  // (the element of a vector is copied out before it is looked at as another type)
  __device__ __forceinline__ typename E::elem elem(int i) const {
    if constexpr (E::kBytes == 4) {
      const uint32_t u = v[i];
      return __builtin_bit_cast(float, u);
    } else {
      const uint32_t u = v[i / 2];
      const uint16_t h = (uint16_t)(i & 1 ? u >> 16 : u);
      return __builtin_bit_cast(typename E::elem, h);
    }
  }
  __device__ __forceinline__ void put(int i, typename E::elem e) {
    if constexpr (E::kBytes == 4) {
      v[i] = __builtin_bit_cast(uint32_t, e);
    } else {
      const uint32_t h = __builtin_bit_cast(uint16_t, e), old = v[i / 2];
      v[i / 2] = i & 1 ? (old & 0xffffu) | (h << 16) : (old & 0xffff0000u) | h;
    }
  }
  __device__ __forceinline__ float get(int i) const { return E::to_f32(elem(i)); }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// v plus that of the lane N further on in the same row of sixteen (DPP row_ror)
template <int N>
__device__ __forceinline__ float turn_add(float v) {
  const int u = __builtin_bit_cast(int, v);
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, 0x120 + N, 0xf, 0xf, false));
}
// Of two values in as many exchanges: the first's sum in lanes 0..31, the second's in
// lanes 32..63, each added in wave_sum's order. (Forward of 4096 x 11008
// bf16: 53 us without the mean's correction, 60 with it as two sums, 56 so.)
__device__ __forceinline__ float wave_sum_halves(float a, float b) {
  const bool low = (threadIdx.x & 32) == 0;
  float v = (low ? a : b) + __shfl_xor(low ? b : a, 32);
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
// Sums of K values over the W waves that hold a row; `at` alternates between
// two places in LDS, so that one barrier per sum is enough (a wave that writes a
// place again has passed the barrier after every wave's reads of it).
template <int W, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (&red)[2][K][16], int& at) {
  static_assert(K == 1 || K == 2, "one or two sums");
  float part;
  if constexpr (K == 1) part = wave_sum(v[0]);
  else part = wave_sum_halves(v[0], v[1]);
  if constexpr (W == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane_of(part, 32 * k);
  } else {
    const int wave = (threadIdx.x >> 6) % W;
    if ((threadIdx.x & (K == 1 ? 63 : 31)) == 0) red[at][K == 1 ? 0 : threadIdx.x >> 5 & 1][wave] = part;
    __syncthreads();
    if constexpr (K == 2 && W == 16) {
      // a wave's value per lane, added by turning rows of sixteen lanes
      float r = red[at][threadIdx.x >> 4 & 1][threadIdx.x & 15];
      r = turn_add<8>(r);
      r = turn_add<4>(r);
      r = turn_add<2>(r);
      r = turn_add<1>(r);
      v[0] = lane_of(r, 0);
      v[1] = lane_of(r, 16);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v[k] += red[at][k][w];
      }
    }
    at ^= 1;
  }
}

// 1 / sqrt in IEEE steps: the row's only one.
__device__ __forceinline__ float inv_sqrt(float v) { return 1.0f / sqrtf(v); }

// The variance plus eps from q[0], the sum of the squares of x - mean, and (layer
// norm) the corrected mean from q[1], the sum of x - mean. The multiply and add of
// the correction's square is one rounding, so an infinite sum of squares stays one;
// a NaN passes the comparison.
template <bool RMS>
__device__ __forceinline__ float spread(const float (&q)[RMS ? 1 : 2], float inv_d, float eps, float& mean) {
  if constexpr (RMS) {
    return fmaf(q[0], inv_d, eps);
  } else {
    const float shift = q[1] * inv_d, var = fmaf(-shift, shift, q[0] * inv_d);
    mean += shift;
    return (var < 0.f ? 0.f : var) + eps;
  }
}

// s / D: the product with 1 / D and what it leaves of s, so that a gradient that is the
// same everywhere has its own mean (a division's steps cost the backward 1 %).
__device__ __forceinline__ float mean_of(float s, const Args& g) {
  const float m = s * g.inv_d;
  return fmaf(fmaf(-m, (float)g.D, s), g.inv_d, m);
}

// Rows of a workgroup: one wave each for W = 1, else one for all.
template <int W>
constexpr int kThreads = W == 1 ? 256 : 64 * W;
template <int W>
constexpr int kRows = W == 1 ? 4 : 1;

// Sixteen waves have no registers for the next row beside their own.
template <int W>
constexpr bool kAhead = W < 16;

// ---- forward --------------------------------------------------------------------
// EVEN: D is a multiple of a piece, so no piece is partly past the row's end.
template <class E, bool RMS, int W, int NC, bool EVEN>
__global__ void __launch_bounds__(kThreads<W>) norm_fwd(const Args g) {
  using P = Piece<E>;
  constexpr int V = P::V, K = RMS ? 1 : 2;
  __shared__ float red[2][1][16], red_q[2][K][16];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x, wave = threadIdx.x >> 6;
  const int64_t rowb = (int64_t)g.D * E::kBytes, step = (int64_t)gridDim.x * kRows<W>;
  int64_t t = (int64_t)blockIdx.x * kRows<W> + (W == 1 ? wave : 0);
  if (t >= g.T) return;  // whole waves, or (W > 1) the whole workgroup
  int where[NC];
  P w[NC], b[NC], x[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    where[c] = (c * 64 * W + lane) * V;
    x[c].template load<EVEN>(g.x + t * rowb, where[c], g.D);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    w[c].template load<EVEN>(g.w, where[c], g.D);
    b[c].v = u32x4_t{};
    if (g.b) b[c].template load<EVEN>(g.b, where[c], g.D);
  }
  int at = 0;
  while (true) {
    const int64_t next = t + step;
    P nx[NC];
    if (kAhead<W> && next < g.T) {
#pragma unroll
      for (int c = 0; c < NC; ++c) nx[c].template load<EVEN>(g.x + next * rowb, where[c], g.D);
    }
    float mean = 0.f;
    if constexpr (!RMS) {
      float s[1] = {};
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += x[c].get(i);
      row_sum<W, 1>(s, red, at);
      mean = s[0] * g.inv_d;
    }
    float q[K] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (where[c] >= g.D) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = x[c].get(i) - mean;
        if (EVEN || where[c] + i < g.D) {
          q[0] = fmaf(d, d, q[0]);
          if constexpr (!RMS) q[K - 1] += d;
        }
      }
    }
    row_sum<W, K>(q, red_q, at);
    const float rstd = inv_sqrt(spread<RMS>(q, g.inv_d, g.eps, mean));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (where[c] >= g.D) continue;
      P y;
      y.v = u32x4_t{};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = (x[c].get(i) - mean) * rstd;
        y.put(i, E::from_f32(fmaf(n, w[c].get(i), b[c].get(i))));
      }
      y.template store<EVEN>(g.y + t * rowb, where[c], g.D);
    }
    if (g.stats && lane == 0) {
      if constexpr (RMS) {
        g.stats[t] = rstd;
      } else {
        g.stats[t] = mean;
        g.stats[g.T + t] = rstd;
      }
    }
    if (next >= g.T) break;
    t = next;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if constexpr (kAhead<W>) x[c] = nx[c];
      else x[c].template load<EVEN>(g.x + t * rowb, where[c], g.D);
    }
  }
}

// Rows wider than sixteen waves hold: a workgroup per row walks it for the mean,
// the variance and y.
template <class E, bool RMS>
__global__ void __launch_bounds__(1024) norm_fwd_wide(const Args g) {
  using P = Piece<E>;
  constexpr int V = P::V, K = RMS ? 1 : 2;
  __shared__ float red[2][1][16], red_q[2][K][16];
  const int64_t rowb = (int64_t)g.D * E::kBytes;
  int at = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    const char* row = g.x + t * rowb;
    float mean = 0.f;
    if constexpr (!RMS) {
      float s[1] = {};
      for (int d = threadIdx.x * V; d < g.D; d += 1024 * V) {
        P x;
        x.load(row, d, g.D);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += x.get(i);
      }
      row_sum<16, 1>(s, red, at);
      mean = s[0] * g.inv_d;
    }
    float q[K] = {};
    for (int d = threadIdx.x * V; d < g.D; d += 1024 * V) {
      P x;
      x.load(row, d, g.D);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float v = x.get(i) - mean;
        if (d + i < g.D) {
          q[0] = fmaf(v, v, q[0]);
          if constexpr (!RMS) q[K - 1] += v;
        }
      }
    }
    row_sum<16, K>(q, red_q, at);
    const float rstd = inv_sqrt(spread<RMS>(q, g.inv_d, g.eps, mean));
    for (int d = threadIdx.x * V; d < g.D; d += 1024 * V) {
      P x, w, b, y;
      x.load(row, d, g.D);
      w.load(g.w, d, g.D);
      b.v = y.v = u32x4_t{};
      if (g.b) b.load(g.b, d, g.D);
#pragma unroll
      for (int i = 0; i < V; ++i) y.put(i, E::from_f32(fmaf((x.get(i) - mean) * rstd, w.get(i), b.get(i))));
      y.store(g.y + t * rowb, d, g.D);
    }
    if (g.stats && threadIdx.x == 0) {
      if constexpr (RMS) {
        g.stats[t] = rstd;
      } else {
        g.stats[t] = mean;
        g.stats[g.T + t] = rstd;
      }
    }
  }
}

// ---- backward -------------------------------------------------------------------
template <bool RMS>
__device__ __forceinline__ void load_stats(const Args& g, int64_t t, float& mean, float& rstd) {
  mean = RMS ? 0.f : g.stats[t];
  rstd = g.stats[RMS ? t : g.T + t];
}

// Rows that a workgroup works on at a time: as many groups of W waves as its
// registers allow, so that the sums over rows meet in LDS before they leave the
// workgroup (one of sixteen waves per CU instead of two of four: 16384 x 4096 bf16
// 94.6 -> 88.9 us, 65536 x 1024 RMS 95 -> 80).
template <int W, int NC>
constexpr int kBwdRows = W == 1 ? (NC == 4 ? 8 : 16) : W == 4 ? (NC == 4 ? 2 : 4) : 1;

// dx of every row and the workgroup's sums of dw (and db) in partial[blockIdx.x].
template <class E, bool RMS, int W, int NC, bool EVEN>
__global__ void __launch_bounds__((64 * W * kBwdRows<W, NC>)) norm_bwd(const Args g) {
  using P = Piece<E>;
  constexpr int V = P::V, K = RMS ? 1 : 2, R = kBwdRows<W, NC>;
  __shared__ float red[R][2][K][16];
  // half of the groups' sums of the weight's gradient, one lane's value apart
  __shared__ float join[R > 1 ? R / 2 * K * NC * V * 64 * W : 1];
  const int lane = threadIdx.x % (64 * W);
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * W));
  const int64_t rowb = (int64_t)g.D * E::kBytes, step = (int64_t)gridDim.x * R;
  int64_t t = (int64_t)blockIdx.x * R + group;
  int where[NC];
  P w[NC];
  float sum[K][NC][V];  // dw, db
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    where[c] = (c * 64 * W + lane) * V;
    w[c].template load<EVEN>(g.w, where[c], g.D);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k) sum[k][c][i] = 0.f;
  }
  int at = 0;
  P x[NC], dy[NC];
  float mean = 0.f, rstd = 0.f;
  // rows past the last are zeros and not stored: every group passes every barrier
  auto load = [&](P (&xs)[NC], P (&ds)[NC], float& m, float& r, int64_t row) {
    if (row < g.T) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        xs[c].template load<EVEN>(g.x + row * rowb, where[c], g.D);
        ds[c].template load<EVEN>(g.dy + row * rowb, where[c], g.D);
      }
      load_stats<RMS>(g, row, m, r);
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) xs[c].v = ds[c].v = u32x4_t{};
      m = r = 0.f;
    }
  };
  load(x, dy, mean, rstd, t);
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < g.T; t0 += step, t += step) {
    P nx[NC], ndy[NC];
    float nmean = 0.f, nrstd = 0.f;
    if constexpr (kAhead<W>) load(nx, ndy, nmean, nrstd, t + step);
    float s[K] = {};  // sum of g n, sum of g (zeros past the row's end: dy is 0 there)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (where[c] >= g.D) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = (x[c].get(i) - mean) * rstd, d = dy[c].get(i), gg = d * w[c].get(i);
        s[0] = fmaf(gg, n, s[0]);
        sum[0][c][i] = fmaf(d, n, sum[0][c][i]);
        if constexpr (!RMS) {
          s[K - 1] += gg;
          sum[K - 1][c][i] += d;
        }
      }
    }
    row_sum<W, K>(s, red[group], at);
    if (t < g.T) {
      const float along = s[0] * g.inv_d, level = RMS ? 0.f : mean_of(s[K - 1], g);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (where[c] >= g.D) continue;
        P dx, r;
        dx.v = r.v = u32x4_t{};
        if (g.dres) r.template load<EVEN>(g.dres + t * rowb, where[c], g.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = (x[c].get(i) - mean) * rstd, gg = dy[c].get(i) * w[c].get(i);
          float v = (fmaf(-n, along, gg) - level) * rstd;
          if (g.dres) v += r.get(i);
          dx.put(i, E::from_f32(v));
        }
        dx.template store<EVEN>(g.y + t * rowb, where[c], g.D);
      }
    }
    if constexpr (kAhead<W>) {
      mean = nmean;
      rstd = nrstd;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c] = nx[c];
        dy[c] = ndy[c];
      }
    } else {
      load(x, dy, mean, rstd, t + step);
    }
  }
  // the groups' sums, halved until the first has them all
#pragma unroll
  for (int half = R / 2; half; half /= 2) {
    if (half < R / 2) __syncthreads();  // the last half's have been read
    float* p = join + (group % half) * (K * NC * V * 64 * W) + lane;
    if (group >= half && group < 2 * half) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int k = 0; k < K; ++k) p[((k * NC + c) * V + i) * 64 * W] = sum[k][c][i];
    }
    __syncthreads();
    if (group < half) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int k = 0; k < K; ++k) sum[k][c][i] += p[((k * NC + c) * V + i) * 64 * W];
    }
  }
  if (group) return;
  float* out = g.partial + (int64_t)blockIdx.x * K * g.D;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (where[c] + i < g.D) {
#pragma unroll
        for (int k = 0; k < K; ++k) out[(int64_t)k * g.D + where[c] + i] = sum[k][c][i];
      }
}

// Rows wider than sixteen waves hold: dx (two walks), the weight's gradient in a
// launch of its own.
template <class E, bool RMS>
__device__ __forceinline__ void bwd_row(const Args& g, int64_t t, float (&red)[2][RMS ? 1 : 2][16], int& at) {
  using P = Piece<E>;
  constexpr int V = P::V, K = RMS ? 1 : 2;
  const int64_t rowb = (int64_t)g.D * E::kBytes;
  float mean, rstd, s[K] = {};
  load_stats<RMS>(g, t, mean, rstd);
  for (int d = threadIdx.x * V; d < g.D; d += 1024 * V) {
    P x, dy, w;
    x.load(g.x + t * rowb, d, g.D);
    dy.load(g.dy + t * rowb, d, g.D);
    w.load(g.w, d, g.D);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float gg = dy.get(i) * w.get(i);
      s[0] = fmaf(gg, (x.get(i) - mean) * rstd, s[0]);
      if constexpr (!RMS) s[K - 1] += gg;
    }
  }
  row_sum<16, K>(s, red, at);
  const float along = s[0] * g.inv_d, level = RMS ? 0.f : mean_of(s[K - 1], g);
  for (int d = threadIdx.x * V; d < g.D; d += 1024 * V) {
    P x, dy, w, r, dx;
    x.load(g.x + t * rowb, d, g.D);
    dy.load(g.dy + t * rowb, d, g.D);
    w.load(g.w, d, g.D);
    r.v = dx.v = u32x4_t{};
    if (g.dres) r.load(g.dres + t * rowb, d, g.D);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = (fmaf(-(x.get(i) - mean) * rstd, along, dy.get(i) * w.get(i)) - level) * rstd;
      if (g.dres) v += r.get(i);
      dx.put(i, E::from_f32(v));
    }
    dx.store(g.y + t * rowb, d, g.D);
  }
}
template <class E, bool RMS>
__global__ void __launch_bounds__(1024) norm_bwd_wide(const Args g) {
  __shared__ float red[2][RMS ? 1 : 2][16];
  int at = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) bwd_row<E, RMS>(g, t, red, at);
}
// A lane's piece of columns over the rows of strip blockIdx.y.
template <class E, bool RMS>
__global__ void __launch_bounds__(256) norm_wgrad_wide(const Args g) {
  using P = Piece<E>;
  constexpr int V = P::V, K = RMS ? 1 : 2;
  const int at = (blockIdx.x * 256 + threadIdx.x) * V;
  if (at >= g.D) return;
  const int64_t rowb = (int64_t)g.D * E::kBytes;
  const int64_t t0 = g.T * blockIdx.y / gridDim.y, t1 = g.T * (blockIdx.y + 1) / gridDim.y;
  float dw[V] = {}, db[V] = {};
  for (int64_t t = t0; t < t1; ++t) {
    float mean, rstd;
    load_stats<RMS>(g, t, mean, rstd);
    P x, dy;
    x.load(g.x + t * rowb, at, g.D);
    dy.load(g.dy + t * rowb, at, g.D);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dw[i] = fmaf(dy.get(i), (x.get(i) - mean) * rstd, dw[i]);
      db[i] += dy.get(i);
    }
  }
  float* out = g.partial + (int64_t)blockIdx.y * K * g.D + at;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (at + i < g.D) {
      out[i] = dw[i];
      if constexpr (!RMS) out[g.D + i] = db[i];
    }
}

// At most kFewRows rows in one launch, without partial sums: a workgroup per row
// for dx, as above, then a workgroup per 64 pieces of columns for dw and db, whose
// sixteen waves take every sixteenth row (x and dy come from L2 there; mean and
// rstd are known, so neither half waits for the other).
constexpr int kFewRows = 256;
template <class E, bool RMS>
__global__ void __launch_bounds__(1024) norm_bwd_few(const Args g, char* dw_out, char* db_out) {
  using P = Piece<E>;
  constexpr int V = P::V, K = RMS ? 1 : 2;
  __shared__ union {
    float sum[2][K][16];
    float cols[16][64 * V];
  } lds;
  if (blockIdx.x < g.T) {
    int at = 0;
    bwd_row<E, RMS>(g, blockIdx.x, lds.sum, at);
    return;
  }
  const int64_t rowb = (int64_t)g.D * E::kBytes;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = (int)(blockIdx.x - g.T) * 64 * V, at = first + lane * V;
  float dw[V] = {}, db[V] = {};
  if (at < g.D) {
#pragma unroll 4
    for (int64_t t = wave; t < g.T; t += 16) {
      float mean, rstd;
      load_stats<RMS>(g, t, mean, rstd);
      P x, dy;
      x.load(g.x + t * rowb, at, g.D);
      dy.load(g.dy + t * rowb, at, g.D);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dw[i] = fmaf(dy.get(i), (x.get(i) - mean) * rstd, dw[i]);
        if constexpr (!RMS) db[i] += dy.get(i);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k) __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) lds.cols[wave][lane * V + i] = k ? db[i] : dw[i];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < 64 * V && first + c < g.D) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 16; ++w) v += lds.cols[w][c];
      char* out = k ? db_out : dw_out;
      if (out) ((typename E::elem*)out)[first + c] = E::from_f32(v);
    }
  }
}

// ---- column sums over parts -------------------------------------------------------
// out0[n] = rnd(sum over parts of partial[part][0][n]), out1 the same of row 1
// (rows == 2): 16 neighbouring columns by 16 parts at a time per workgroup, the
// sixteen sums of a column added in order.
template <class E>
__global__ void __launch_bounds__(256) sum_parts(const float* partial, int parts, int rows, int N, char* out0, char* out1) {
  __shared__ float red[16][17];
  const int64_t len = (int64_t)rows * N;
  const int c = threadIdx.x & 15, p0 = threadIdx.x >> 4;
  const int64_t n = (int64_t)blockIdx.x * 16 + c;
  float s = 0.f;
  if (n < len) {
    int p = p0;
    for (; p + 48 < parts; p += 64) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = partial[(int64_t)(p + 16 * i) * len + n];
#pragma unroll
      for (int i = 0; i < 4; ++i) s += v[i];
    }
    for (; p < parts; p += 16) s += partial[(int64_t)p * len + n];
  }
  red[p0][c] = s;
  __syncthreads();
  if (threadIdx.x < 16 && n < len) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += red[i][c];
    if (n < N) {
      if (out0) ((typename E::elem*)out0)[n] = E::from_f32(v);
    } else if (out1) {
      ((typename E::elem*)out1)[n - N] = E::from_f32(v);
    }
  }
}
template <class E>
static int launch_sum_parts(const float* partial, int parts, int rows, int64_t N, void* out0, void* out1, hipStream_t s) {
  hipLaunchKernelGGL((sum_parts<E>), dim3((unsigned)((rows * N + 15) / 16)), dim3(256), 0, s, partial, parts, rows, (int)N,
                     (char*)out0, (char*)out1);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

// ---- launches -----------------------------------------------------------------------
// Waves per row and pieces per lane for rows of D elements; w = 0: wide.
struct Shape {
  int w, nc;
};
static inline Shape shape_of(int64_t D, size_t e) {
  const int64_t p = (D * (int64_t)e + 15) / 16;  // pieces
  if (p <= 64) return {1, 1};
  if (p <= 128) return {1, 2};
  if (p <= 256) return {1, 4};
  if (p <= 512) return {4, 2};
  if (p <= 1024) return {4, 4};
  if (p <= 2048) return {16, 2};
  return {0, 0};
}
// The backward walks rows that need sixteen waves and are not whole pieces: their
// last piece's addresses would not fit in a lane's 128 registers.
static inline Shape bwd_shape_of(int64_t D, size_t e) {
  const Shape f = shape_of(D, e);
  return f.w == 16 && D * (int64_t)e % 16 ? Shape{0, 0} : f;
}
static inline int64_t groups(int64_t T, int rows, int64_t most) {
  const int64_t n = (T + rows - 1) / rows;
  return n < most ? n : most;
}
// Workgroups of the backward, each of which leaves a row of partial sums: one per CU.
static inline int bwd_groups(const Shape& f, int64_t T, int64_t D, size_t e) {
  const int ncu = dev_ncu();
  if (f.w == 0) {  // strips of norm_wgrad_wide: about four workgroups per CU
    const int64_t cols = (D * (int64_t)e + 4095) / 4096, s = 4 * ncu / cols;
    return (int)groups(T, 16, s < 1 ? 1 : s > 64 ? 64 : s);
  }
  const int rows = f.w == 1 ? (f.nc == 4 ? kBwdRows<1, 4> : kBwdRows<1, 2>)
                   : f.w == 4 ? (f.nc == 4 ? kBwdRows<4, 4> : kBwdRows<4, 2>)
                              : 1;
  return (int)groups(T, rows, ncu);
}
static inline size_t bwd_bytes(int64_t T, int64_t D, bool rms, size_t e) {
  if (T <= kFewRows) return 0;
  return (size_t)bwd_groups(bwd_shape_of(D, e), T, D, e) * (rms ? 1 : 2) * D * 4;
}

template <class E, bool RMS, int W, int NC>
static void launch_fwd(const Args& g, hipStream_t s) {
  const dim3 grid((unsigned)groups(g.T, kRows<W>, (W == 1 ? 8 : W == 4 ? 8 : 2) * dev_ncu()));
  if (g.D % Piece<E>::V == 0)
    hipLaunchKernelGGL((norm_fwd<E, RMS, W, NC, true>), grid, dim3(kThreads<W>), 0, s, g);
  else
    hipLaunchKernelGGL((norm_fwd<E, RMS, W, NC, false>), grid, dim3(kThreads<W>), 0, s, g);
}
template <class E, bool RMS>
static int fwd(const Args& g, hipStream_t s) {
  StageScope scope(STAGE_NORM_FWD, s);
  const Shape f = shape_of(g.D, E::kBytes);
  if (f.w == 1 && f.nc == 1) launch_fwd<E, RMS, 1, 1>(g, s);
  else if (f.w == 1 && f.nc == 2) launch_fwd<E, RMS, 1, 2>(g, s);
  else if (f.w == 1) launch_fwd<E, RMS, 1, 4>(g, s);
  else if (f.w == 4 && f.nc == 2) launch_fwd<E, RMS, 4, 2>(g, s);
  else if (f.w == 4) launch_fwd<E, RMS, 4, 4>(g, s);
  else if (f.w == 16) launch_fwd<E, RMS, 16, 2>(g, s);
  else
    hipLaunchKernelGGL((norm_fwd_wide<E, RMS>), dim3((unsigned)groups(g.T, 1, 2 * dev_ncu())), dim3(1024), 0, s, g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}
template <class E, bool RMS, int W, int NC>
static void launch_bwd(const Args& g, int n, hipStream_t s) {
  if (W == 16 || g.D % Piece<E>::V == 0)
    hipLaunchKernelGGL((norm_bwd<E, RMS, W, NC, true>), dim3(n), dim3(64 * W * kBwdRows<W, NC>), 0, s, g);
  else if constexpr (W < 16)
    hipLaunchKernelGGL((norm_bwd<E, RMS, W, NC, false>), dim3(n), dim3(64 * W * kBwdRows<W, NC>), 0, s, g);
}
template <class E, bool RMS>
static int bwd(const Args& g, void* dw, void* db, hipStream_t s) {
  StageScope scope(STAGE_NORM_BWD, s);
  if (g.T <= kFewRows) {  // (without a row dw and db are zeros)
    const int per = 64 * Piece<E>::V;
    hipLaunchKernelGGL((norm_bwd_few<E, RMS>), dim3((unsigned)(g.T + (g.D + per - 1) / per)), dim3(1024), 0, s, g, (char*)dw,
                       (char*)db);
    return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
  }
  const Shape f = bwd_shape_of(g.D, E::kBytes);
  const int n = bwd_groups(f, g.T, g.D, E::kBytes);
  if (f.w == 1 && f.nc == 1) launch_bwd<E, RMS, 1, 1>(g, n, s);
  else if (f.w == 1 && f.nc == 2) launch_bwd<E, RMS, 1, 2>(g, n, s);
  else if (f.w == 1) launch_bwd<E, RMS, 1, 4>(g, n, s);
  else if (f.w == 4 && f.nc == 2) launch_bwd<E, RMS, 4, 2>(g, n, s);
  else if (f.w == 4) launch_bwd<E, RMS, 4, 4>(g, n, s);
  else if (f.w == 16) launch_bwd<E, RMS, 16, 2>(g, n, s);
  else {
    hipLaunchKernelGGL((norm_bwd_wide<E, RMS>), dim3((unsigned)groups(g.T, 1, 2 * dev_ncu())), dim3(1024), 0, s, g);
    const int per = 256 * Piece<E>::V;
    hipLaunchKernelGGL((norm_wgrad_wide<E, RMS>), dim3((g.D + per - 1) / per, n), dim3(256), 0, s, g);
  }
  if (hipGetLastError() != hipSuccess) return SWIGLU_ERR_LAUNCH;
  return launch_sum_parts<E>(g.partial, n, RMS ? 1 : 2, g.D, dw, db, s);
}

template <class E>
int run_fwd(const Args& g, bool rms, hipStream_t s) {
  return rms ? fwd<E, true>(g, s) : fwd<E, false>(g, s);
}
template <class E>
int run_bwd(const Args& g, bool rms, void* dw, void* db, hipStream_t s) {
  return rms ? bwd<E, true>(g, dw, db, s) : bwd<E, false>(g, dw, db, s);
}

}  // namespace norm
}  // namespace swiglu

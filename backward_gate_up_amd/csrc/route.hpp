// route.hpp -- the router of a mixture of experts, gfx950:
//   l = x Wr^T (fp32 sums), p = softmax(l), the k largest per token in
//   descending order (equal logits: the lower index), their p as weights,
//   divided by their sum when renormalised.
//
// One launch forms the logits, with K split over workgroups where there are few
// tokens so that many CUs read the router's weight (one alone pulls 25 GB/s from
// HBM: 256 KiB took it 10 us); a second one adds the parts and picks, one wave
// per token. Few tokens: 16 experts and 16 tokens to a workgroup. Many: 32 tokens
// and every 128 experts, bound by each CU's reading of the weight from L2 (E D
// values per 32 tokens) and by LDS. Picking in the first launch measured 20 us
// more at 8192 tokens: its waves wait for one another's tokens.
//
// The order of the logits decides which experts run, so it is made exact: an
// fp32 sum is off by at most gamma |x| |w_e| (gamma counts the roundings of the
// chain, the norms are summed on the way), and logits of the leading
// candidates that lie within twice that of a neighbour are recomputed in
// fp64, the products of bf16 and fp16 being exact, before the order is taken.
#pragma once
#include "few.hpp"

namespace swiglu {
namespace route {

constexpr int kMaxExperts = few::kMaxExperts;

struct Args {
  const char* x;   // [T, D]
  const char* w;   // [E, D]
  float* wts;      // [T, k]
  int* ids;        // [T, k]
  int T, D, E, k, renorm;
  float* part;     // [splits][T][E] logits, then [splits][E] and [splits][T] sums of squares
  int splits;
  int many;        // which of the two kernels formed the logits
};

// Monotone map of fp32 to unsigned: larger value, larger key; NaN above all.
// No value has key 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return v != v ? 0xffffffffu : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k == 0xffffffffu ? 0x7fc00000u : (k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Sum of squares of a lane's 16 bytes, added to s (fp32, for the bound only).
template <class E>
__device__ __forceinline__ float add_squares(u32x4_t v, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // A copy, since a bit cast of a vector's element v[i] reads element 0.
    const uint32_t b = v[i];
    if constexpr (std::is_same<E, Bf16>::value) {
      typedef __bf16 v2 __attribute__((ext_vector_type(2)));
      s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2, b), __builtin_bit_cast(v2, b), s, false);
    } else if constexpr (std::is_same<E, Fp16>::value) {
      typedef _Float16 v2 __attribute__((ext_vector_type(2)));
      s = __builtin_amdgcn_fdot2(__builtin_bit_cast(v2, b), __builtin_bit_cast(v2, b), s, false);
    } else {
      const float f = __builtin_bit_cast(float, b);
      s = fmaf(f, f, s);
    }
  }
  return s;
}

template <class E>
__device__ __forceinline__ double chunk_dot(u32x4_t a, u32x4_t b, double s) {
  constexpr int n = 16 / E::kBytes;
  typedef typename E::elem vec __attribute__((ext_vector_type(n)));
  const vec av = __builtin_bit_cast(vec, a), bv = __builtin_bit_cast(vec, b);
#pragma unroll
  for (int i = 0; i < n; ++i) s = fma((double)E::to_f32(av[i]), (double)E::to_f32(bv[i]), s);
  return s;
}

// x[t] . w[e0] and x[t] . w[e1] in fp64 by one wave, the same on every lane.
// Two 1 KiB pieces of each row are in flight: more registers would cost
// route_pick more waves than the few tokens that come here gain.
template <class E>
__device__ __forceinline__ void exact_logits(const Args& g, int t, int e0, int e1, int lane, double (&out)[2]) {
  const int kb = g.D * E::kBytes;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc32(g.x + (int64_t)t * kb, kb);
  const __amdgpu_buffer_rsrc_t w0 = make_rsrc32(g.w + (int64_t)e0 * kb, kb);
  const __amdgpu_buffer_rsrc_t w1 = make_rsrc32(g.w + (int64_t)e1 * kb, kb);
  double s0 = 0.0, s1 = 0.0;
#pragma unroll 1
  for (int o = lane * 16; o - lane * 16 < kb; o += 2048) {
    u32x4_t a[2], b[2], c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = few::load16(xr, o + 1024 * i);
      b[i] = few::load16(w0, o + 1024 * i);
      c[i] = few::load16(w1, o + 1024 * i);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s0 = chunk_dot<E>(a[i], b[i], s0);
      s1 = chunk_dot<E>(a[i], c[i], s1);
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    s0 += __shfl_xor(s0, d);
    s1 += __shfl_xor(s1, d);
  }
  out[0] = s0;
  out[1] = s1;
}

// Largest value over the wave, on every lane: a running maximum along the
// rows of 16 lanes, then across them; lane 63 ends up with all of it.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
  return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8
  v = dpp_max<0x112, 0xf>(v);
  v = dpp_max<0x114, 0xf>(v);
  v = dpp_max<0x118, 0xf>(v);
  v = dpp_max<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_max<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Top-k, softmax and exact order of one token by one wave. l: its logits,
// expert i * 64 + lane in l[i]; bound: the largest |error| of one of them.
template <class E, int NPL>
__device__ __forceinline__ void choose(const Args& g, int t, const float (&l)[NPL], float bound, int lane) {
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = i * 64 + lane < g.E ? order_key(l[i]) : 0u;

  // Candidates in descending order of the fp32 logit, lane c holding the
  // c-th: the k largest and whatever follows within twice the bound.
  int my_id = -1, n = 0;
  float my_l = 0.f, kth = 0.f, mx = 0.f;
  const int most = min(64, g.E);
  for (; n < most; ++n) {
    uint32_t best = key[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 64 + lane;
      }
    const uint32_t top = wave_max(best);
    const uint64_t who = __ballot(best == top);
    // the lowest index among equal ones
    int e = __builtin_amdgcn_readlane(at, __ffsll((unsigned long long)who) - 1);
    for (uint64_t m = who & (who - 1); m; m &= m - 1)
      e = min(e, __builtin_amdgcn_readlane(at, __ffsll((unsigned long long)m) - 1));
    const float v = key_value(top);
    if (n == 0) mx = v;
    if (n >= g.k && !(bound > 0.f && v >= kth - 2.f * bound)) break;  // exact logits: the k first
    if (lane == n) {
      my_id = e;
      my_l = v;
    }
    if (n == g.k - 1) kth = v;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e == i * 64 + lane) key[i] = 0u;
  }
  // softmax over all experts from the fp32 logits
  float sum = 0.f;
  if (!g.renorm) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (i * 64 + lane < g.E) sum += expf(l[i] - mx);
    sum = wave_sum(sum);
  }
  // neighbours closer than the bound: both recomputed in fp64
  const float next = __shfl_down(my_l, 1), prev = __shfl_up(my_l, 1);
  const bool near =
      lane < n && ((lane + 1 < n && !(my_l - next > 2.f * bound)) || (lane > 0 && !(prev - my_l > 2.f * bound)));
  uint64_t todo = bound > 0.f ? __ballot(near) : 0ull;
  int rank = lane;
  if (todo) {
    double exact = my_l;
    while (todo) {
      const int c0 = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      const int c1 = todo ? __ffsll((unsigned long long)todo) - 1 : c0;
      todo &= todo - 1;
      double v[2];
      exact_logits<E>(g, t, __builtin_amdgcn_readlane(my_id, c0), __builtin_amdgcn_readlane(my_id, c1), lane, v);
      if (lane == c0) exact = v[0];
      else if (lane == c1) exact = v[1];
    }
    // rank among the candidates: larger first, equal ones by index; NaN first
    rank = 0;
    for (int c = 0; c < n; ++c) {
      const double v = __shfl(exact, c);
      const int id = __builtin_amdgcn_readlane(my_id, c);
      const bool vn = v != v, mn = exact != exact;
      const bool ahead = vn ? (!mn || id < my_id) : (!mn && (v > exact || (v == exact && id < my_id)));
      if (c != lane && ahead) ++rank;
    }
    my_l = (float)exact;
  }
  const bool mine = lane < n && rank < g.k;
  const float ex = mine ? expf(my_l - mx) : 0.f;
  const float den = g.renorm ? wave_sum(ex) : sum;
  if (mine) {
    g.wts[(int64_t)t * g.k + rank] = ex / den;
    g.ids[(int64_t)t * g.k + rank] = my_id;
  }
}

// Sums of squares of the operands a stream shows it (the weights' where asked).
template <class E, int NT, int MT>
struct Squares {
  bool weights;
  float x[MT] = {}, w[NT] = {};
  __device__ __forceinline__ void token(int m, u32x4_t v) { x[m] = add_squares<E>(v, x[m]); }
  __device__ __forceinline__ void weight(int n, u32x4_t v) {
    if (weights) w[n] = add_squares<E>(v, w[n]);
  }
};
// One stage's products from zero, then added: the matrix instruction rounds its
// sum in a way of its own (an error of up to 5 units of 2^-24 of the sum of
// magnitudes was measured over 32 products and the addend), so a chain of them
// loses more than a chain of additions.
template <class S, int SH, int NT, int MT, class Issue, class See>
__device__ __forceinline__ void add_stage(few::Ring<S, SH>& r, const S& st, f32x4_t (&sum)[NT][MT], int lane, Issue&& issue,
                                          See&& see) {
  f32x4_t acc[NT][MT] = {};
  r.step(st, acc, lane, issue, see);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) sum[n][m] += acc[n][m];
}
// Over the four lanes that hold one row's chunks: every lane gets row lane & 15's.
__device__ __forceinline__ float over_chunks(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Largest error of a logit over |x| |w|: two matrix instructions of 32 exact
// products, counted as 8 roundings each (fp32: eight of 4 rounded ones, 4 each),
// then the additions of the stages and of the parts; 1 % for the norms' roundings.
template <class E>
__device__ __forceinline__ float gamma_of(int stages, int parts) {
  return 1.01f * (float)((E::kBytes == 4 ? 32 : 16) + stages + parts) * 0x1p-24f;
}

// Few tokens: 16 experts (grid x), a part of K (y), XR tokens (z). 3.8 us for
// T = 1, E = 64, D = 2048, of which an empty kernel takes 1.7: latency.
constexpr int kPartWaves = 4, kMaxSplits = 4;
template <class E, int XR>
__global__ void __launch_bounds__(kPartWaves * 64, 2) route_logits(const Args g) {
  using S = few::RowStream<E, 1, XR, 1, 16384>;
  __shared__ __attribute__((aligned(1024))) char lds[kPartWaves * 16384];
  __shared__ float x2[kPartWaves][16], w2[kPartWaves][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * 16, t0 = blockIdx.z * XR, tc = min(XR, g.T - t0);
  few::Args a{};
  a.K = g.D;
  S st;
  const int kb = g.D * E::kBytes;
  st.init(a, g.x + (int64_t)t0 * kb, (uint32_t)(tc * kb), 0, lane);
  st.weight(0, few::Weight{g.w, 0}, 0, e0, g.E);
#pragma unroll
  for (int j = 0; j < S::XD; ++j) st.token_row(j, st.x_row(j, lane) < tc ? (uint32_t)st.x_row(j, lane) * kb : kOOB, lane);
  const int stages = S::stages(g.D), parts = g.splits * kPartWaves, part = blockIdx.y * kPartWaves + wave;
  int s = stages * part / parts;
  const int s1 = stages * (part + 1) / parts, n = s1 - s;
  auto issue = [&](uint32_t slot) {
    st.issue(slot, s, s < s1, lane);
    ++s;
  };
  few::Ring<S, 1> r;
  r.start(lds + wave * 16384, issue);
  f32x4_t acc[1][1] = {};
  Squares<E, 1, 1> sq{true};
#pragma unroll 1
  for (int i = 0; i < n; ++i) add_stage(r, st, acc, lane, issue, sq);
  ring::wait_vmcnt<0>();
  __syncthreads();
  float* red = (float*)lds;
  *(f32x4_t*)(red + wave * 256 + lane * 4) = acc[0][0];
  const float xv = over_chunks(sq.x[0]), wv = over_chunks(sq.w[0]);
  if (lane < 16) {
    x2[wave][lane] = xv;
    w2[wave][lane] = wv;
  }
  __syncthreads();
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4, e = e0 + col, t = t0 + row;
  const int at = ((row >> 2) * 16 + col) * 4 + (row & 3);
  float v = 0.f, vx = 0.f, vw = 0.f;
#pragma unroll
  for (int w = 0; w < kPartWaves; ++w) {
    v += red[w * 256 + at];
    vx += x2[w][row];
    vw += w2[w][col];
  }
  float* pw = g.part + (int64_t)g.splits * g.T * g.E;
  float* px = pw + g.splits * g.E;
  if (row < tc && e < g.E) g.part[((int64_t)blockIdx.y * g.T + t) * g.E + e] = v;
  if (row == 0 && blockIdx.z == 0 && e < g.E) pw[blockIdx.y * g.E + e] = vw;
  if (col == 0 && blockIdx.x == 0 && row < tc) px[(int64_t)blockIdx.y * g.T + t] = vx;
}

// Whether a row holds nothing but zeros; one wave, the same on every lane.
template <class E>
__device__ __forceinline__ bool all_zero(const char* row, int kb, int lane) {
  const __amdgpu_buffer_rsrc_t r = make_rsrc32(row, kb);
  uint32_t bits = 0;
#pragma unroll 1
  for (int o = lane * 16; o - lane * 16 < kb; o += 1024) {
    const u32x4_t v = few::load16(r, o);
    bits |= v[0] | v[1] | v[2] | v[3];
  }
  return !__any((bits & (E::kBytes == 2 ? 0x7fff7fffu : 0x7fffffffu)) != 0u);
}

// Second launch: one wave per token. T = 8192, E = 128, k = 8, D = 4096: 15 us, bound
// by its instructions (the wave-wide maxima of k rounds); 3.7 us at T = 1.
template <class E, int NPL>
__global__ void __launch_bounds__(256, NPL <= 4 ? 8 : 2) route_pick(const Args g) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= g.T) return;
  const float* pw = g.part + (int64_t)g.splits * g.T * g.E;
  const float* px = pw + g.splits * g.E;
  // all parts in flight at once; those past the splits and the experts read as zeros
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(g.part, (int64_t)g.splits * g.T * g.E * 4);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(pw, g.splits * g.E * 4);
  float l[NPL], wmax = 0.f, x2 = 0.f;
  float v[NPL][kMaxSplits], w[NPL][kMaxSplits], xp[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = i * 64 + lane;
      const bool in = e < g.E && s < g.splits;
      const uint32_t at = (uint32_t)((int64_t)s * g.T + t) * (uint32_t)g.E + e;
      v[i][s] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rp, in ? at * 4u : kOOB, 0, 0));
      w[i][s] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rw, in ? (uint32_t)(s * g.E + e) * 4u : kOOB, 0, 0));
    }
    xp[s] = s < g.splits ? px[(int64_t)s * g.T + t] : 0.f;
  }
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) x2 += xp[s];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    float sum = 0.f, sw = 0.f;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) {
      sum += v[i][s];
      sw += w[i][s];
    }
    l[i] = sum;
    wmax = fmaxf(wmax, sw);
  }
  // not negative, so the bits order as the values do
  wmax = __builtin_bit_cast(float, wave_max(__builtin_bit_cast(uint32_t, wmax)));
  const int parts = g.splits * (g.many ? 1 : kPartWaves), stages = (g.D * E::kBytes + 127) >> 7;
  // Squares and products below 2^-126 vanish, which counts as up to 2^-126 each; the
  // logits of a token of zeros (padding) are exact.
  const float least = (float)g.D * 0x1p-125f;
  const bool zeros = __builtin_expect(x2 == 0.f, 0) && all_zero<E>(g.x + (int64_t)t * g.D * E::kBytes, g.D * E::kBytes, lane);
  const float bound =
      zeros ? 0.f : gamma_of<E>((stages + parts - 1) / parts, parts) * sqrtf(x2 + least) * sqrtf(wmax + least) + least;
  choose<E, NPL>(g, t, l, bound, lane);
}

// Many tokens: 32 (grid x), a part of K (y). Each of the 4 waves takes 32 of
// every 128 experts and a quarter of the token rows' loads. T = 8192, E = 128,
// D = 4096, fp16: 22.8 us, 2.9 TB/s of tokens and 377 TFLOP/s; every 32 tokens read
// the whole weight (1 MiB), so the CUs draw 12 TB/s from L2.
constexpr int kManyTok = 32, kManyRing = 60 * 1024;
template <class E>
__global__ void __launch_bounds__(256, 2) route_logits_many(const Args g) {
  using S = few::RowStream<E, 2, kManyTok, 4, kManyRing>;
  __shared__ __attribute__((aligned(1024))) char lds[kManyRing];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * kManyTok, tc = min(kManyTok, g.T - t0);
  few::Args a{};
  a.K = g.D;
  S st;
  const int kb = g.D * E::kBytes;
  st.init(a, g.x + (int64_t)t0 * kb, (uint32_t)(tc * kb), wave, lane);
  const int xrow = st.x_row(0, lane);
  st.token_row(0, xrow < tc ? (uint32_t)xrow * kb : kOOB, lane);
  const int stages = S::stages(g.D), s0 = stages * (int)blockIdx.y / g.splits, s1 = stages * ((int)blockIdx.y + 1) / g.splits;
  const int passes = (g.E + 127) / 128;
  int s = s0, pass = 0;
  auto set_weights = [&] {
#pragma unroll
    for (int n = 0; n < 2; ++n) st.weight(n, few::Weight{g.w, 0}, 0, pass * 128 + wave * 32 + n * 16, g.E);
  };
  auto issue = [&](uint32_t slot) {
    st.issue(slot, s, s < s1 && pass < passes, lane);
    if (++s < s1) return;
    s = s0;
    if (++pass < passes) set_weights();
  };
  set_weights();
  few::Ring<S, 4> r;
  r.start(lds, issue);
  float* part = g.part + ((int64_t)blockIdx.y * g.T + t0) * g.E;
  float* pw = g.part + (int64_t)g.splits * g.T * g.E;
  float* px = pw + g.splits * g.E;
  for (int p = 0; p < passes; ++p) {
    f32x4_t acc[2][2] = {};
    Squares<E, 2, 2> sq{blockIdx.x == 0};
#pragma unroll 1
    for (int i = s0; i < s1; ++i) add_stage(r, st, acc, lane, issue, sq);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int e = p * 128 + wave * 32 + n * 16 + (lane & 15);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * m + 4 * (lane >> 4) + j;
          if (e < g.E && row < tc) part[(int64_t)row * g.E + e] = acc[n][m][j];
        }
      const float v = over_chunks(sq.w[n]);
      if (blockIdx.x == 0 && lane < 16 && e < g.E) pw[blockIdx.y * g.E + e] = v;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float v = over_chunks(sq.x[m]);
      if (p == 0 && wave == 0 && lane < 16 && 16 * m + lane < tc) px[(int64_t)blockIdx.y * g.T + t0 + 16 * m + lane] = v;
    }
  }
  ring::wait_vmcnt<0>();
}

// Which kernel forms the logits, by the tokens from which the one for many is ahead on
// most sizes (both, us): bf16 E=64, D=4096 T=512 17.8/13.5 few, T=1024 18.3/14.8, T=1536
// 18.8/19.8; E=128, D=4096 T=512 18.2/15.5, T=1024 18.2/21.1; E=256, D=7168 T=1024
// 40.4/36.5, T=1536 41.1/47.5. fp32 E=64, D=4096 T=1024 37.0/25.1, T=2048 43.6/40.1, T=4096
// 54.9/61.5; E=256, D=7168 T=1024 114/69, T=2048 116/119; E=160, D=5120 T=2048 85/73.
// (Few experts would stay with the other one for longer: E=8, D=1024 fp32 T=8192 34/17.)
static inline bool route_many(int64_t T, size_t e) { return T >= (e == 4 ? 2048 : 1024); }
// Workgroups along K: few tokens, about 128 over all, each wave with at least one
// stage; many, about two per CU.
static inline int route_splits(int64_t T, int64_t D, int64_t E, size_t e) {
  const int64_t stages = ((int64_t)D * e + 127) / 128;
  int64_t s, most;
  if (route_many(T, e)) {
    s = 512 / ((T + kManyTok - 1) / kManyTok);
    most = stages;
  } else {
    s = 128 / ((E + 15) / 16 * ((T + 15) / 16));
    most = stages / kPartWaves;
  }
  if (s > most) s = most;
  return s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : (int)s;
}
static inline size_t route_bytes(int64_t T, int64_t D, int64_t E, size_t e) {
  return T == 0 ? 0 : (size_t)route_splits(T, D, E, e) * (size_t)(T * E + E + T) * 4;
}

#define SWIGLU_ROUTE_LAUNCH(kernel, grid, threads)                               \
  do {                                                                           \
    StageScope scope(STAGE_ROUTE, stream);                                       \
    hipLaunchKernelGGL((kernel), dim3 grid, dim3(threads), 0, stream, g);        \
    if (hipGetLastError() != hipSuccess) return SWIGLU_ERR_LAUNCH;               \
  } while (0)

template <class E>
int run_route(Args g, hipStream_t stream) {
  if (g.T == 0) return SWIGLU_OK;
  g.splits = route_splits(g.T, g.D, g.E, E::kBytes);
  g.many = route_many(g.T, E::kBytes);
  const unsigned blocks = (g.E + 15) / 16, tiles = (g.T + 15) / 16;
  if (g.many) SWIGLU_ROUTE_LAUNCH((route_logits_many<E>), ((g.T + kManyTok - 1) / kManyTok, g.splits), 256);
  else if (g.T <= 8) SWIGLU_ROUTE_LAUNCH((route_logits<E, 8>), (blocks, g.splits, 1), kPartWaves * 64);
  else SWIGLU_ROUTE_LAUNCH((route_logits<E, 16>), (blocks, g.splits, tiles), kPartWaves * 64);
  const unsigned groups = (g.T + 3) / 4;
  if (g.E <= 64) SWIGLU_ROUTE_LAUNCH((route_pick<E, 1>), (groups), 256);
  else if (g.E <= 128) SWIGLU_ROUTE_LAUNCH((route_pick<E, 2>), (groups), 256);
  else if (g.E <= 256) SWIGLU_ROUTE_LAUNCH((route_pick<E, 4>), (groups), 256);
  else SWIGLU_ROUTE_LAUNCH((route_pick<E, 16>), (groups), 256);
  return SWIGLU_OK;
}
#undef SWIGLU_ROUTE_LAUNCH

}  // namespace route
}  // namespace swiglu

// route.hpp -- the router of a mixture of experts, gfx950:
//   l = x Wr^T (fp32 sums), p = softmax(l), the k largest per token in
//   descending order (equal logits: the lower index), their p as weights,
//   divided by their sum when renormalised.
//
// The order of the logits decides which experts run, so it is made exact: a
// second MFMA on the operands' magnitudes gives S = sum |x w| with each logit,
// and |error| <= gamma S bounds the fp32 rounding of its sum (gamma counts the
// roundings of the chain). Logits of the leading candidates that lie within
// twice that bound of a neighbour are recomputed in fp64, the products of
// bf16 and fp16 being exact, before the order is taken.
#pragma once
#include "few.hpp"

namespace swiglu {
namespace route {

constexpr int kTok = 16;      // tokens per workgroup: one MFMA row block
constexpr int kWaves = 8;     // waves, splitting K
constexpr int kPass = 8;      // expert blocks of 16 per pass over K
constexpr int kMaxExperts = few::kMaxExperts;

struct Args {
  const char* x;   // [T, D]
  const char* w;   // [E, D]
  float* wts;      // [T, k]
  int* ids;        // [T, k]
  int T, D, E, k, renorm;
};

// Monotone map of fp32 to unsigned: larger value, larger key; NaN above all.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  if (v != v) return 0xffffffffu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <class E>
__device__ __forceinline__ u32x4_t magnitude(u32x4_t v) {
  const uint32_t m = E::kBytes == 4 ? 0x7fffffffu : 0x7fff7fffu;
  return u32x4_t{v[0] & m, v[1] & m, v[2] & m, v[3] & m};
}

template <class E>
__device__ __forceinline__ double chunk_dot(u32x4_t a, u32x4_t b) {
  constexpr int n = 16 / E::kBytes;
  typedef typename E::elem vec __attribute__((ext_vector_type(n)));
  const vec av = __builtin_bit_cast(vec, a), bv = __builtin_bit_cast(vec, b);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < n; ++i) s = fma((double)E::to_f32(av[i]), (double)E::to_f32(bv[i]), s);
  return s;
}

// x[t] . w[e] in fp64 by one wave; the same value on every lane.
template <class E>
__device__ __forceinline__ double exact_logit(const Args& g, int t, int e, int lane) {
  const char* xr = g.x + (int64_t)t * g.D * E::kBytes;
  const char* wr = g.w + (int64_t)e * g.D * E::kBytes;
  double s = 0.0;
  for (int64_t o = lane * 16; o < (int64_t)g.D * E::kBytes; o += 1024)
    s += chunk_dot<E>(few::load16(xr + o), few::load16(wr + o));
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = max64(v, __shfl_xor(v, d));
  return v;
}

// Top-k, softmax and exact order of one token by one wave. l: its E logits
// (LDS; used up), bound: the largest |error| of one of them.
template <class E>
__device__ __forceinline__ void choose(const Args& g, int t, float* l, float bound, int lane) {
  // softmax over all experts from the fp32 logits
  float mx = -__builtin_inff();
  for (int e = lane; e < g.E; e += 64) mx = fmaxf(mx, l[e]);
#pragma unroll
  for (int d = 32; d; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  float sum = 0.f;
  for (int e = lane; e < g.E; e += 64) sum += expf(l[e] - mx);
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);

  // Candidates in descending order of the fp32 logit, lane c holding the
  // c-th: the k largest and whatever follows within twice the bound.
  int my_id = -1;
  float my_l = 0.f;
  int n = 0;
  float kth = 0.f;
  for (; n < 64 && n < g.E; ++n) {
    uint64_t best = 0;
    for (int e = lane; e < g.E; e += 64) {
      const float v = l[e];
      // chosen ones are marked by a NaN of their own; a computed NaN is never that pattern
      if (__builtin_bit_cast(uint32_t, v) != 0xffffffffu)
        best = max64(best, ((uint64_t)order_key(v) << 32) | (uint32_t)(0xffffffffu - e));
    }
    best = wave_max(best);
    const int e = (int)(0xffffffffu - (uint32_t)best);
    const float v = l[e];
    if (n >= g.k && !(v >= kth - 2.f * bound)) break;
    if (lane == n) {
      my_id = e;
      my_l = v;
    }
    if (n == g.k - 1) kth = v;
    __builtin_amdgcn_wave_barrier();
    if (lane == 0) l[e] = __builtin_bit_cast(float, 0xffffffffu);
    __builtin_amdgcn_wave_barrier();
  }
  // neighbours closer than the bound: both recomputed in fp64
  double exact = my_l;
  const float next = __shfl_down(my_l, 1), prev = __shfl_up(my_l, 1);
  const bool near = lane < n && ((lane + 1 < n && !(my_l - next > 2.f * bound)) || (lane > 0 && !(prev - my_l > 2.f * bound)));
  uint64_t todo = bound > 0.f ? __ballot(near) : 0ull;
  while (todo) {
    const int c = __ffsll((unsigned long long)todo) - 1;
    todo &= todo - 1;
    const double v = exact_logit<E>(g, t, __shfl(my_id, c), lane);
    if (lane == c) exact = v;
  }
  // rank among the candidates: larger first, equal ones by index; NaN first
  int rank = 0;
  for (int c = 0; c < n; ++c) {
    const double v = __shfl(exact, c);
    const int id = __shfl(my_id, c);
    const bool vn = v != v, mn = exact != exact;
    const bool ahead = vn ? (!mn || id < my_id) : (!mn && (v > exact || (v == exact && id < my_id)));
    if (c != lane && ahead) ++rank;
  }
  const bool mine = lane < n && rank < g.k;
  const float ex = mine ? expf((float)exact - mx) : 0.f;
  float den = sum;
  if (g.renorm) {
    den = ex;
#pragma unroll
    for (int d = 32; d; d >>= 1) den += __shfl_xor(den, d);
  }
  if (mine) {
    g.wts[(int64_t)t * g.k + rank] = ex / den;
    g.ids[(int64_t)t * g.k + rank] = my_id;
  }
}

template <class E>
__global__ void __launch_bounds__(kWaves * 64, 1) route_topk(const Args g) {
  // logits [16][E + 1], then the waves' sums of one of the two products
  extern __shared__ __attribute__((aligned(16))) float sh[];
  __shared__ uint32_t bound_bits[kTok];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * kTok, tc = min(kTok, g.T - t0);
  const int ldl = g.E + 1;
  float* logits = sh;
  float* red = sh + ((kTok * ldl + 3) & ~3);
  if (threadIdx.x < kTok) bound_bits[threadIdx.x] = 0u;
  const int64_t kb = (int64_t)g.D * E::kBytes;
  const int steps = (int)((kb + 63) >> 6), per = (steps + kWaves - 1) / kWaves;
  const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
  const int co = (lane >> 4) * 16;  // the lane's 16-byte chunk of a 64-byte step
  const char* xp = g.x + (int64_t)(t0 + min(lane & 15, tc - 1)) * kb;
  for (int b0 = 0; b0 * 16 < g.E; b0 += kPass) {
    f32x4_t acc[kPass] = {}, mag[kPass] = {};
    const int nb = min(kPass, (g.E + 15) / 16 - b0);
    for (int s = s0; s < s1; ++s) {
      const int64_t o = (int64_t)s * 64 + co;
      const bool in = o < kb;
      const u32x4_t zero{0, 0, 0, 0};
      u32x4_t xv = few::load16(xp + (in ? o : 0));
      xv = in ? xv : zero;
      const u32x4_t xm = magnitude<E>(xv);
#pragma unroll
      for (int b = 0; b < kPass; ++b) {
        if (b < nb) {
          const int row = min((b0 + b) * 16 + (lane & 15), g.E - 1);
          u32x4_t wv = few::load16(g.w + row * kb + (in ? o : 0));
          wv = in ? wv : zero;
          acc[b] = few::step_mfma<E>(xv, wv, acc[b]);
          mag[b] = few::step_mfma<E>(xm, magnitude<E>(wv), mag[b]);
        }
      }
    }
    for (int what = 0; what < 2; ++what) {
#pragma unroll
      for (int b = 0; b < kPass; ++b) *(f32x4_t*)(red + (wave * kPass + b) * 256 + lane * 4) = what ? mag[b] : acc[b];
      __syncthreads();
      for (int i = threadIdx.x; i < kPass * 256; i += kWaves * 64) {
        const int col = i & 15, row = (i >> 4) & 15, b = i >> 8;
        const int e = (b0 + b) * 16 + col;
        if (e < g.E && row < tc) {
          const int at = b * 256 + ((row >> 2) * 16 + col) * 4 + (row & 3);
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) v += red[w * kPass * 256 + at];
          // magnitudes are not negative, so their bits order as they do (a NaN
          // above all); a NaN logit takes one fixed pattern (see choose)
          if (what) atomicMax(&bound_bits[row], __builtin_bit_cast(uint32_t, fabsf(v)));
          else logits[row * ldl + e] = v != v ? __builtin_nanf("") : v;
        }
      }
      __syncthreads();
    }
  }
  // roundings of one logit's chain: a matrix instruction of 32 exact products
  // (fp32: four of 4 rounded ones) counted as 8 (16), then the waves' sums
  const float gamma = (float)(per * (E::kBytes == 4 ? 16 : 8) + kWaves) * 0x1p-24f;
  for (int r = wave; r < tc; r += kWaves)
    choose<E>(g, t0 + r, logits + r * ldl, gamma * __builtin_bit_cast(float, bound_bits[r]), lane);
}

static inline size_t lds_bytes(int E) {
  return (size_t)(((kTok * (E + 1) + 3) & ~3) + kWaves * kPass * 256) * 4;
}

template <class E>
int run_route(const Args& g, hipStream_t stream) {
  if (g.T == 0) return SWIGLU_OK;
  const size_t lds = lds_bytes(g.E);
  if (lds > 65536 &&
      hipFuncSetAttribute((const void*)route_topk<E>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
    return SWIGLU_ERR_LAUNCH;
  StageScope scope(STAGE_ROUTE, stream);
  hipLaunchKernelGGL((route_topk<E>), dim3((g.T + kTok - 1) / kTok), dim3(kWaves * 64), lds, stream, g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

}  // namespace route
}  // namespace swiglu

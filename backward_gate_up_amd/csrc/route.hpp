// route.hpp -- the router of a mixture of experts, gfx950:
//   l = x Wr^T (fp32 sums), p = softmax(l), the k largest per token in
//   descending order (equal logits: the lower index), their p as weights,
//   divided by their sum when renormalised.
//
// A workgroup takes 16 MT tokens and all experts: its NW waves split K, each
// streams the router's weight as the operand of v_mfma_f32_16x16x32 through a
// ring of registers, the sums meet in LDS, and one wave per token picks the
// experts. One token is bound by the latency of that chain, thousands by each
// CU's reading of the weight from L2 (E D values per 16 MT tokens).
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
    if constexpr (std::is_same<E, Bf16>::value) {
      typedef __bf16 v2 __attribute__((ext_vector_type(2)));
      s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2, v[i]), __builtin_bit_cast(v2, v[i]), s, false);
    } else if constexpr (std::is_same<E, Fp16>::value) {
      typedef _Float16 v2 __attribute__((ext_vector_type(2)));
      s = __builtin_amdgcn_fdot2(__builtin_bit_cast(v2, v[i]), __builtin_bit_cast(v2, v[i]), s, false);
    } else {
      const float f = __builtin_bit_cast(float, v[i]);
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
// Four 1 KiB pieces of each row are in flight.
template <class E>
__device__ __forceinline__ void exact_logits(const Args& g, int t, int e0, int e1, int lane, double (&out)[2]) {
  const int kb = g.D * E::kBytes;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc32(g.x + (int64_t)t * kb, kb);
  const __amdgpu_buffer_rsrc_t w0 = make_rsrc32(g.w + (int64_t)e0 * kb, kb);
  const __amdgpu_buffer_rsrc_t w1 = make_rsrc32(g.w + (int64_t)e1 * kb, kb);
  double s0 = 0.0, s1 = 0.0;
#pragma unroll 1
  for (int o = lane * 16; o - lane * 16 < kb; o += 4096) {
    u32x4_t a[4], b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = few::load16(xr, o + 1024 * i);
      b[i] = few::load16(w0, o + 1024 * i);
      c[i] = few::load16(w1, o + 1024 * i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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

// Top-k, softmax and exact order of one token by one wave. l: its E logits
// (LDS), bound: the largest |error| of one of them. NPL: logits per lane.
template <class E, int NPL>
__device__ __forceinline__ void choose(const Args& g, int t, const float* l, float bound, int lane) {
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = i * 64 + lane < g.E ? order_key(l[i * 64 + lane]) : 0u;

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
    if (n >= g.k && !(v >= kth - 2.f * bound)) break;
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
      if (i * 64 + lane < g.E) sum += expf(l[i * 64 + lane] - mx);
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

// NB: expert blocks of 16 per pass over K; U: steps in flight.
template <class E, int NW, int MT, int NB, int U>
__global__ void __launch_bounds__(NW * 64, 1) route_topk(const Args g) {
  constexpr int kTok = 16 * MT, kHalf = NW > 8 ? 8 : NW;
  // logits [16 MT][E + 1], then the sums of kHalf waves
  extern __shared__ __attribute__((aligned(16))) float sh[];
  __shared__ float x2[kTok], w2[kMaxExperts];
  __shared__ uint32_t w2max;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * kTok, tc = min(kTok, g.T - t0);
  const int ldl = g.E + 1;
  float* logits = sh;
  float* red = sh + ((kTok * ldl + 3) & ~3);
  for (int i = threadIdx.x; i < kTok; i += NW * 64) x2[i] = 0.f;
  for (int i = threadIdx.x; i < g.E; i += NW * 64) w2[i] = 0.f;
  if (threadIdx.x == 0) w2max = 0u;
  __syncthreads();
  const int kb = g.D * E::kBytes;
  const int steps = (kb + 63) >> 6, per = (steps + NW - 1) / NW;
  const int s0 = wave * per, s1 = min(steps, s0 + per);
  const int end = min(s1 * 64, kb);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc32(g.x + (int64_t)t0 * kb, tc * kb);
  uint32_t x_off[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x_off[m] = (uint32_t)min(16 * m + (lane & 15), tc - 1) * (uint32_t)kb;
  for (int b0 = 0; b0 * 16 < g.E; b0 += NB) {
    const int nb = min(NB, (g.E + 15) / 16 - b0), rows = min(NB * 16, g.E - b0 * 16);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc32(g.w + (int64_t)b0 * 16 * kb, rows * kb);
    const uint32_t w_off = (uint32_t)(lane & 15) * (uint32_t)kb, blk = 16u * (uint32_t)kb;
    struct Buf {
      u32x4_t x[MT], w[NB];
    } buf[U];
    // rows past E and chunks past the run or K read as zeros
    auto load = [&](Buf& b, int off) {
      const bool in = off < end;
#pragma unroll
      for (int m = 0; m < MT; ++m) b.x[m] = few::load16(xr, in ? x_off[m] + off : kOOB);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (i < nb) b.w[i] = few::load16(wr, in ? w_off + i * blk + off : kOOB);
    };
    f32x4_t acc[NB][MT] = {};
    float xs[MT] = {}, ws[NB] = {};
    int off = s0 * 64 + (lane >> 4) * 16;
#pragma unroll
    for (int u = 0; u < U; ++u) load(buf[u], off + 64 * u);
    for (int s = s0; s < s1; s += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int m = 0; m < MT; ++m) xs[m] = add_squares<E>(buf[u].x[m], xs[m]);
#pragma unroll
        for (int i = 0; i < NB; ++i)
          if (i < nb) {
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[i][m] = few::step_mfma<E>(buf[u].x[m], buf[u].w[i], acc[i][m]);
            ws[i] = add_squares<E>(buf[u].w[i], ws[i]);
          }
        load(buf[u], off + 64 * (U + u));
      }
      off += 64 * U;
    }
    // Norms: any order of these sums will do, they only decide what is recomputed.
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v = xs[m] + __shfl_xor(xs[m], 16);
      v += __shfl_xor(v, 32);
      if (b0 == 0 && lane < 16) atomicAdd(&x2[16 * m + lane], v);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (i < nb) {
        float v = ws[i] + __shfl_xor(ws[i], 16);
        v += __shfl_xor(v, 32);
        const int e = (b0 + i) * 16 + lane;
        if (lane < 16 && e < g.E) atomicAdd(&w2[e], v);
      }
    // logits: the upper half of the waves hands over to the lower, which meet in LDS
    if constexpr (NW > 8) {
      if (wave >= kHalf) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (i < nb) *(f32x4_t*)(red + (((wave - kHalf) * NB + i) * MT + m) * 256 + lane * 4) = acc[i][m];
      }
      __syncthreads();
      if (wave < NW - kHalf) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (i < nb) acc[i][m] += *(const f32x4_t*)(red + ((wave * NB + i) * MT + m) * 256 + lane * 4);
      }
    }
    if (wave < kHalf) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (i < nb) *(f32x4_t*)(red + ((wave * NB + i) * MT + m) * 256 + lane * 4) = acc[i][m];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nb * MT * 256; i += NW * 64) {
      const int col = i & 15, row = (i >> 4) & 15, m = (i >> 8) % MT, b = (i >> 8) / MT;
      const int e = (b0 + b) * 16 + col, t = 16 * m + row;
      const int at = (b * MT + m) * 256 + ((row >> 2) * 16 + col) * 4 + (row & 3);
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kHalf; ++w) v += red[w * NB * MT * 256 + at];
      if (e < g.E && t < tc) logits[t * ldl + e] = v;
    }
    __syncthreads();
  }
  // not negative, so the bits order as the values do (a NaN above all)
  for (int i = threadIdx.x; i < g.E; i += NW * 64) atomicMax(&w2max, __builtin_bit_cast(uint32_t, fabsf(w2[i])));
  __syncthreads();
  // roundings of one logit's chain: a matrix instruction of 32 exact products
  // (fp32: four of 4 rounded ones) counted as 8 (16), then the waves' sums;
  // 1 % for the roundings of the norms
  const float gamma = 1.01f * (float)(per * (E::kBytes == 4 ? 16 : 8) + NW) * 0x1p-24f;
  const float wn = __builtin_bit_cast(float, w2max);
  for (int r = wave; r < tc; r += NW) {
    const float bound = gamma * sqrtf(x2[r]) * sqrtf(wn);
    const float* l = logits + r * ldl;
    if (g.E <= 64) choose<E, 1>(g, t0 + r, l, bound, lane);
    else if (g.E <= 128) choose<E, 2>(g, t0 + r, l, bound, lane);
    else choose<E, 16>(g, t0 + r, l, bound, lane);
  }
}

template <class E, int NW, int MT, int NB, int U>
static int launch(const Args& g, hipStream_t stream) {
  const size_t lds = (size_t)(((16 * MT * (g.E + 1) + 3) & ~3) + (NW > 8 ? 8 : NW) * NB * MT * 256) * 4;
  // above 64 KiB of dynamic LDS the kernel has to be told, once per device
  static std::atomic<bool> told[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return SWIGLU_ERR_DEVICE;
  if (!told[dev].load(std::memory_order_relaxed)) {
    if (hipFuncSetAttribute((const void*)route_topk<E, NW, MT, NB, U>, hipFuncAttributeMaxDynamicSharedMemorySize,
                            152 * 1024) != hipSuccess)
      return SWIGLU_ERR_LAUNCH;
    told[dev].store(true, std::memory_order_relaxed);
  }
  StageScope scope(STAGE_ROUTE, stream);
  hipLaunchKernelGGL((route_topk<E, NW, MT, NB, U>), dim3((g.T + 16 * MT - 1) / (16 * MT)), dim3(NW * 64), lds, stream,
                     g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

template <class E>
int run_route(const Args& g, hipStream_t stream) {
  if (g.T == 0) return SWIGLU_OK;
  if (g.T > 2048 && g.E <= 128) return launch<E, 8, 2, 8, 2>(g, stream);
  if (g.E <= 64) return launch<E, 16, 1, 4, 2>(g, stream);
  return launch<E, 16, 1, 8, 1>(g, stream);
}

}  // namespace route
}  // namespace swiglu

// w4.hpp -- 4-bit weights: quantisation, the layout of few.hpp's W4Stream, and
// the way back. One pass each, mostly over HBM: 11008 x 4096 in bf16, g = 128, takes
// w4_quantize 35 us (3.25 TB/s), w4_pack 16 us (2.9: its reads of 4 bytes are 16 rows
// apart) and w4_unpack 28 us (4.1 TB/s), which long prompts pay for each weight.
#pragma once
#include "few.hpp"

namespace swiglu {
namespace w4 {

// Records of a packed weight (see few::Weight): bytes of one, records and
// bytes per expert, bytes in all.
struct Layout {
  int rec;
  int64_t recs, expert;
  size_t total;
};
static inline Layout layout(int64_t experts, int64_t N, int64_t K, int group, bool zeros) {
  Layout l;
  l.rec = 1024 + 32 * (128 / group) + (zeros ? 32 : 0);
  l.recs = ((N + 15) / 16) * ((K + 127) / 128);
  l.expert = l.recs * l.rec;
  l.total = (size_t)(experts * l.expert);
  return l;
}

// codes [X][N][K/2], scales [X][N][K/g], zeros [X][N][K/g] (or NULL) to
// records. One thread per 16-byte lane slot; rows and K past the matrix get
// code and scale 0.
__global__ void w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, char* out, Layout l,
                        int64_t experts, int N, int K, int group) {
  const int64_t n = experts * l.recs * 64;
  const int nkt = (K + 127) / 128, gp = 128 / group, ng = K / group;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    const int lane = (int)(i & 63);
    const int64_t tile = i >> 6, x = tile / l.recs, in = tile % l.recs;
    const int row = (int)(in / nkt) * 16 + (lane & 15), kt = (int)(in % nkt);
    const int64_t r = x * N + row;
    char* rec = out + tile * l.rec;
    u32x4_t v{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = kt * 128 + 32 * s + 8 * (lane >> 4);
      if (row < N && k < K) {
        const uint32_t b = *(const uint32_t*)(codes + (r * K + k) / 2);  // K is a multiple of 32
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t byte = (b >> (8 * p)) & 0xffu;
          v[s] |= ((byte & 15u) << (4 * p)) | ((byte >> 4) << (16 + 4 * p));
        }
      }
    }
    ((u32x4_t*)rec)[lane] = v;
    if (lane < 16) {
      uint32_t z = 0;
      for (int g = 0; g < gp; ++g) {
        const int at = kt * gp + g;
        const bool ok = row < N && at < ng;
        ((uint16_t*)(rec + 1024))[lane * gp + g] = ok ? scales[r * ng + at] : (uint16_t)0;
        if (zeros && ok) z |= (uint32_t)(zeros[r * ng + at] & 15) << (4 * g);
      }
      if (zeros) ((uint16_t*)(rec + 1024 + 32 * gp))[lane] = (uint16_t)z;
    }
  }
}

// Records back to rows: W = rnd(scale * (code - zero)), eight K of one row per thread.
template <class E>
__global__ void w4_unpack(const char* data, Layout l, int has_zeros, int64_t experts, int N, int K, int group,
                          typename E::elem* w) {
  const int nkt = (K + 127) / 128, gp = 128 / group, k8 = K / 8;
  const int64_t n = experts * N * k8, step = (int64_t)gridDim.x * blockDim.x;
  typedef typename E::elem vec8 __attribute__((ext_vector_type(8)));
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    const int64_t r = i / k8, x = r / N;
    const int row = (int)(r % N), k = (int)(i % k8) * 8, in = k & 127;
    const char* rec = data + x * l.expert + ((int64_t)(row >> 4) * nkt + (k >> 7)) * l.rec;
    const int lane = (row & 15) + 16 * ((in >> 3) & 3), g = in / group;
    const uint32_t v = ((const uint32_t*)rec)[lane * 4 + (in >> 5)];
    const typename E::elem sc = ((const typename E::elem*)(rec + 1024))[(row & 15) * gp + g];
    const int z = has_zeros ? (((const uint16_t*)(rec + 1024 + 32 * gp))[row & 15] >> (4 * g)) & 15 : 8;
    vec8 o;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      o[2 * p] = E::from_f32(E::to_f32(sc) * (float)((int)((v >> (4 * p)) & 15u) - z));
      o[2 * p + 1] = E::from_f32(E::to_f32(sc) * (float)((int)((v >> (16 + 4 * p)) & 15u) - z));
    }
    *(vec8*)(w + r * K + k) = o;
  }
}

// Quantisation of rows to codes, scales (and zero points). Without zero
// points: scale = rnd(max |w| / 7.5), code = clamp(round(w / scale) + 8); with
// them: scale = rnd((max(w, 0) - min(w, 0)) / 15), zero = round(-min / scale),
// code = clamp(round(w / scale) + zero). The rounded scale is the one that is
// divided by. A NaN makes its group's scale NaN, so that no finite weight stands in
// its place. Eight elements per thread; a group is 4 to 16 neighbouring lanes.
template <class E>
__global__ void w4_quantize(const typename E::elem* w, int64_t n8, int group, uint32_t* codes,
                            typename E::elem* scales, uint8_t* zeros) {
  typedef typename E::elem vec8 __attribute__((ext_vector_type(8)));
  const int lanes = group / 8;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  // every lane of a wave takes part in the exchanges: the bound is rounded up to a wave
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < ((n8 + 63) & ~(int64_t)63); i += step) {
    const bool in = i < n8;
    const vec8 v = *(const vec8*)(w + (in ? i : 0) * 8);
    float lo = 0.f, hi = 0.f;
    int nan = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      nan |= v[j] != v[j];
      lo = fminf(lo, E::to_f32(v[j]));
      hi = fmaxf(hi, E::to_f32(v[j]));
    }
    for (int d = 1; d < lanes; d <<= 1) {
      lo = fminf(lo, __shfl_xor(lo, d));
      hi = fmaxf(hi, __shfl_xor(hi, d));
      nan |= __shfl_xor(nan, d);
    }
    const typename E::elem sc =
        E::from_f32(nan ? __builtin_nanf("") : zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.5f);
    const float sf = E::to_f32(sc);
    const float z = zeros ? (sf > 0.f ? fminf(fmaxf(rintf(-lo / sf), 0.f), 15.f) : 0.f) : 8.f;
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = sf > 0.f ? rintf(E::to_f32(v[j]) / sf) + z : z;
      c |= (uint32_t)fminf(fmaxf(q, 0.f), 15.f) << (4 * j);
    }
    if (!in) continue;
    codes[i] = c;
    if (i % lanes == 0) {
      scales[i / lanes] = sc;
      if (zeros) zeros[i / lanes] = (uint8_t)z;
    }
  }
}

}  // namespace w4
}  // namespace swiglu

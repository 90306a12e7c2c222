// few.hpp -- products of few token rows with streamed weights, gfx950: the
// SwiGLU block as one dense MLP or as a mixture of experts, with weights in
// the nn.Linear layout (16-bit or fp32 rows) or as 4-bit codes.
//
//   gate/up   A[p] = SiLU(x[t] Wg_e^T) * (x[t] Wu_e^T)      p = (token t, choice j), e = ids[p]
//   down      y[t] = sum over the token's pairs p of w[p] (A[p] Wd_e^T)
//
// A dense block is the case of one expert that every token chooses with
// weight 1; a plain 4-bit product y = x W^T is its down kernel alone.
//
// What bounds it: with a handful of tokens per expert each weight is used a
// few times, so the time is that of reading the chosen experts' weights once
// from HBM. A wave streams 16 weight rows (an MFMA column block) straight
// into registers, 16 bytes per lane in the operand order of
// v_mfma_f32_16x16x32 (lane l: row l % 16, 16-byte chunk l / 16 of each
// 64-byte step), so no weight passes through LDS. Tokens are the MFMA's other
// operand: row l % 16 of the expert's token list, gathered. Rows past the
// list repeat its last token and are dropped afterwards: an MFMA row depends
// on no other row, so neither they nor another token's NaN can leak.
//
// Experts are visited per chunk of 64 tokens (grid z): each workgroup reads
// the chunk's ids, finds its expert as the n-th one that occurs, and lists
// the pairs that chose it. ids outside [0, E) choose nothing. No sorting pass,
// no atomics on results; every sum is formed in a fixed order.
#pragma once
#include "kernels.hpp"

namespace swiglu {
namespace few {

constexpr int kChunk = 64;              // tokens per grid z slice
constexpr int kMaxTopK = 32;            // choices per token
constexpr int kMaxPairs = kChunk * kMaxTopK;
constexpr int kMaxExperts = 1024;

// One weight as the kernels address it. Rows: E matrices [N, K], row-major.
// 4 bits: per 16 rows and 128 K one tile of 1 KiB, lane l's 16 bytes holding
// row l % 16, K 32 s + 8 (l / 16) .. + 7 in dword s; inside a dword the
// nibble of the even K 2p is at bit 4p, of the odd K 2p + 1 at bit 16 + 4p.
// Scales [E][N/16][K/128][16][128/g] in the storage type; zero points
// [E][N/16][K/128][16] as 128/g nibbles of a 16-bit word.
struct Weight {
  const char* w;
  const char* scale;
  const char* zero;  // nullptr: every zero point is 8
  int64_t expert;    // bytes (rows) or 1 KiB tiles (4 bits) per expert
};

struct Args {
  const char* x;     // gate/up: [T, K] tokens; down: [T * k, K] pairs (dense: [T, K])
  Weight w0, w1;     // gate/up: gate and up; down: w0
  char* out;         // gate/up: A [T * k, N]; down: y [T, N]
  const int* ids;    // [T, k]; nullptr: dense
  const float* wts;  // [T, k]; nullptr: dense
  int T, k, E, N, K;
  uint32_t kinv;     // ceil(65536 / k): p / k = p * kinv >> 16 for a chunk's p < 2048, k <= 32
};

// ---- MFMA steps -------------------------------------------------------------
// c[token row 4 (l / 16) + j][weight row l % 16] += a (tokens) . w (weights)
// over one 64-byte step of K.
template <class E>
__device__ __forceinline__ f32x4_t step_mfma(u32x4_t a, u32x4_t w, f32x4_t c) {
  if constexpr (std::is_same<E, Bf16>::value) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, w), c,
                                                   0, 0, 0);
  } else if constexpr (std::is_same<E, Fp16>::value) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, w), c, 0,
                                                  0, 0);
  } else {
    // fp32: four 16x16x4 products; the i-th takes element i of every lane's
    // chunk, K = 4 (l / 16) + i of the step on both sides
    const f32x4_t af = __builtin_bit_cast(f32x4_t, a), wf = __builtin_bit_cast(f32x4_t, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(af[i], wf[i], c, 0, 0, 0);
    return c;
  }
}

__device__ __forceinline__ u32x4_t load16(const char* p) { return *(const u32x4_t*)p; }
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// ---- weight streams ---------------------------------------------------------
// A stream adds the products of K steps [s0, s1) to acc[n][m]: NT weight blocks
// of 16 rows x MT token blocks of 16. A ring of U steps stays in flight: each
// step's registers are refilled as soon as its products are issued. Offsets
// past the end of the run or of K go out of the buffers' range, so those loads
// return zeros without a memory access: no remainder code, and neither the next
// row nor a NaN there is multiplied in.
//
// Tokens: rows of K elements at row_off[m] from x (bytes).

// Rows of 16-bit or fp32 weights; a step is 64 bytes of K.
// R: registers a lane may hold (512 per SIMD lane over its waves).
template <class E, int NT, int MT, int R>
struct RowStream {
  static constexpr int kFit = (R - 40 - 4 * NT * MT) / (4 * (NT + MT));
  static constexpr int U = kFit >= 16 ? 16 : kFit >= 8 ? 8 : 4;
  __amdgpu_buffer_rsrc_t w[NT], x;
  uint32_t w_off, x_off[MT];
  int kb;  // bytes of K

  __device__ __forceinline__ void init(const Weight* const (&wt)[NT], int e, int row0, int N, int K, const char* xb,
                                       const uint32_t (&row_off)[MT], uint32_t x_bytes, int lane) {
    kb = K * E::kBytes;
    const int rows = min(16, N - row0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      w[n] = make_rsrc32(wt[n]->w + (int64_t)e * wt[n]->expert + (int64_t)row0 * kb, rows * kb);
    x = make_rsrc32(xb, (int)x_bytes);
    w_off = (uint32_t)min(lane & 15, rows - 1) * (uint32_t)kb;
#pragma unroll
    for (int m = 0; m < MT; ++m) x_off[m] = row_off[m];
  }
  static __device__ __forceinline__ int steps(int K) { return (K * E::kBytes + 63) >> 6; }

  struct Buf {
    u32x4_t w[NT], x[MT];
  };
  __device__ __forceinline__ void load(Buf& b, int off, int end) const {
    const bool in = off < end;
#pragma unroll
    for (int n = 0; n < NT; ++n) b.w[n] = load16(w[n], in ? w_off + off : kOOB);
#pragma unroll
    for (int m = 0; m < MT; ++m) b.x[m] = load16(x, in ? x_off[m] + off : kOOB);
  }
  __device__ __forceinline__ void run(f32x4_t (&acc)[NT][MT], int s0, int s1, int lane) const {
    const int end = min(s1 * 64, kb);
    int off = s0 * 64 + (lane >> 4) * 16;
    Buf b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(b[u], off + 64 * u, end);
    for (int s = s0; s < s1; s += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[n][m] = step_mfma<E>(b[u].x[m], b[u].w[n], acc[n][m]);
        load(b[u], off + 64 * (U + u), end);
      }
      off += 64 * U;
    }
  }
};

// 4-bit codes; a step is one tile of 128 K. The products run on integers: the
// nibble q goes into the mantissa of 128 (bf16) or 64 (fp16), which makes the
// operand OFF + q exactly with one shift and one and-or per two values. Per
// group of g the fp32 sum of x (OFF + q) is corrected by (OFF + z) times the
// sum of x (one more MFMA against ones, shared by all weight blocks) and
// scaled, so a scale costs two operations per output and group and no weight is
// rounded. The offset costs accuracy of about OFF / 5 fp32 roundings of the
// group's sum, 2^-19 of it in bf16: far below the storage type's half step.
template <class E, int G, int NT, int MT, int R>
struct W4Stream {
  static constexpr int GP = 128 / G;  // groups per tile
  static constexpr int U = R < 256 || MT > 1 ? 1 : 2;
  static constexpr float kOff = std::is_same<E, Bf16>::value ? 128.0f : 64.0f;
  __amdgpu_buffer_rsrc_t w[NT], s[NT], z[NT], x;
  uint32_t x_off[MT];
  int kb, lane;
  bool has_zero;

  __device__ __forceinline__ void init(const Weight* const (&wt)[NT], int e, int row0, int N, int K, const char* xb,
                                       const uint32_t (&row_off)[MT], uint32_t x_bytes, int ln) {
    const int nkt = steps(K);
    kb = K * 2;
    lane = ln;
    has_zero = wt[0]->zero != nullptr;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int64_t tile = (int64_t)e * wt[n]->expert + (int64_t)(row0 >> 4) * nkt;
      w[n] = make_rsrc32(wt[n]->w + tile * 1024, nkt * 1024);
      s[n] = make_rsrc32(wt[n]->scale + tile * (32 * GP), nkt * (32 * GP));
      z[n] = make_rsrc32(wt[n]->zero + tile * 32, has_zero ? nkt * 32 : 0);
    }
    x = make_rsrc32(xb, (int)x_bytes);
#pragma unroll
    for (int m = 0; m < MT; ++m) x_off[m] = row_off[m];
  }
  static __device__ __forceinline__ int steps(int K) { return (K + 127) >> 7; }

  struct Buf {
    u32x4_t w[NT], x[4][MT];
    uint32_t s[NT][GP == 4 ? 2 : 1];
    uint32_t z[NT];
  };
  __device__ __forceinline__ void load(Buf& b, int t, int end) const {
    const bool in = t < end;
    const uint32_t row = lane & 15;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      b.w[n] = load16(w[n], in ? (uint32_t)t * 1024 + lane * 16 : kOOB);
      const uint32_t so = in ? ((uint32_t)t * 16 + row) * (2 * GP) : kOOB;
      if constexpr (GP == 1) b.s[n][0] = __builtin_amdgcn_raw_buffer_load_b16(s[n], so, 0, 0);
      else if constexpr (GP == 2) b.s[n][0] = __builtin_amdgcn_raw_buffer_load_b32(s[n], so, 0, 0);
      else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(s[n], so, 0, 0);
        b.s[n][0] = v[0];
        b.s[n][1] = v[1];
      }
      b.z[n] = 0x8888u;
      if (has_zero) b.z[n] = __builtin_amdgcn_raw_buffer_load_b16(z[n], in ? ((uint32_t)t * 16 + row) * 2 : kOOB, 0, 0);
    }
    const int off = t * 256 + (lane >> 4) * 16, xe = in ? kb : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) b.x[i][m] = load16(x, off + 64 * i < xe ? x_off[m] + off + 64 * i : kOOB);
  }
  // eight codes of one dword as the MFMA operand OFF + q
  static __device__ __forceinline__ u32x4_t widen(uint32_t v) {
    if constexpr (std::is_same<E, Bf16>::value) {
      constexpr uint32_t m = 0x000f000fu, o = 0x43004300u;  // 128 + q: mantissa step 1
      return u32x4_t{(v & m) | o, ((v >> 4) & m) | o, ((v >> 8) & m) | o, ((v >> 12) & m) | o};
    } else {
      constexpr uint32_t m = 0x00f000f0u, o = 0x54005400u;  // 64 + q: mantissa step 1/16
      return u32x4_t{((v << 4) & m) | o, (v & m) | o, ((v >> 4) & m) | o, ((v >> 8) & m) | o};
    }
  }
  static __device__ __forceinline__ u32x4_t ones() {
    constexpr uint32_t o = std::is_same<E, Bf16>::value ? 0x3f803f80u : 0x3c003c00u;
    return u32x4_t{o, o, o, o};
  }
  static __device__ __forceinline__ float scale_of(const uint32_t (&s)[GP == 4 ? 2 : 1], int g) {
    const uint32_t h = (s[g >> 1] >> ((g & 1) * 16)) & 0xffffu;
    return E::to_f32(__builtin_bit_cast(typename E::elem, (uint16_t)h));
  }
  __device__ __forceinline__ void tile(const Buf& b, f32x4_t (&acc)[NT][MT]) const {
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      f32x4_t part[NT][MT] = {}, xs[MT] = {};
#pragma unroll
      for (int i = 4 / GP * g; i < 4 / GP * (g + 1); ++i) {
#pragma unroll
        for (int m = 0; m < MT; ++m) xs[m] = step_mfma<E>(b.x[i][m], ones(), xs[m]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const u32x4_t q = widen(b.w[n][i]);
#pragma unroll
          for (int m = 0; m < MT; ++m) part[n][m] = step_mfma<E>(b.x[i][m], q, part[n][m]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float sc = scale_of(b.s[n], g);
        const float off = kOff + (float)((b.z[n] >> (4 * g)) & 15u);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][m][j] = fmaf(sc, fmaf(-off, xs[m][j], part[n][m][j]), acc[n][m][j]);
      }
    }
  }
  __device__ __forceinline__ void run(f32x4_t (&acc)[NT][MT], int s0, int s1, int) const {
    Buf b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(b[u], s0 + u, s1);
    for (int t = s0; t < s1; t += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Buf c = b[u];
        load(b[u], t + U + u, s1);
        tile(c, acc);
      }
    }
  }
};

// FMT 0: rows; 32, 64, 128: 4 bits with groups of that size
template <class E, int FMT, int NT, int MT, int R>
struct StreamOf {
  using type = W4Stream<E, FMT, NT, MT, R>;
};
template <class E, int NT, int MT, int R>
struct StreamOf<E, 0, NT, MT, R> {
  using type = RowStream<E, NT, MT, R>;
};

// ---- a chunk's choices --------------------------------------------------------
// ids of the chunk's pairs, and the experts that occur, in ascending order.
struct Choices {
  int16_t id[kMaxPairs];          // -1: chooses nothing
  int16_t expert[kMaxExperts];    // n-th expert that occurs
  unsigned seen[kMaxExperts / 32];
  int hits;
};

// All threads; ends with a barrier.
__device__ __forceinline__ void read_choices(Choices& c, const Args& g, int t0, int tc) {
  const int P = tc * g.k;
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += blockDim.x) c.seen[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < P; i += blockDim.x) {
    const int e = g.ids[(int64_t)t0 * g.k + i];
    const bool ok = (unsigned)e < (unsigned)g.E;
    c.id[i] = ok ? (int16_t)e : (int16_t)-1;
    if (ok) atomicOr(&c.seen[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const int words = (g.E + 31) >> 5;
    unsigned v = lane < words ? c.seen[lane] : 0u;
    int before = __popc(v);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up(before, d);
      if (lane >= d) before += o;
    }
    if (lane == 31) c.hits = before;
    before -= __popc(v);
    while (v) {
      c.expert[before++] = (int16_t)(lane * 32 + __ffs((int)v) - 1);
      v &= v - 1;
    }
  }
  __syncthreads();
}

// One wave: the pairs that chose e, ranks [64 pass, 64 pass + 64), into
// list[0 .. 63] in ascending order. Returns how many pairs chose e in all.
__device__ __forceinline__ int list_pairs(const Choices& c, int P, int e, int pass, int16_t* list, int lane) {
  int n = 0;
  for (int r = 0; r < P; r += 64) {
    const bool hit = r + lane < P && c.id[r + lane] == e;
    const uint64_t m = __ballot(hit);
    const int at = n + __popcll(m & ((1ull << lane) - 1)) - 64 * pass;
    if (hit && at >= 0 && at < 64) list[at] = (int16_t)(r + lane);
    n += __popcll(m);
  }
  // the list is this wave's own: wait for its writes, no barrier
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return n;
}

// ---- gate/up ------------------------------------------------------------------
// NW waves split K. Registers per lane: two workgroups of 4 waves or one of 8
// share a CU's four SIMDs, so 256.
template <class E, int FMT, int NW, int MT>
__device__ __forceinline__ void gateup_block(const Args& g, int e, int row0, int t0, const int16_t* list, int n,
                                             float* red) {
  using S = typename StreamOf<E, FMT, 2, MT, 256>::type;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = min(16 * m + (lane & 15), n - 1);
    row[m] = (uint32_t)(list ? (list[i] * g.kinv) >> 16 : i) * (uint32_t)(g.K * E::kBytes);
  }
  S s;
  const Weight* const w[2] = {&g.w0, &g.w1};
  s.init(w, e, row0, g.N, g.K, g.x + (int64_t)t0 * g.K * E::kBytes, row, (uint32_t)(min(kChunk, g.T - t0) * g.K) * E::kBytes,
         lane);
  const int steps = S::steps(g.K), per = (steps + NW - 1) / NW;
  f32x4_t acc[2][MT] = {};
  s.run(acc, wave * per, min(steps, (wave + 1) * per), lane);
  // the waves' sums meet in LDS; thread -> (token row, hidden column), waves added in order
#pragma unroll
  for (int n2 = 0; n2 < 2; ++n2)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *(f32x4_t*)(red + (((wave * 2 + n2) * MT + m) * 64 + lane) * 4) = acc[n2][m];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 256; i += NW * 64) {
    const int col = i & 15, row = i >> 4;  // token row of the list, hidden column
    const int at = ((row >> 4) * 64 + ((row & 15) >> 2) * 16 + col) * 4 + (row & 3);
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      gate += red[(v * 2 + 0) * MT * 256 + at];
      up += red[(v * 2 + 1) * MT * 256 + at];
    }
    const int h = row0 + col;
    if (row < n && h < g.N) {
      const int64_t p = list ? (int64_t)t0 * g.k + list[row] : t0 + row;
      // g and u stay in fp32; A is rounded once, to the storage type the
      // down projection's matrix instructions take
      ((typename E::elem*)g.out)[p * g.N + h] = E::from_f32(gate * sigmoid_f32<E>(gate) * up);
    }
  }
  __syncthreads();
}

template <class E, int FMT, int NW>
__global__ void __launch_bounds__(NW * 64, 2) few_gateup(const Args g) {
  __shared__ Choices ch;
  __shared__ int16_t list[64];
  __shared__ int count;  // pairs that chose the workgroup's expert
  __shared__ __attribute__((aligned(16))) float red[NW * 2 * 4 * 256];
  const int t0 = blockIdx.z * kChunk, tc = min(kChunk, g.T - t0);
  const int row0 = blockIdx.x * 16;
  int e = 0, total = tc;
  const bool routed = g.ids != nullptr;
  if (routed) {
    read_choices(ch, g, t0, tc);
    if ((int)blockIdx.y >= ch.hits) return;
    e = ch.expert[blockIdx.y];
  }
  for (int pass = 0; 64 * pass < total; ++pass) {
    if (routed) {
      if (threadIdx.x < 64) {
        const int n = list_pairs(ch, tc * g.k, e, pass, list, threadIdx.x);
        if (threadIdx.x == 0) count = n;
      }
      __syncthreads();
      total = count;
    }
    const int n = min(64, total - 64 * pass);
    const int16_t* l = routed ? list : nullptr;
    if (n <= 16) gateup_block<E, FMT, NW, 1>(g, e, row0, t0, l, n, red);
    else if (n <= 32) gateup_block<E, FMT, NW, 2>(g, e, row0, t0, l, n, red);
    else gateup_block<E, FMT, NW, 4>(g, e, row0, t0, l, n, red);
  }
}

// ---- down -----------------------------------------------------------------------
// The K axis of an output tile is the list of (expert that occurs, K step); the
// workgroup's NW waves take equal runs of it. At an expert's end the block of
// sums is weighted and added to the wave's own [token][column] tile in LDS.
template <int NW>
struct DownShared {
  Choices ch;
  float wts[kMaxPairs];
  int16_t list[NW][64];
  float y[NW][kChunk * 16];
};

template <class E, int FMT, int NW, int MT>
__device__ __forceinline__ void down_block(const Args& g, DownShared<NW>& sh, int e, int row0, int t0, int n, int s0,
                                           int s1) {
  using S = typename StreamOf<E, FMT, 1, MT, NW == 16 ? 128 : 256>::type;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool routed = g.ids != nullptr;
  const int16_t* list = sh.list[wave];
  uint32_t row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = min(16 * m + (lane & 15), n - 1);
    row[m] = (uint32_t)(routed ? list[i] : i) * (uint32_t)(g.K * E::kBytes);
  }
  S s;
  const Weight* const w[1] = {&g.w0};
  s.init(w, e, row0, g.N, g.K, g.x + (int64_t)t0 * g.k * g.K * E::kBytes, row,
         (uint32_t)(min(kChunk, g.T - t0) * g.k * g.K) * E::kBytes, lane);
  f32x4_t acc[1][MT] = {};
  s.run(acc, s0, s1, lane);
  float* y = sh.y[wave];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    // one group of 16 lanes (4 token rows) at a time: a token listed twice
    // for one expert is then added twice, in order
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      if ((lane >> 4) == q) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 16 * m + 4 * q + j;
          if (i < n) {
            const int p = routed ? list[i] : i;
            float* at = y + (routed ? (p * g.kinv) >> 16 : (uint32_t)p) * 16 + (lane & 15);
            *at += (routed ? sh.wts[p] : 1.0f) * acc[0][m][j];
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

template <class E, int FMT, int NW>
__global__ void __launch_bounds__(NW * 64, NW == 16 ? 4 : 2) few_down(const Args g) {
  __shared__ __attribute__((aligned(16))) DownShared<NW> sh;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.z * kChunk, tc = min(kChunk, g.T - t0);
  const int row0 = blockIdx.x * 16;
  const bool routed = g.ids != nullptr;
  int hits = 1;
  if (routed) {
    for (int i = threadIdx.x; i < tc * g.k; i += blockDim.x) sh.wts[i] = g.wts[(int64_t)t0 * g.k + i];
    read_choices(sh.ch, g, t0, tc);
    hits = sh.ch.hits;
  }
  for (int i = lane; i < tc * 16; i += 64) sh.y[wave][i] = 0.f;
  const int steps = StreamOf<E, FMT, 1, 1, 256>::type::steps(g.K);
  const int all = hits * steps;
  int at = (int)((int64_t)all * wave / NW);
  const int end = (int)((int64_t)all * (wave + 1) / NW);
  while (at < end) {
    const int slot = at / steps, s0 = at - slot * steps, s1 = min(steps, s0 + (end - at));
    const int e = routed ? sh.ch.expert[slot] : 0;
    int total = tc;
    for (int pass = 0; 64 * pass < total; ++pass) {
      if (routed) total = list_pairs(sh.ch, tc * g.k, e, pass, sh.list[wave], lane);
      const int n = min(64, total - 64 * pass);
      if (n <= 16) down_block<E, FMT, NW, 1>(g, sh, e, row0, t0, n, s0, s1);
      else if (n <= 32) down_block<E, FMT, NW, 2>(g, sh, e, row0, t0, n, s0, s1);
      else down_block<E, FMT, NW, 4>(g, sh, e, row0, t0, n, s0, s1);
    }
    at += s1 - s0;
  }
  __syncthreads();
  // four columns of one token per thread; the waves' sums in order
  for (int i = threadIdx.x; i < tc * 4; i += blockDim.x) {
    f32x4_t v{};
#pragma unroll
    for (int w = 0; w < NW; ++w) v += *(const f32x4_t*)(sh.y[w] + i * 4);
    const int t = t0 + (i >> 2), n = row0 + (i & 3) * 4;
    if (n >= g.N) continue;  // N is a multiple of 8: all four columns or none
    typename E::vec4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = E::from_f32(v[j]);
    *(typename E::vec4*)((typename E::elem*)g.out + (int64_t)t * g.N + n) = o;
  }
}

// ---- launches ---------------------------------------------------------------------
// A whole call; the host has checked it.
struct Call {
  const char* x;
  Weight wg, wu, wd;  // linear: wd only
  char* a;            // workspace: the A plane, [T * k, H]
  char* y;
  const int* ids;
  const float* wts;
  int64_t T, D, H;
  int k, E;
  hipStream_t stream;
};

template <class E, int FMT, int NW>
static int launch_gateup(const Args& g, int slots, hipStream_t s) {
  StageScope scope(STAGE_FEW_GATEUP, s);
  const dim3 grid((g.N + 15) / 16, slots, (g.T + kChunk - 1) / kChunk);
  hipLaunchKernelGGL((few_gateup<E, FMT, NW>), grid, dim3(NW * 64), 0, s, g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}
template <class E, int FMT, int NW>
static int launch_down(const Args& g, hipStream_t s) {
  StageScope scope(STAGE_FEW_DOWN, s);
  const dim3 grid((g.N + 15) / 16, 1, (g.T + kChunk - 1) / kChunk);
  hipLaunchKernelGGL((few_down<E, FMT, NW>), grid, dim3(NW * 64), 0, s, g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

// y = x W^T (dense), or the down projection of a block.
template <class E, int FMT>
int run_down(const Call& c, const char* x, int64_t K, int64_t N) {
  const Args g{x, c.wd, c.wd, c.y, c.ids, c.wts, (int)c.T, c.k, c.E, (int)N, (int)K, (65535u + c.k) / c.k};
  const int64_t groups = (N + 15) / 16 * ((c.T + kChunk - 1) / kChunk);
  if (groups >= 1024) return launch_down<E, FMT, 4>(g, c.stream);
  if (groups >= 512 || c.T > 16) return launch_down<E, FMT, 8>(g, c.stream);
  return launch_down<E, FMT, 16>(g, c.stream);
}

template <class E, int FMT>
int run_block(const Call& c) {
  const Args g{c.x, c.wg, c.wu, c.a, c.ids, c.wts, (int)c.T, c.k, c.E, (int)c.H, (int)c.D, (65535u + c.k) / c.k};
  const int64_t pairs = (c.T < kChunk ? c.T : kChunk) * c.k;
  const int slots = c.ids ? (int)(pairs < c.E ? pairs : c.E) : 1;
  const int64_t groups = (c.H + 15) / 16 * slots * ((c.T + kChunk - 1) / kChunk);
  const int rc = groups >= 512 ? launch_gateup<E, FMT, 4>(g, slots, c.stream) : launch_gateup<E, FMT, 8>(g, slots, c.stream);
  return rc ? rc : run_down<E, FMT>(c, c.a, c.H, c.D);
}

}  // namespace few
}  // namespace swiglu

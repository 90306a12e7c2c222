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
// from HBM. Every wave streams its own run of K through a private ring in LDS
// with direct-to-LDS loads of whole 128-byte lines (16 weight rows and the
// expert's token rows side by side), and reads them back as the operands of
// v_mfma_f32_16x16x32; the waves never wait for one another inside the run.
// Loading the operands straight into registers measured 27 GB/s per CU: a
// wave's 64 lanes then touch 16 rows, neighbouring lanes different lines, and
// the address unit takes each 16-byte piece on its own.
//
// Rows of the token operand past the expert's list are zeros or repeats and
// are dropped afterwards: an MFMA row depends on no other row, so neither
// they nor another token's NaN can leak.
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
// 4 bits: E x [N/16][K/128] records, each 1 KiB of codes (lane l's 16 bytes
// hold row l % 16, K 32 s + 8 (l / 16) .. + 7 in dword s; inside a dword the
// nibble of the even K 2p is at bit 4p, of the odd K 2p + 1 at bit 16 + 4p),
// then the scales [16][128/g] in the storage type, then, where the weight has
// zero points, 16 words of 16 bits with 128/g nibbles each.
struct Weight {
  const char* w;
  int64_t expert;  // bytes per expert
};

struct Args {
  const char* x;     // gate/up: [T, K] tokens; down: [T * k, K] pairs (dense: [T, K])
  Weight w0, w1;     // gate/up: gate and up; down: w0
  char* out;         // gate/up: A [T * k, N] (in two parts [T * k][2][N]); down: y [T, N]
  const int* ids;    // [T, k]; nullptr: dense
  const float* wts;  // [T, k]; nullptr: dense
  int T, k, E, N, K;
  uint32_t kinv;     // ceil(65536 / k): p / k = p * kinv >> 16 for a chunk's p < 2048, k <= 32
  int zeros;         // 4 bits: the weights have zero points (else every one is 8)
  int once;          // rows of whole 128-byte lines, read once
  int splits;        // down: workgroups per output tile
  float* partial;    // down, splits > 1: [splits][T][N]
  unsigned* ctr;     // gate/up: n_ctr arrival counters to clear for the down launch;
  int n_ctr;         // down, splits > 1: one per (chunk, output tile)
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

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// A descriptor that is the same on every lane, in scalar registers, as the loads
// from inline assembly take it. A vector instruction's write of a scalar
// register needs 5 wait states before a memory instruction reads it, and the
// compiler does not know that the assembly is one: they are put here.
// (tests/test_serve_isa.py looks for such pairs in the compiled kernels.)
__device__ __forceinline__ i32x4_t scalar_rsrc(i32x4_t r) {
#pragma unroll
  for (int i = 0; i < 3; ++i) r[i] = __builtin_amdgcn_readfirstlane(r[i]);
  r[3] = kRsrcWord3;
  asm volatile("s_nop 4" : "+s"(r));
  return r;
}

// dma16 for whole lines that are read once: a non-temporal load leaves L2 to the
// tokens (T = 16, E = 64: 165 -> 147 us; where rows share lines, K = 1000, they
// come twice and it costs 20 %).
__device__ __forceinline__ void dma16_once(uint32_t lds, i32x4_t rs, uint32_t voff, uint32_t soff) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  soff = __builtin_amdgcn_readfirstlane(soff);
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds" ::"v"(voff), "s"(rs), "s"(soff), "{m0}"(lds)
               : "memory");
}

// Four bytes per lane to LDS address lds + 4 * lane (see dma16).
__device__ __forceinline__ void dma4(uint32_t lds, i32x4_t rs, uint32_t voff, uint32_t soff) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  soff = __builtin_amdgcn_readfirstlane(soff);
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(rs), "s"(soff), "{m0}"(lds)
               : "memory");
}

// ---- streams ------------------------------------------------------------------
// A stage holds some K of NT weight blocks of 16 rows and of XR token rows; its
// products are added to acc[n][m]. A wave's stages run through its ring of NS
// slots: a stage waits for its own loads only (vmcnt counts a wave's loads in
// issue order), its slot is read, and refilled with the stage NS further on,
// of whichever weight rows or expert that belongs to. Stages past the end and
// bytes past K are asked for beyond the buffers' range, which loads zeros
// without a memory access: no remainder code, and neither the next row nor a
// NaN there is multiplied in.
//
// XR: token rows per stage, 16 to 64, or fewer (what one load instruction
// covers): then rows XR .. 15 of the operand repeat them. A longer list of
// tokens takes several passes over the weights.
//
// SH: waves that share the token rows. 1: the ring is the wave's own, with rows
// and weights side by side, and the waves split K. Else the ring is those
// waves' together: each loads its part of the rows and its own weight blocks,
// and they split the weight rows. With more than 16 token rows a private copy
// of them would leave no LDS for weights in flight.

// Rows of 16-bit or fp32 values: a stage is 128 bytes of K, 16 rows x 128 B in
// two loads of 8 rows. Chunk c of row r sits at position c ^ kc_swz(r), so the
// 16 rows one read takes fall on distinct banks.
template <class E, int NT, int XR, int SH, int LDS>
struct RowStream {
  static constexpr int MT = XR < 16 ? 1 : XR / 16;
  static constexpr int XD = XR / 8 / SH;   // token loads per stage and wave
  static constexpr int D = 2 * NT + XD;    // loads per stage and wave
  static constexpr int SLOT = SH * D * 1024;
  static constexpr int NS = LDS / SLOT < 8 ? LDS / SLOT : 8;
  static_assert(NS >= 2 && XD >= 1 && (NS - 1) * D <= 63, "ring");
  i32x4_t rw[NT], rx;
  uint32_t w_off[2], x_off[XD];
  int kb, share, w_at;  // share: the wave's part of the token rows; w_at: its weights in a slot
  bool once;            // no line of the weights is read twice

  static __host__ __device__ __forceinline__ int stages(int K) { return (K * E::kBytes + 127) >> 7; }
  // the token row (0 .. XR - 1) whose chunk this lane fetches in load j
  __device__ __forceinline__ int x_row(int j, int lane) const { return 8 * (share * XD + j) + (lane >> 3); }

  // what does not change over a launch
  __device__ __forceinline__ void init(const Args& g, const char* xb, uint32_t x_bytes, int wave, int lane) {
    share = SH > 1 ? wave : 0;
    w_at = XR * 128 + share * NT * 2048;
    kb = g.K * E::kBytes;
    once = g.once != 0;
    rx = scalar_rsrc(rsrc_words(xb, x_bytes));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 8 * j + (lane >> 3);
      w_off[j] = (uint32_t)r * (uint32_t)kb + chunk(r, lane);
    }
  }
  // the byte of a stage's 128 that this lane fetches of row r
  static __device__ __forceinline__ uint32_t chunk(int r, int lane) { return ((lane & 7) ^ kc_swz(r)) << 4; }
  // load j's token row starts at byte `row` of the tokens (kOOB: there is none)
  __device__ __forceinline__ void token_row(int j, uint32_t row, int lane) {
    x_off[j] = row == kOOB ? kOOB : row + chunk(x_row(j, lane), lane);
  }
  // block n: rows row0 .. row0 + 15 of expert e's weight; rows past N read as zeros
  __device__ __forceinline__ void weight(int n, const Weight& wt, int e, int row0, int N) {
    const int rows = max(0, min(16, N - row0));
    rw[n] = scalar_rsrc(rsrc_words(wt.w + (int64_t)e * wt.expert + (int64_t)row0 * kb, (int64_t)rows * kb));
  }
  // Loads stage s into the slot; not live: zeros. K advances through the scalar
  // offset, which the range check leaves out, so the lanes' offsets change only
  // in a partial last stage, where those past K go out of range.
  __device__ __forceinline__ void issue(uint32_t slot, int s, bool live, int lane) const {
    const uint32_t at = (uint32_t)s * 128u;
    if (live && kb - (int)at >= 128) {
      if (once) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) dma16_once(slot + w_at + n * 2048 + j * 1024, rw[n], w_off[j], at);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) dma16(slot + w_at + n * 2048 + j * 1024, rw[n], w_off[j], at);
      }
#pragma unroll
      for (int j = 0; j < XD; ++j) dma16(slot + (share * XD + j) * 1024, rx, x_off[j], at);
      return;
    }
    const int left = live ? kb - (int)at : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        dma16(slot + w_at + n * 2048 + j * 1024, rw[n], (int)chunk(8 * j + (lane >> 3), lane) < left ? w_off[j] : kOOB, at);
#pragma unroll
    for (int j = 0; j < XD; ++j)
      dma16(slot + (share * XD + j) * 1024, rx, (int)chunk(x_row(j, lane), lane) < left ? x_off[j] : kOOB, at);
  }
  struct Nothing {
    __device__ __forceinline__ void token(int, u32x4_t) {}
    __device__ __forceinline__ void weight(int, u32x4_t) {}
  };
  __device__ __forceinline__ void compute(const char* slot, f32x4_t (&acc)[NT][MT], int lane) const {
    compute(slot, acc, lane, Nothing{});
  }
  // `see` is shown every operand on the way
  template <class See>
  __device__ __forceinline__ void compute(const char* slot, f32x4_t (&acc)[NT][MT], int lane, See&& see) const {
    const int r = lane & 15, c = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = r * 128 + (((4 * h + c) ^ kc_swz(r)) << 4);
      const int ax = XR < 16 ? (r & 7) * 128 + (((4 * h + c) ^ kc_swz(r & 7)) << 4) : at;
      u32x4_t xv[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        xv[m] = *(const u32x4_t*)(slot + m * 2048 + ax);
        see.token(m, xv[m]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4_t wv = *(const u32x4_t*)(slot + w_at + n * 2048 + at);
        see.weight(n, wv);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = step_mfma<E>(xv[m], wv, acc[n][m]);
      }
    }
  }
};

// 4-bit codes; a stage is one record of 128 K. The products run on integers:
// the nibble q goes into the mantissa of 128 (bf16) or 64 (fp16), which makes
// the operand OFF + q exactly with one shift and one and-or per two values.
// Per group of g the fp32 sum of x (OFF + q) is corrected by (OFF + z) times
// the sum of x (one more MFMA against ones, shared by all weight blocks) and
// scaled, so a scale costs two operations per output and group and no weight
// is rounded. The offset costs accuracy of about OFF / 5 fp32 roundings of the
// group's sum, 2^-19 of it in bf16: far below the storage type's half step.
// Token rows are 256 B per stage; chunk c of row r at position c ^ (r & 15).
template <class E, int G, int NT, int XR, int SH, int LDS>
struct W4Stream {
  static constexpr int GP = 128 / G;  // groups per record
  static constexpr int MT = XR < 16 ? 1 : XR / 16;
  static constexpr int XD = XR / 4 / SH;
  static constexpr int D = 2 * NT + XD;
  static constexpr int WS = 1024 + 256;  // a record's place in a slot
  static constexpr int SLOT = SH * (NT * WS + XD * 1024);
  static constexpr int NS = LDS / SLOT < 8 ? LDS / SLOT : 8;
  static_assert(NS >= 2 && XD >= 1 && (NS - 1) * D <= 63, "ring");
  static constexpr float kOff = std::is_same<E, Bf16>::value ? 128.0f : 64.0f;
  i32x4_t rw[NT], rx;
  uint32_t x_off[XD], scale_off, mask, base;
  int kb, rec, zeros, share, w_at;

  static __host__ __device__ __forceinline__ int stages(int K) { return (K + 127) >> 7; }
  __device__ __forceinline__ int x_row(int j, int lane) const { return 4 * (share * XD + j) + (lane >> 4); }

  __device__ __forceinline__ void init(const Args& g, const char* xb, uint32_t x_bytes, int wave, int lane) {
    share = SH > 1 ? wave : 0;
    w_at = XR * 256 + share * NT * WS;
    kb = g.K * 2;
    zeros = g.zeros;
    rec = 1024 + 32 * GP + (zeros ? 32 : 0);
    scale_off = 1024 + lane * 4 < rec ? 1024 + lane * 4 : kOOB;
    constexpr bool kBf = std::is_same<E, Bf16>::value;
    asm("s_mov_b32 %0, %1" : "=s"(mask) : "i"(kBf ? 0x000f000f : 0x00f000f0));
    asm("v_mov_b32 %0, %1" : "=v"(base) : "i"(kBf ? 0x43004300 : 0x54005400));
    rx = scalar_rsrc(rsrc_words(xb, x_bytes));
  }
  __device__ __forceinline__ void weight(int n, const Weight& wt, int e, int row0, int N) {
    const int len = row0 < N ? stages(kb >> 1) * rec : 0;
    rw[n] = scalar_rsrc(rsrc_words(wt.w + (int64_t)e * wt.expert + (int64_t)(row0 >> 4) * len, len));
  }
  // the same block for the compiler's loads
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t records(const Weight& wt, int e, int row0, int N) const {
    const int len = row0 < N ? stages(kb >> 1) * rec : 0;
    return make_rsrc(wt.w + (int64_t)e * wt.expert + (int64_t)(row0 >> 4) * len, len);
  }
  static __device__ __forceinline__ uint32_t chunk(int r, int lane) { return ((lane & 15) ^ (r & 15)) << 4; }
  __device__ __forceinline__ void token_row(int j, uint32_t row, int lane) {
    x_off[j] = row == kOOB ? kOOB : row + chunk(x_row(j, lane), lane);
  }
  __device__ __forceinline__ void issue(uint32_t slot, int s, bool live, int lane) const {
    const uint32_t at = (uint32_t)s * (uint32_t)rec, atx = (uint32_t)s * 256u;
    if (live && kb - (int)atx >= 256) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        dma16(slot + w_at + n * WS, rw[n], lane * 16, at);
        dma4(slot + w_at + n * WS + 1024, rw[n], scale_off, at);
      }
#pragma unroll
      for (int j = 0; j < XD; ++j) dma16(slot + (share * XD + j) * 1024, rx, x_off[j], atx);
      return;
    }
    const int left = live ? kb - (int)atx : 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      dma16(slot + w_at + n * WS, rw[n], live ? lane * 16 : kOOB, at);
      dma4(slot + w_at + n * WS + 1024, rw[n], live ? scale_off : kOOB, at);
    }
#pragma unroll
    for (int j = 0; j < XD; ++j)
      dma16(slot + (share * XD + j) * 1024, rx, (int)chunk(x_row(j, lane), lane) < left ? x_off[j] : kOOB, atx);
  }
  // Eight codes of one dword as the MFMA operand OFF + q: 128 + q in bf16 (mantissa
  // step 1), 64 + q in fp16 (step 1/16). mask and base come from init, where the
  // compiler cannot see their values: it would take an and and an or with
  // literals for what v_and_or_b32 does from registers. (The instruction itself
  // must stay the compiler's: a matrix instruction that reads a vector
  // instruction's result needs wait states, which it does not put after assembly.)
  __device__ __forceinline__ u32x4_t widen(uint32_t v) const {
    if constexpr (std::is_same<E, Bf16>::value)
      return u32x4_t{(v & mask) | base, ((v >> 4) & mask) | base, ((v >> 8) & mask) | base, ((v >> 12) & mask) | base};
    else
      return u32x4_t{((v << 4) & mask) | base, (v & mask) | base, ((v >> 4) & mask) | base, ((v >> 8) & mask) | base};
  }
  static __device__ __forceinline__ u32x4_t ones() {
    constexpr uint32_t o = std::is_same<E, Bf16>::value ? 0x3f803f80u : 0x3c003c00u;
    return u32x4_t{o, o, o, o};
  }
  // fp16 with two or more blocks of token rows: OFF + z is taken off the codes
  // (exactly, one packed addition per two) rather than off the sums, which
  // saves the products with ones: T = 33, N = 8208, K = 6144 31.0 -> 26.8 us,
  // T = 17 22.3 -> 21.2. There is no such addition for bf16.
  static constexpr bool kExact = std::is_same<E, Fp16>::value && MT > 1;
  static __device__ __forceinline__ u32x4_t less(u32x4_t v, float off) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const h2 o = {(_Float16)off, (_Float16)off};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = v[i];  // a copy: a bit cast of a vector's element reads element 0
      const h2 d = __builtin_bit_cast(h2, b) - o;
      v[i] = __builtin_bit_cast(uint32_t, d);
    }
    return v;
  }
  // Where the offset cannot be taken off a sum: x (OFF + q) and (OFF + z) x are
  // infinities of one sign where x is one (their difference NaN), and large finite x
  // (bf16, from about 1e34 on) overflow in both. Either leaves a sum that is not finite,
  // and those are formed again from x and s (q - z), in fp64, for one token row at a
  // time: lane l takes row l % 16 of the weights and the K that its codes have. Other
  // rows keep their values. Stages [s0, s1); block(n): the record descriptor of weight
  // block n; row(i): where the tokens' buffer has operand row i, or kOOB. Costs
  // nothing but the test where every sum is finite, and a pass over the
  // codes for each row and block where one is not.
  template <class Block, class Row>
  __device__ __forceinline__ void settle(f32x4_t (&acc)[NT][MT], int s0, int s1, int lane, Block&& block, Row&& row) const {
    if constexpr (kExact) return;
    f32x4_t all{};  // finite only if every sum is
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) all += acc[n][m];
    const bool bad = !(fabsf((all[0] + all[1]) + (all[2] + all[3])) < __builtin_inff());
    if (__builtin_expect(!__any(bad), 1)) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const __amdgpu_buffer_rsrc_t w = block(n);
#pragma unroll 1
      for (int at = 0; at < 4 * MT; ++at) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i)
          if (at == i) v = acc[n][i / 4][i % 4];
        for (uint64_t left = __ballot(!(fabsf(v) < __builtin_inff())); left;) {
          const int c = (__ffsll((unsigned long long)left) - 1) >> 4;  // operand row i is on lanes 16 c .. 16 c + 15
          const int i = 16 * (at >> 2) + 4 * c + (at & 3);
          double sum = again(w, row(i), s0, s1, lane);
          sum += __shfl_xor(sum, 16);
          sum += __shfl_xor(sum, 32);
          if ((lane >> 4) == c && !(fabsf(v) < __builtin_inff())) v = (float)sum;
          left &= ~(0xffffull << (16 * c));
        }
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i)
          if (at == i) acc[n][i / 4][i % 4] = v;
      }
    }
  }
  // The lane's part of one token row's product with weight row l % 16.
  __device__ __forceinline__ double again(__amdgpu_buffer_rsrc_t w, uint32_t row, int s0, int s1, int lane) const {
    const int r = lane & 15, c = lane >> 4;
    // rx's base and size, for the compiler's loads
    const __amdgpu_buffer_rsrc_t x = make_rsrc32((const void*)((uint64_t)(uint32_t)rx[0] | (uint64_t)(uint32_t)rx[1] << 32), rx[2]);
    typedef typename E::elem vec8 __attribute__((ext_vector_type(8)));
    double sum = 0.0;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const uint32_t at = (uint32_t)s * (uint32_t)rec;
      const u32x4_t code = load16(w, at + lane * 16);
      const uint32_t zs =
          zeros ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(w, at + 1024 + 32 * GP + r * 2, 0, 0) : 0x8888u;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int k = s * 128 + 32 * d + 8 * c;  // of the row; K is a multiple of 32
        if (2 * k >= kb || row == kOOB) continue;
        const int q = d * GP / 4;
        const uint16_t sb = __builtin_amdgcn_raw_buffer_load_b16(w, at + 1024 + (r * GP + q) * 2, 0, 0);
        const float scale = E::to_f32(__builtin_bit_cast(typename E::elem, sb)), z = (float)((zs >> (4 * q)) & 15u);
        const vec8 xv = __builtin_bit_cast(vec8, load16(x, row + 2 * (uint32_t)k));
        const uint32_t v = code[d];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          sum = fma((double)E::to_f32(xv[2 * p]), (double)(scale * ((float)((v >> (4 * p)) & 15u) - z)), sum);
          sum = fma((double)E::to_f32(xv[2 * p + 1]), (double)(scale * ((float)((v >> (16 + 4 * p)) & 15u) - z)), sum);
        }
      }
    }
    return sum;
  }
  __device__ __forceinline__ void compute(const char* slot, f32x4_t (&acc)[NT][MT], int lane) const {
    const int r = lane & 15, c = lane >> 4, rr = XR < 16 ? r & (XR - 1) : r;
    u32x4_t code[NT];
    typename E::elem sc[NT][GP];
    uint32_t z[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      code[n] = *(const u32x4_t*)(slot + w_at + n * WS + lane * 16);
      const typename E::elem* sp = (const typename E::elem*)(slot + w_at + n * WS + 1024) + r * GP;
#pragma unroll
      for (int q = 0; q < GP; ++q) sc[n][q] = sp[q];
      z[n] = zeros ? *(const uint16_t*)(slot + w_at + n * WS + 1024 + 32 * GP + r * 2) : 0x8888u;
    }
#pragma unroll
    for (int q = 0; q < GP; ++q) {
      f32x4_t part[NT][MT] = {}, xs[MT] = {};
#pragma unroll
      for (int i = 4 / GP * q; i < 4 / GP * (q + 1); ++i) {
        u32x4_t xv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          xv[m] = *(const u32x4_t*)(slot + (16 * m + rr) * 256 + (((4 * i + c) ^ rr) << 4));
          if constexpr (!kExact) xs[m] = step_mfma<E>(xv[m], ones(), xs[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u32x4_t w = widen(code[n][i]);
          if constexpr (kExact) w = less(w, kOff + (float)((z[n] >> (4 * q)) & 15u));
#pragma unroll
          for (int m = 0; m < MT; ++m) part[n][m] = step_mfma<E>(xv[m], w, part[n][m]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float s = E::to_f32(sc[n][q]);
        const float off = kOff + (float)((z[n] >> (4 * q)) & 15u);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[n][m][j] = fmaf(s, kExact ? part[n][m][j] : fmaf(-off, xs[m][j], part[n][m][j]), acc[n][m][j]);
      }
    }
  }
};

// FMT 0: rows; 32, 64, 128: 4 bits with groups of that size
template <class E, int FMT, int NT, int XR, int SH, int LDS>
struct StreamOf {
  using type = W4Stream<E, FMT, NT, XR, SH, LDS>;
};
template <class E, int NT, int XR, int SH, int LDS>
struct StreamOf<E, 0, NT, XR, SH, LDS> {
  using type = RowStream<E, NT, XR, SH, LDS>;
};

// A ring: step() = wait for the oldest stage, multiply it, and fetch the stage
// that `issue` (a callable: LDS slot address) says is next. In a shared ring the
// barrier that publishes a stage also says that the one before it has been
// read, so that one's slot is refilled, and NS - 1 stages are in flight.
template <class S, int SH>
struct Ring {
  char* lds;
  uint32_t addr;
  int slot;
  template <class Issue>
  __device__ __forceinline__ void start(char* p, Issue&& issue) {
    lds = p;
    addr = lds_addr(p);
    slot = 0;
#pragma unroll 1
    for (int i = 0; i < (SH > 1 ? S::NS - 1 : S::NS); ++i) issue(addr + i * S::SLOT);
  }
  template <int NT, class Issue, class... See>
  __device__ __forceinline__ void step(const S& st, f32x4_t (&acc)[NT][S::MT], int lane, Issue&& issue, See&&... see) {
    if constexpr (SH > 1) {
      ring::wait_vmcnt<(S::NS - 2) * S::D>();
      ring::lds_barrier();
      issue(addr + (slot ? slot - 1 : S::NS - 1) * S::SLOT);
      st.compute(lds + slot * S::SLOT, acc, lane, see...);
    } else {
      ring::wait_vmcnt<(S::NS - 1) * S::D>();
      st.compute(lds + slot * S::SLOT, acc, lane, see...);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read
      issue(addr + slot * S::SLOT);
    }
    slot = slot + 1 == S::NS ? 0 : slot + 1;
  }
};

// ---- a chunk's choices --------------------------------------------------------
// ids of the chunk's pairs, and which experts occur.
struct Choices {
  int16_t id[kMaxPairs];              // -1: chooses nothing
  unsigned seen[kMaxExperts / 32];    // bit per expert
  int upto[kMaxExperts / 32];         // experts that occur up to and with this word
  // the n-th expert that occurs (n < upto's last)
  __device__ __forceinline__ int expert(int n, int lane) const {
    const int u = lane < kMaxExperts / 32 ? upto[lane] : 0x7fffffff;
    const int word = __ffsll((unsigned long long)__ballot(u > n)) - 1;
    unsigned v = __builtin_amdgcn_readfirstlane(seen[word]);
    for (int before = __builtin_amdgcn_readlane(u, word) - __popc(v); before < n; ++before) v &= v - 1;
    return word * 32 + __ffs((int)v) - 1;
  }
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
    int n = lane < kMaxExperts / 32 ? __popc(c.seen[lane]) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up(n, d);
      if (lane >= d) n += o;
    }
    if (lane < kMaxExperts / 32) c.upto[lane] = n;
  }
  __syncthreads();
}

// The pairs that chose one expert, as one wave holds them: lane i has the i-th
// (its index in the chunk), n of them.
struct Picked {
  int pair, n;
};

// One wave: the pairs that chose e, ranks [64 pass, 64 pass + 64); total: how
// many chose e in all. list: 64 entries of the wave's own.
__device__ __forceinline__ Picked list_pairs(const Choices& c, int P, int e, int pass, int16_t* list, int lane,
                                             int& total) {
  int n = 0;
  for (int r = 0; r < P; r += 64) {
    const bool hit = r + lane < P && c.id[r + lane] == e;
    const uint64_t m = __ballot(hit);
    const int at = n + __popcll(m & ((1ull << lane) - 1)) - 64 * pass;
    if (hit && at >= 0 && at < 64) list[at] = (int16_t)(r + lane);
    n += __popcll(m);
  }
  __builtin_amdgcn_wave_barrier();
  total = n;
  const int got = min(64, n - 64 * pass);
  return {lane < got ? (int)list[lane] : 0, got};
}
// The same from a mask of at most 64 pairs, in registers.
__device__ __forceinline__ Picked mask_pairs(uint64_t m, int lane) {
  const bool in = (m >> lane) & 1;
  const int rank = __popcll(m & ((1ull << lane) - 1));
  // lanes in the mask send their index to lane `rank`, the others to lane 63,
  // which then only matters when the mask is full and nobody else sends
  const int v = __builtin_amdgcn_ds_permute((in ? rank : 63) * 4, lane);
  return {v, (int)__popcll(m)};
}

// Walks the experts that occur in a chunk, and for each the passes of at most
// XR of its pairs. Dense: one expert, all tokens.
struct Walk {
  const Args* g;
  const Choices* ch;  // more than 64 pairs
  int16_t* list;
  int P, id;          // id: lane's pair's expert (at most 64 pairs)
  uint64_t left;
  int hits, i, e, first, total;
  Picked p;           // pairs [first, first + 64) of the expert's list

  // All threads (a barrier in the last case). Stands before the first expert.
  __device__ __forceinline__ void open(const Args& a, Choices& c, int16_t* scratch, int t0, int tc, int lane) {
    g = &a;
    ch = &c;
    list = scratch;
    P = tc * a.k;
    i = -1;
    first = total = 0;
    left = 0;
    if (!a.ids) {
      hits = 1;
    } else if (P <= 64) {
      id = lane < P ? a.ids[(int64_t)t0 * a.k + lane] : -1;
      left = __ballot((unsigned)id < (unsigned)a.E);
      hits = 0;
      for (uint64_t l = left; l; ++hits)
        l &= ~__ballot(id == __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)l) - 1));
    } else {
      read_choices(c, a, t0, tc);
      hits = __builtin_amdgcn_readfirstlane(c.upto[kMaxExperts / 32 - 1]);
    }
  }
  // The n-th expert (n >= i), first pass.
  __device__ __forceinline__ void expert(int n, int lane) {
    first = 0;
    if (!g->ids) {
      e = 0;
      p = {lane, P};
      total = P;
    } else if (P <= 64) {
      for (; i < n; ++i) {
        e = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
        left &= ~__ballot(id == e);
      }
      p = mask_pairs(__ballot(id == e), lane);
      total = p.n;
    } else {
      e = ch->expert(n, lane);
      p = list_pairs(*ch, P, e, 0, list, lane, total);
    }
    i = n;
  }
  // Moves to the expert's next pass, if there is one.
  __device__ __forceinline__ bool next_pass(int XR, int lane) {
    if (first + XR >= total) return false;
    first += XR;
    if ((first & 63) == 0) p = list_pairs(*ch, P, e, first >> 6, list, lane, total);
    return true;
  }
  __device__ __forceinline__ int rows(int XR) const { return min(XR, total - first); }
  // lane i: the pass's i-th pair
  __device__ __forceinline__ int pair(int i) const { return __shfl(p.pair, ((first & 63) + i) & 63); }
};

// Whether A is held in two parts (few_down): at 8 token rows per stage, in 4 bits 4, where
// the second part takes operand rows that are free. More rows would double the
// products and the LDS reads of tokens, so there A is rounded once, as the
// framework's other paths do, and y's error in 64 bits is 1.4 times that of fp32
// sums alone (fp16 T = 37 2.9e-4 of the norm against 2.1e-4, bf16 T = 64 2.35e-3
// against 1.66e-3) instead of 1.0.
static __host__ __device__ constexpr bool halves(int rows, size_t e) { return rows <= 8 && e == 2; }

// The largest finite value of a 16-bit type (A's two parts; fp32 has one).
template <class E>
__device__ __forceinline__ constexpr float largest() {
  return std::is_same<E, Bf16>::value ? 0x1.fep127f : 65504.f;
}

// ---- gate/up ------------------------------------------------------------------
// An item is a tile of hidden columns of one pass; the workgroup takes a run of
// items. SH = 1: 16 HB columns, the waves take equal parts of K and their sums
// meet in LDS; SH = NW: 16 HB columns per wave, all of K. The rings run on
// from item to item: while one is finished, the loads of the next are in flight.
// Bound by HBM where there is enough to read: E = 64, T = 16, k = 8, D = 2048,
// H = 1408, bf16: 93 us for the 55 or so experts that occur, 651 MB, 7.0 TB/s; the
// 64 rows of E = 8, T = 64, D = 4096, H = 11008 266 us, 5.4 TB/s, LDS reads of the
// token rows being on the way. One token of E = 8, D = 1024, H = 2816 (23 MB) is
// 9 us: start, a first load's latency and the reduction. In 4 bits (E = 64, T = 8)
// 31 us, 4.1 TB/s, where widening the codes is half of the wave's instructions.
// RING: bytes of LDS for the workgroup's rings. PLAIN: y = x W^T instead, one
// weight block per 16 columns and no SwiGLU (dense, w0 and out = y).
template <class E, int FMT, int HB, int XR, int NW, int SH, int RING, bool PLAIN>
__global__ void __launch_bounds__(NW * 64, (SH == 1 && FMT != 0 && XR < 16 ? 3 : 2)) few_gateup(const Args g) {
  constexpr int NT = PLAIN ? HB : 2 * HB, COLS = 16 * HB * SH;
  constexpr bool HALVES = !PLAIN && halves(XR, E::kBytes);
  using S = typename StreamOf<E, FMT, NT, XR, SH, (SH > 1 ? RING : RING / NW)>::type;
  constexpr int MT = S::MT;
  __shared__ __attribute__((aligned(1024))) char lds[RING];
  __shared__ __attribute__((aligned(16))) float red[SH > 1 ? 4 : NW * NT * MT * 256];
  __shared__ Choices ch;
  __shared__ int16_t list[NW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.z * kChunk, tc = min(kChunk, g.T - t0);
  if (blockIdx.x == 0 && blockIdx.z == 0)
    for (int i = threadIdx.x; i < g.n_ctr; i += NW * 64) g.ctr[i] = 0u;
  Walk use;  // the item being multiplied
  use.open(g, ch, list[wave], t0, tc, lane);
  const int tiles = (g.N + COLS - 1) / COLS, items = use.hits * tiles;
  // (divisions are done by vector instructions: back to scalar registers)
  int left = __builtin_amdgcn_readfirstlane((int)((int64_t)items * blockIdx.x / gridDim.x));
  const int last = __builtin_amdgcn_readfirstlane((int)((int64_t)items * (blockIdx.x + 1) / gridDim.x));
  if (left >= last) return;
  int nth = __builtin_amdgcn_readfirstlane(left / tiles), tile = left - nth * tiles;  // the item: expert, tile
  left = last - left;
  Walk get = use;  // the item being loaded
  S st;
  st.init(g, g.x + (int64_t)t0 * g.K * E::kBytes, (uint32_t)(tc * g.K) * E::kBytes, wave, lane);
  const int stages = S::stages(g.K), per = SH > 1 ? stages : (stages + NW - 1) / NW;
  const int s0 = SH > 1 ? 0 : wave * per, s1 = min(stages, s0 + per);
  const int wcol = SH > 1 ? 16 * HB * wave : 0;  // the wave's first column of a tile

  // loading side: the next stage of the current item, then the next item
  int get_nth = nth, get_tile = tile, get_left = left, get_s = s0;
  auto set_rows = [&] {
    const int n = get.rows(XR);
#pragma unroll
    for (int j = 0; j < S::XD; ++j) {
      const int i = st.x_row(j, lane), pair = get.pair(i);
      st.token_row(j, i < n ? ((pair * g.kinv) >> 16) * (uint32_t)(g.K * E::kBytes) : kOOB, lane);
    }
  };
  auto set_weights = [&] {
    const int row0 = get_tile * COLS + wcol;
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      if constexpr (PLAIN) {
        st.weight(b, g.w0, get.e, row0 + 16 * b, g.N);
      } else {
        st.weight(2 * b, g.w0, get.e, row0 + 16 * b, g.N);
        st.weight(2 * b + 1, g.w1, get.e, row0 + 16 * b, g.N);
      }
    }
  };
  auto issue = [&](uint32_t slot) {
    st.issue(slot, get_s, get_left > 0 && get_s < s1, lane);
    if (++get_s < s0 + per || get_left == 0) return;
    get_s = s0;
    if (get.next_pass(XR, lane)) {
      set_rows();
      return;
    }
    if (--get_left == 0) return;
    const bool turn = ++get_tile == tiles;
    if (turn) {
      get_tile = 0;
      ++get_nth;
    }
    if (get.first || turn) {
      get.expert(get_nth, lane);
      set_rows();
    }
    set_weights();
  };
  get.expert(nth, lane);
  set_rows();
  set_weights();
  Ring<S, SH> r;
  r.start(lds + (SH > 1 ? 0 : wave * (RING / NW)), issue);

  // g and u stay in fp32; A is rounded to the storage type the down
  // projection's matrix instructions take. That one rounding would add as much
  // error to y as y's own, so where the token operand has room for a second set
  // of rows (halves) what it left goes into those.
  auto store = [&](int pair, int h, float gate, float up) {
    const float a = PLAIN ? gate : gate * sigmoid_f32<E>(gate) * up;
    const int64_t p = (int64_t)t0 * g.k + pair;
    typename E::elem* out = (typename E::elem*)g.out + (HALVES ? 2 * p : p) * g.N + h;
    if constexpr (!HALVES) {
      out[0] = E::from_f32(a);
      return;
    }
    // Past the type's range (fp16: 65504) the first part is its largest value, and
    // the second holds the rest up to as much again; an infinity leaves nothing
    // (Inf - Inf would be NaN).
    const float size = fabsf(a);
    const bool inf = size == __builtin_inff();
    const typename E::elem hi = E::from_f32(size > largest<E>() && !inf ? copysignf(largest<E>(), a) : a);
    out[0] = hi;
    out[g.N] = E::from_f32(inf ? 0.f : a - E::to_f32(hi));
  };
  use.expert(nth, lane);
  while (true) {
    f32x4_t acc[NT][MT] = {};
#pragma unroll 1
    for (int s = 0; s < per; ++s) r.step(st, acc, lane, issue);
    const int n = use.rows(XR), row0 = tile * COLS + wcol;
    if constexpr (FMT != 0)
      st.settle(
          acc, s0, s1, lane,
          [&](int b) {
            return st.records(PLAIN || b % 2 == 0 ? g.w0 : g.w1, use.e, row0 + 16 * (PLAIN ? b : b / 2), g.N);
          },
          [&](int i) { return i < n ? ((use.pair(i) * g.kinv) >> 16) * (uint32_t)(g.K * E::kBytes) : kOOB; });
    if constexpr (SH > 1) {
      // the wave has all of K: lane -> hidden column l % 16, token rows 4 (l / 16) + j
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 16 * m + 4 * (lane >> 4) + j, pair = use.pair(i);
#pragma unroll
          for (int b = 0; b < HB; ++b) {
            const int h = row0 + 16 * b + (lane & 15);
            if (i < n && h < g.N) store(pair, h, acc[PLAIN ? b : 2 * b][m][j], acc[PLAIN ? b : 2 * b + 1][m][j]);
          }
        }
    } else {
      ring::lds_barrier();  // the last item's sums have been read
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) *(f32x4_t*)(red + (((wave * NT + n) * MT + m) * 64 + lane) * 4) = acc[n][m];
      ring::lds_barrier();
      // thread -> (token row of the pass, hidden column); the waves' sums in order
#pragma unroll 1
      for (int i0 = 0; i0 < HB * MT * 256; i0 += NW * 64) {
        const int i = i0 + threadIdx.x, b = i / (MT * 256);
        if (HB * MT * 256 % (NW * 64) != 0 && b >= HB) break;  // whole waves
        const int col = i & 15, row = (i >> 4) % (16 * MT);
        const int at = ((row >> 4) * 64 + ((row & 15) >> 2) * 16 + col) * 4 + (row & 3);
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
          gate += red[(v * NT + (PLAIN ? b : 2 * b)) * MT * 256 + at];
          if constexpr (!PLAIN) up += red[(v * NT + 2 * b + 1) * MT * 256 + at];
        }
        const int pair = use.pair(row), h = row0 + 16 * b + col;
        if (row < n && h < g.N) store(pair, h, gate, up);
      }
    }
    if (use.next_pass(XR, lane)) continue;
    if (--left == 0) break;
    const bool turn = ++tile == tiles;
    if (turn) {
      tile = 0;
      ++nth;
    }
    if (use.first || turn) use.expert(nth, lane);
  }
  ring::wait_vmcnt<0>();  // no load may land in LDS after the workgroup's end
}

// ---- down -----------------------------------------------------------------------
// The K axis of an output tile is the list of (expert that occurs, K stage);
// equal runs of it go to the splits x NW / SH groups of SH waves (16 NT columns
// for each wave of a group). At an expert's end the block of sums is weighted
// and added to the wave's own [token][column] tile in LDS. TC: tokens that tile
// has room for. Groups of a shared ring meet at barriers, so they take equally
// many steps; more than one of them only for a dense product.
// HALVES: A comes as two values (see few_gateup), in rows 0 .. XR - 1 and
// XR .. 2 XR - 1 of the token operand, which repeats nothing then: no more
// matrix instructions than with one. Measured where few_gateup was: 51 us for
// 326 MB (6.3 TB/s), 149 us (4.8 TB/s), 8.7 us for 11.5 MB, and 23 us in 4 bits.
// W4, T = 33, N = 11008, K = 4096, g = 64, fp16: 19.0 us, 25 MB: bound by the waves'
// instructions (codes to widen, LDS reads of the tokens, a scale per group and
// output) on the 172 of 256 CUs that have a tile of 64 columns.
template <class E, int FMT, int NT, int XR, int NW, int SH, int RING, int TC, bool HALVES>
__global__ void __launch_bounds__(NW * 64, (SH == 1 && FMT != 0 && XR < 16 ? 3 : 2)) few_down(const Args g) {
  using S = typename StreamOf<E, FMT, NT, (HALVES ? 2 * XR : XR), SH, RING / (NW / SH)>::type;
  static_assert(!HALVES || 2 * XR <= 16, "one block of token rows");
  constexpr int PARTS = HALVES ? 2 : 1;
  constexpr int MT = S::MT, C = 16 * NT, KG = NW / SH;  // KG: groups
  __shared__ __attribute__((aligned(1024))) char lds[RING];
  __shared__ __attribute__((aligned(16))) float ysum[NW][TC * C];
  __shared__ Choices ch;
  __shared__ int16_t list[NW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.z * kChunk, tc = min(kChunk, g.T - t0);
  const int wg0 = blockIdx.x * C * SH, col0 = wg0 + wave % SH * C;  // the workgroup's, the wave's columns
  const int group = wave / SH;
  const bool routed = g.ids != nullptr;
  float* y = ysum[wave];
  for (int i = lane; i < tc * C; i += 64) y[i] = 0.f;
  Walk use;
  use.open(g, ch, list[wave], t0, tc, lane);
  const int stages = S::stages(g.K), parts = g.splits * KG, part = blockIdx.y * KG + group;
  // (divisions are done by vector instructions: back to scalar registers)
  int at = __builtin_amdgcn_readfirstlane((int)((int64_t)use.hits * stages * part / parts));
  const int end = __builtin_amdgcn_readfirstlane((int)((int64_t)use.hits * stages * (part + 1) / parts));
  const int nth = __builtin_amdgcn_readfirstlane(at / stages);
  // groups that meet at barriers enter together, one without a stage too
  if (KG > 1 && SH > 1 ? use.hits > 0 : at < end) {
    Walk get = use;
    S st;
    const uint32_t row_bytes = PARTS * (uint32_t)g.K * E::kBytes;  // of a pair
    st.init(g, g.x + (int64_t)t0 * g.k * row_bytes, (uint32_t)(tc * g.k) * row_bytes, wave % SH, lane);
    auto set_rows = [&] {
      const int n = get.rows(XR);
#pragma unroll
      for (int j = 0; j < S::XD; ++j) {
        const int i = st.x_row(j, lane) % XR, half = st.x_row(j, lane) / XR, pair = get.pair(i);
        st.token_row(j, i < n ? (uint32_t)pair * row_bytes + (uint32_t)(half * g.K) * E::kBytes : kOOB, lane);
      }
    };
    // the run's stages of the n-th expert
    const int run0 = at;
    auto begin_of = [&](int n) { return max(0, run0 - n * stages); };
    auto end_of = [&](int n) { return min(stages, end - n * stages); };
    int get_s = 0, get_end = 0;
    bool more = at < end;
    auto open_expert = [&](int n) {
      get.expert(n, lane);
      set_rows();
#pragma unroll
      for (int b = 0; b < NT; ++b) st.weight(b, g.w0, get.e, col0 + 16 * b, g.N);
      get_s = begin_of(n);
      get_end = end_of(n);
    };
    auto issue = [&](uint32_t slot) {
      st.issue(slot, get_s, more, lane);
      if (!more || ++get_s < get_end) return;
      if (get.next_pass(XR, lane)) {
        set_rows();
        get_s = begin_of(get.i);
        return;
      }
      more = (get.i + 1) * stages < end;
      if (more) open_expert(get.i + 1);
    };
    open_expert(nth);
    Ring<S, SH> r;
    r.start(lds + group * (RING / KG), issue);
    for (int n = nth; n * stages < end; ++n) {
      use.expert(n, lane);
      const int count = end_of(n) - begin_of(n);
      do {
        const int rows = use.rows(XR), mine = use.pair(lane);
        const float wt = routed && lane < rows ? g.wts[(int64_t)t0 * g.k + mine] : 1.0f;
        f32x4_t acc[NT][MT] = {};
#pragma unroll 1
        for (int s = 0; s < count; ++s) r.step(st, acc, lane, issue);
        if constexpr (FMT != 0)
          st.settle(
              acc, begin_of(n), end_of(n), lane,
              [&](int b) { return st.records(g.w0, use.e, col0 + 16 * b, g.N); },
              [&](int i) {
                return i < PARTS * XR && i % XR < rows
                           ? (uint32_t)use.pair(i % XR) * row_bytes + (uint32_t)(i / XR * g.K) * E::kBytes
                           : kOOB;
              });
        // lane i: the i-th pair's token; pairs come in order, so a token that is
        // listed twice for one expert is the next one's too
        const int tok = (int)((uint32_t)mine * g.kinv >> 16), next = __shfl(tok, (lane + 1) & 63);
        if (!__any(lane + 1 < rows && tok == next)) {
          // all rows side by side (T = 64, N = 8944, K = 2176 in 4 bits: 16.5 us, one
          // row after another 24.1)
          float old[NT][MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = 16 * m + 4 * (lane >> 4) + j;
              const int at = __shfl(tok, row & 63) * C + (lane & 15);
#pragma unroll
              for (int b = 0; b < NT; ++b) old[b][m][j] = row < rows ? y[at + 16 * b] : 0.f;
            }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = 16 * m + 4 * (lane >> 4) + j;
              const int at = __shfl(tok, row & 63) * C + (lane & 15);
              const float f = __shfl(wt, row & 63);
#pragma unroll
              for (int b = 0; b < NT; ++b) {
                float v = acc[b][m][j];
                if constexpr (HALVES) v += __shfl_xor(v, 4 * XR);  // row + XR: what A's rounding left
                if (row < rows) y[at + 16 * b] = fmaf(f, v, old[b][m][j]);
              }
            }
          continue;
        }
        // one row at a time: the token's rows are added in order
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll 1
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = 16 * m + 4 * q + j, i = HALVES ? row % XR : row;
              if (i < rows && row < PARTS * XR) {
                const int pair = __builtin_amdgcn_readlane(mine, i);
                const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wt), i));
                if ((lane >> 4) == q) {
#pragma unroll
                  for (int b = 0; b < NT; ++b)
                    y[((pair * g.kinv) >> 16) * C + 16 * b + (lane & 15)] += f * acc[b][m][j];
                }
              }
            }
      } while (use.next_pass(XR, lane));
    }
    if constexpr (SH > 1 && KG > 1) {
      // one dead step for a group with a stage less than another
      f32x4_t none[NT][MT] = {};
      if (end - run0 < (use.hits * stages + parts - 1) / parts) r.step(st, none, lane, issue);
    }
    ring::wait_vmcnt<0>();  // no load may land in LDS after the rings' end
  }
  __syncthreads();
  // four columns of one token per thread; the waves' sums of a column in order
  constexpr int Q = C * SH / 4;  // such quads per token
  const bool direct = g.splits == 1;
  for (int i = threadIdx.x; i < tc * Q; i += NW * 64) {
    const int row = i / Q, q = i % Q;
    f32x4_t v{};
    if constexpr (SH > 1) {
#pragma unroll
      for (int w = 0; w < KG; ++w) v += *(const f32x4_t*)(ysum[w * SH + q / (C / 4)] + row * C + q % (C / 4) * 4);
    } else {
#pragma unroll
      for (int w = 0; w < NW; ++w) v += *(const f32x4_t*)(ysum[w] + i * 4);
    }
    const int t = t0 + row, n = wg0 + q * 4;
    if (n >= g.N) continue;  // N is a multiple of 8: all four columns or none
    if (direct) {
      typename E::vec4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = E::from_f32(v[j]);
      *(typename E::vec4*)((typename E::elem*)g.out + (int64_t)t * g.N + n) = o;
    } else {
      store_partial(g.partial + ((int64_t)blockIdx.y * g.T + t0) * g.N, tc, g.N, row, n, v);
    }
  }
  if (direct || !g.ctr) return;  // without counters another launch adds them (few_sum)
  // Arrival, as in stream_gemm: device-coherent partials, each wave waits for
  // its own, then one atomic add; the last workgroup adds the splits in order.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  int* arrived = (int*)lds;
  if (threadIdx.x == 0)
    *arrived = __hip_atomic_fetch_add(g.ctr + blockIdx.z * gridDim.x + blockIdx.x, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(g.splits - 1);
  __syncthreads();
  if (!*arrived) return;
  for (int i = threadIdx.x; i < tc * Q; i += NW * 64) {
    const int row = i / Q, n = wg0 + i % Q * 4;
    if (n >= g.N) continue;
    // eight at a time in flight; those past the splits read as zeros
    const __amdgpu_buffer_rsrc_t part =
        make_rsrc(g.partial + (int64_t)t0 * g.N, ((int64_t)(g.splits - 1) * g.T + tc) * g.N * 4);
    f32x4_t v{};
    for (int s0 = 0; s0 < g.splits; s0 += 8) {
      u32x4_t b[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        b[s] = __builtin_amdgcn_raw_buffer_load_b128(
            part, s0 + s < g.splits ? (uint32_t)(((s0 + s) * g.T + row) * g.N + n) * 4u : kOOB, 0, kCoherentPolicy);
#pragma unroll
      for (int s = 0; s < 8; ++s) v += __builtin_bit_cast(f32x4_t, b[s]);
    }
    typename E::vec4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = E::from_f32(v[j]);
    *(typename E::vec4*)((typename E::elem*)g.out + (int64_t)(t0 + row) * g.N + n) = o;
  }
}

// y = rnd(sum of the splits' partial sums), four values per thread.
template <class E>
__global__ void __launch_bounds__(256) few_sum(const float* partial, typename E::elem* y, int64_t quads, int splits) {
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
  typename E::vec4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = E::from_f32(v[j]);
  ((typename E::vec4*)y)[i] = o;
}

// ---- launches ---------------------------------------------------------------------
// Token rows per stage (8: as few as a load instruction covers, 8 or in 4 bits
// 4). Dense: what the tokens need. Routed: what an expert's share of a chunk's
// pairs mostly needs; a more crowded expert takes several passes over its
// weights. Where it pays to go up was measured with E = 16, D = 2048, H = 1408,
// k = 8 and E = 6, D = 3056, H = 1264, k = 3 (4 bits: D = 2688, H = 1024), by
// the average load of an expert:
//   16 rows against 64, 16 bits   load 10: 63.5/72.9, 53.9/64.6 us
//                                 load 12: 78.9/74.1, 58.6/68.4
//                                 load 16: 91.3/76.0, 69.3/71.2
//   fp32, bound by its products   load 10: 113/210, 82/139
//                                 load 24: 207/216, 136/149; load 32: 276/220, 164/153
//   4 bits, 16 rows against 32    load 12: 49.3/51.7, 39.6/46.2
//                                 load 16: 64.0/53.4, 47.9/48.2
//   32 against 64                 load 16: 53.4/63.2, 48.2/51.2
// Above 16 rows waves have to share them, and 8 waves cannot share the loads of
// 32 rows of 128 bytes.
struct Shape {
  int rows;  // token rows
  bool own;  // private rings, several workgroups of 4 waves per CU; else one of 8 waves
  int per;   // such workgroups per CU
};
static inline Shape shape_of(int64_t T, int64_t k, int64_t E, bool routed, bool w4, size_t e) {
  // load <= m E: m pairs per expert on average
  const int64_t few = w4 ? 4 : 8, load = routed ? (T < kChunk ? T : kChunk) * k : 0;
  int rows = 64;
  if (T <= few || (routed && 4 * load <= few * E)) rows = 8;
  else if (T <= 16 || (routed && load <= (e == 4 ? 24 : w4 ? 12 : 10) * E)) rows = 16;
  else if (w4 && (T <= 32 || (routed && load <= 20 * E))) rows = 32;
  return {rows, rows <= 16, rows > 16 ? 1 : w4 && rows == 8 ? 3 : 2};
}

// The down projection's workgroups: columns of a tile, waves, and workgroups per
// tile, so that all CUs pull weights. One workgroup of many waves per tile adds
// its sums in LDS; several leave partial sums and count arrivals, which costs
// about 3 us: only where there are too few tiles, or chunks too long for the waves'
// [token][column] tiles. Whole blocks in us with K split over workgroups of 4 waves, and
// unsplit with 16, 8 and 4 waves (rows: bf16, 2 of 8 experts, H = 5632, T = 12; 4 bits: the
// dense block, H = 5632, T = 1):
//   D =  1024,   64 tiles   rows 52/76/74/74       4 bits 13.1/12.5/11.5/12.1
//   D =  2048,  128 tiles   rows 82/95/92/93       4 bits 14.4/13.7/12.9/13.7
//   D =  2560,  160 tiles   rows 121/126/123/123   4 bits 17.6/14.5/13.5/14.3
//   D =  4096,  256 tiles   rows 155/155/153/154   4 bits 17.2/15.9/14.9/15.9
//   D =  6144,  384 tiles   rows 271/276/275/269   4 bits 20.5/23.6/19.5/19.0
//   D = 16384, 1024 tiles   rows 703/689/677/675   4 bits 42.3/51.4/42.2/41.6
// and with H = 11008, D = 4096: rows T = 16 201/217/211 unsplit, 4 bits 21.6/21.1/22.4. So 16
// waves for the fewest tiles, whose K is cut finest, and fewer from 384 and 1024 on.
// (In 4 bits below 160 tiles the split is 1 to 3 us behind; rows need it.)
struct DownShape {
  int cols, waves, splits;
};
static inline DownShape down_shape(const Shape& f, int64_t T, int64_t D) {
  const int cols = f.own ? 16 : 128, most = f.own ? 8 : 32;
  const int64_t tiles = (D + cols - 1) / cols * ((T + kChunk - 1) / kChunk);
  if (f.own && T <= 16 && tiles >= 160) return {cols, tiles < 384 ? 16 : tiles < 1024 ? 8 : 4, 1};
  const int64_t s = (256 * f.per + tiles - 1) / tiles;
  return {cols, f.own ? 4 : 8, (int)(s > most ? most : s)};
}
// Workspace of a block: the A plane, then where the down projection is split
// one counter per output tile and the partial sums, each 256-byte aligned.
struct BlockPlan {
  size_t ctr, partial, total;
  DownShape down;
  int n_ctr;
};
static inline BlockPlan block_plan(const Shape& f, int64_t T, int64_t D, int64_t H, int64_t k, size_t e) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  if (T == 0) return BlockPlan{};  // no tiles
  BlockPlan p;
  p.down = down_shape(f, T, D);
  p.n_ctr = p.down.splits > 1 ? (int)((D + p.down.cols - 1) / p.down.cols * ((T + kChunk - 1) / kChunk)) : 0;
  p.ctr = up((size_t)T * k * H * e * (halves(f.rows, e) ? 2 : 1));
  p.partial = p.ctr + up((size_t)p.n_ctr * 4);
  p.total = p.partial + (p.down.splits > 1 ? up((size_t)p.down.splits * T * D * 4) : 0);
  return p;
}

// A whole call; the host has checked it.
struct Call {
  const char* x;
  Weight wg, wu, wd;  // linear: wd only
  char* ws;           // workspace (block_plan)
  char* y;
  const int* ids;
  const float* wts;
  int64_t T, D, H;
  int k, E, zeros;
  hipStream_t stream;
};

// Workgroups with private rings that share a CU.
template <int FMT, int XR>
constexpr int groups_per_cu() { return FMT != 0 && XR < 16 ? 3 : 2; }

// TC: tokens a private down tile has room for, 16 or a whole chunk.
template <class E, int FMT, int HB, int XR, int NW, int SH, bool PLAIN>
static int launch_gateup(const Args& g, int slots, hipStream_t s) {
  StageScope scope(PLAIN ? STAGE_FEW_DOWN : STAGE_FEW_GATEUP, s);
  constexpr int PER = SH > 1 || NW > 4 || XR > 16 ? 1 : groups_per_cu<FMT, XR>();
  constexpr int RING = SH > 1 ? 147456 : NW > 4 ? 16384 * NW : XR > 16 ? (FMT ? 86016 : 98304) : PER == 2 ? 65536 : 32768;
  const int64_t items = (int64_t)slots * ((g.N + 16 * HB * SH - 1) / (16 * HB * SH)), fit = PER * dev_ncu();
  const dim3 grid((unsigned)(items < fit ? items : fit), 1, (g.T + kChunk - 1) / kChunk);
  hipLaunchKernelGGL((few_gateup<E, FMT, HB, XR, NW, SH, RING, PLAIN>), grid, dim3(NW * 64), 0, s, g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}
// NW: waves; SHARE: those that share the rows when there are more than 16.
template <class E, int FMT, int XR, int NW, int SHARE, int TC, bool HALVES>
static int launch_down(const Args& g, hipStream_t s) {
  StageScope scope(STAGE_FEW_DOWN, s);
  constexpr bool kOwn = XR <= 16;
  constexpr int SH = kOwn ? 1 : SHARE, PER = groups_per_cu<FMT, XR>();
  constexpr int RING = !kOwn     ? 122880
                       : NW > 4  ? (FMT != 0 && XR == 16 ? 16384 : 8192) * NW
                       : PER > 2 ? (TC > 16 ? 32768 : 40960)
                                 : (TC > 16 ? 57344 : 65536);
  const dim3 grid((g.N + 16 * SH - 1) / (16 * SH), g.splits, (g.T + kChunk - 1) / kChunk);
  hipLaunchKernelGGL((few_down<E, FMT, 1, XR, NW, SH, RING, TC, HALVES>), grid, dim3(NW * 64), 0, s, g);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

static inline Args args_of(const Call& c, const char* x, int64_t N, int64_t K, char* out) {
  return Args{x, c.wd, c.wd, out, c.ids, c.wts, (int)c.T, c.k, c.E, (int)N, (int)K, (65535u + c.k) / c.k,
              c.zeros, 0, 1, nullptr, nullptr, 0};
}
template <class E, int FMT, int XR, bool HALVES>
static int down_own(const Args& g, int waves, hipStream_t s) {
  if (g.T > 16) return launch_down<E, FMT, XR, 4, 1, kChunk, HALVES>(g, s);
  // 16 rows of 4 bits need rings too long for 16 waves
  constexpr int kMost = FMT != 0 && XR == 16 ? 8 : 16;
  if (waves == 16) return launch_down<E, FMT, XR, kMost, 1, 16, HALVES>(g, s);
  if (waves == 8) return launch_down<E, FMT, XR, 8, 1, 16, HALVES>(g, s);
  return launch_down<E, FMT, XR, 4, 1, 16, HALVES>(g, s);
}
template <class E, int FMT>
static int down_for(const Args& g, const Shape& f, int waves, hipStream_t s) {
  if (f.rows == 8) return down_own<E, FMT, FMT ? 4 : 8, halves(8, E::kBytes)>(g, waves, s);
  if (f.rows == 16) return down_own<E, FMT, 16, false>(g, waves, s);
  if constexpr (FMT != 0) {
    if (f.rows == 32) return launch_down<E, FMT, 32, 8, 8, kChunk, false>(g, s);
  }
  return launch_down<E, FMT, 64, 8, 8, kChunk, false>(g, s);
}
// Private rings: 4 waves, or 8 where each CU would run one workgroup at most and K
// is long (4-bit N = 4096: K = 11008 10.6 -> 9.5 us, K = 4096 5.4 -> 5.6 us).
template <class E, int FMT, int XR, bool PLAIN>
static int gateup_own(const Args& g, int slots, hipStream_t s) {
  const int64_t items = (int64_t)slots * ((g.N + 15) / 16) * ((g.T + kChunk - 1) / kChunk);
  const int stages = StreamOf<E, FMT, 1, 16, 1, 16384>::type::stages(g.K);
  if (items <= dev_ncu() && stages >= 48) return launch_gateup<E, FMT, 1, XR, 8, 1, PLAIN>(g, slots, s);
  return launch_gateup<E, FMT, 1, XR, 4, 1, PLAIN>(g, slots, s);
}
template <class E, int FMT>
static int gateup_for(const Args& g, const Shape& f, int slots, hipStream_t s) {
  if (f.rows == 8) return gateup_own<E, FMT, FMT ? 4 : 8, false>(g, slots, s);
  if (f.rows == 16) return gateup_own<E, FMT, 16, false>(g, slots, s);
  // With so few tiles of 128 columns that most CUs would idle, tiles of 16 whose
  // waves split K on private rings, each row loaded by one of them (4 bits: 32
  // rows at a time, more leave no room).
  const int64_t tiles = (int64_t)slots * ((g.N + 127) / 128) * ((g.T + kChunk - 1) / kChunk);
  if (8 * tiles < 3 * dev_ncu()) return launch_gateup<E, FMT, 1, FMT ? 32 : 64, 4, 1, false>(g, slots, s);
  if constexpr (FMT != 0) {
    if (f.rows == 32) return launch_gateup<E, FMT, 1, 32, 8, 8, false>(g, slots, s);
  }
  return launch_gateup<E, FMT, 1, 64, 8, 8, false>(g, slots, s);
}

// y = x W^T (dense). At most 16 rows: items of 16 columns, or 32 where those still
// give every workgroup one (K = 4096, g = 128, 16 columns/32 in us: N = 24576 T = 1
// 12.6/11.8, T = 16 17.5/16.6; N = 32000 15.9/16.0, 21.3/16.9; N = 65536 31.8/28.7,
// 51.1/40.5, 4.8 TB/s at T = 1; N = 128256 61.4/56.0, 101/80). More: tiles of 64 columns
// with two groups of 4 waves along K; where those are few, K is split over
// workgroups as well and a second launch adds the parts. A part has 6 records at
// least (us with none, 12, 6, 3 or 1; bf16, g = 64, T = 48: N = 1248, K = 9792 46.5, 16.9,
// 14.6, 14.9, 15.2; N = 4096, K = 4096 22.2, 16.6, 13.7, 13.8, 14.0; N = 2048, K = 1408 13.2,
// 13.2, 13.4, 11.2, 11.1; N = 256, K = 4096 22.0, 16.0, 13.6, 12.1, 10.4: the fewest columns
// would take shorter parts).
static inline int linear_splits(int64_t T, int64_t N, int64_t K) {
  if (shape_of(T, 1, 1, false, true, 2).own) return 1;
  const int64_t tiles = (N + 63) / 64 * ((T + kChunk - 1) / kChunk), most = (K + 127) / 128 / 6;
  int64_t s = 256 / tiles;
  if (s > most) s = most;
  return s < 2 ? 1 : s > 16 ? 16 : (int)s;
}
static inline size_t linear_bytes(int64_t T, int64_t N, int64_t K) {
  const int s = linear_splits(T, N, K);
  return s > 1 ? (size_t)s * T * N * 4 : 0;
}

template <class E, int FMT>
int run_linear(const Call& c) {
  Args g = args_of(c, c.x, c.D, c.H, c.y);
  const Shape f = shape_of(c.T, 1, 1, false, true, 2);
  const bool wide = (c.D + 31) / 32 >= 3 * dev_ncu();
  if (f.rows == 8) {
    if (wide) return launch_gateup<E, FMT, 2, 4, 4, 1, true>(g, 1, c.stream);
    return gateup_own<E, FMT, 4, true>(g, 1, c.stream);
  }
  if (f.rows == 16) {
    if (wide) return launch_gateup<E, FMT, 2, 16, 4, 1, true>(g, 1, c.stream);
    return gateup_own<E, FMT, 16, true>(g, 1, c.stream);
  }
  g.splits = linear_splits(c.T, c.D, c.H);
  g.partial = (float*)c.ws;
  const int rc = f.rows == 32 ? launch_down<E, FMT, 32, 8, 4, kChunk, false>(g, c.stream)
                              : launch_down<E, FMT, 64, 8, 4, kChunk, false>(g, c.stream);
  if (rc || g.splits == 1) return rc;
  StageScope scope(STAGE_FEW_DOWN, c.stream);
  const int64_t quads = c.T * c.D / 4;
  hipLaunchKernelGGL((few_sum<E>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, c.stream, (const float*)c.ws,
                     (typename E::elem*)c.y, quads, g.splits);
  return hipGetLastError() == hipSuccess ? SWIGLU_OK : SWIGLU_ERR_LAUNCH;
}

template <class E, int FMT>
int run_block(const Call& c) {
  const Shape f = shape_of(c.T, c.k, c.E, c.ids != nullptr, FMT != 0, E::kBytes);
  const BlockPlan p = block_plan(f, c.T, c.D, c.H, c.k, E::kBytes);
  Args g = args_of(c, c.x, c.H, c.D, c.ws);
  g.w0 = c.wg;
  g.w1 = c.wu;
  g.once = c.D * E::kBytes % 128 == 0;
  g.ctr = (unsigned*)(c.ws + p.ctr);
  g.n_ctr = p.n_ctr;
  const int64_t pairs = (c.T < kChunk ? c.T : kChunk) * c.k;
  const int slots = c.ids ? (int)(pairs < c.E ? pairs : c.E) : 1;
  const int rc = gateup_for<E, FMT>(g, f, slots, c.stream);
  if (rc) return rc;
  Args d = args_of(c, c.ws, c.D, c.H, c.y);
  d.once = c.H * E::kBytes % 128 == 0;
  d.splits = p.down.splits;
  d.partial = (float*)(c.ws + p.partial);
  d.ctr = g.ctr;
  return down_for<E, FMT>(d, f, p.down.waves, c.stream);
}

}  // namespace few
}  // namespace swiglu

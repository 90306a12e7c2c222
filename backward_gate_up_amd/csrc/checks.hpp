// checks.hpp -- host-side argument validation shared by the C entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "swiglu_mlp.h"

namespace swiglu {

static inline size_t elt_bytes(int dt) { return dt == SWIGLU_FP32 ? 4 : (dt == SWIGLU_BF16 || dt == SWIGLU_FP16 ? 2 : 0); }

static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

struct Range {
  const void* p;
  size_t n;
};
static inline bool overlap(Range a, Range b) {
  if (a.n == 0 || b.n == 0) return false;
  uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Pointers to non-empty buffers must be non-NULL and 16-byte aligned;
// a buffer of zero bytes (T = 0) may be NULL.
static inline int check_ptrs(const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    if (r[i].n > 0 && !r[i].p) return SWIGLU_ERR_NULL;
  for (int i = 0; i < n; ++i)
    if (r[i].p && !aligned16(r[i].p)) return SWIGLU_ERR_ALIGN;
  return SWIGLU_OK;
}

// Largest D or H (the leading dimensions of every operand) for which the
// kernels' 32-bit per-lane byte offsets stay in range: a tile spans 256 rows
// of an operand, at offsets up to 256 * ld * elt_bytes, and each buffer
// descriptor holds at most 2^31 - 1 bytes. 16-bit: 4194296; fp32: 2097144
// (multiples of 8).
static inline int64_t max_ld(size_t e) { return ((0x7fffffffLL / (256 * (int64_t)e)) / 8) * 8; }

static inline int check_shape(int64_t T, int64_t D, int64_t H, size_t e) {
  if (T < 0 || D <= 0 || H <= 0) return SWIGLU_ERR_SHAPE;
  if ((D & 7) || (H & 7)) return SWIGLU_ERR_SHAPE;
  if (D > max_ld(e) || H > max_ld(e)) return SWIGLU_ERR_SHAPE;
  // token rows are int32 inside the kernels, and so is every launch's tile
  // count (64-row tiles of T times 64-column tiles of the wider of D and H)
  if (T > 0x7fffffffLL) return SWIGLU_ERR_SHAPE;
  const int64_t w = (D > H ? D : H) / 64 + 1;
  if ((T / 64 + 1) > 0x3fffffffLL / w) return SWIGLU_ERR_SHAPE;
  return SWIGLU_OK;
}

static inline int check_device() {
  static int cached[64];  // 0 unknown, 1 ok, 2 bad
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return SWIGLU_ERR_DEVICE;
  if (cached[dev] == 0) {
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) return SWIGLU_ERR_DEVICE;
    cached[dev] = strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
  }
  return cached[dev] == 1 ? SWIGLU_OK : SWIGLU_ERR_DEVICE;
}

}  // namespace swiglu

// What the kernels of the paged caches share: the checked view of a batch's rows and pages and powers of two;
// and what the 8-bit ones do: e4m3 conversions and the power-of-two scales.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "cpattn.h"

namespace cpattn {
namespace kv {

// Sites of the status word of the cache kernels (bits 8 and up).
enum Site { kSitePage = 32, kSiteTokens = 33, kSiteWait = 34, kSiteRows = 35 };

__device__ __forceinline__ void report(int32_t* status, int site) {
  if (status != nullptr) atomicCAS(status, 0, CP_ERR_INVALID_ARG | (site << 8));
}

// row_start[i] clamped to what the caller's arrays hold.
__device__ __forceinline__ int64_t row_at(const cp_kv_rows& r, int i) {
  const int64_t x = __ldg(r.row_start + i);
  return x < 0 ? 0 : (x > r.n_rows ? r.n_rows : x);
}

// Page of `ord`-th page of sequence b, or -1 where the table does not reach or names no page.
__device__ __forceinline__ int64_t page_at(const cp_kv_rows& r, int64_t n_pages, int b, int64_t ord) {
  if (ord < 0 || ord >= r.max_pages) return -1;
  const int64_t p = __ldg(r.page_table + static_cast<int64_t>(b) * r.max_pages + ord);
  return p < n_pages ? p : -1;  // a negative entry is no page either
}

// The last sequence b in [0, n_seqs) with key(b) <= x, found by the whole warp: 32 probes a round,
// so one round for up to 32 sequences and three for the largest batch.  key is non-decreasing
// with key(0) <= x; for other keys the answer is still in range.
template <class Key>
__device__ __forceinline__ int find_seq(int n_seqs, int64_t x, int lane, Key key) {
  int lo = 0, n = n_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < n && key(at) <= x;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int hit = m == 0u ? 0 : 31 - __clz(m);
    const int rest = n - hit * step;
    lo += hit * step;
    n = step < rest ? step : rest;
  }
  return lo;
}

// Two fp32 to two e4m3 bytes (first in the low byte): round to nearest even, saturating; NaN stays.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 bytes to f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// |x| where it counts for a scale: infinities and NaN do not.
__device__ __forceinline__ float magnitude(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;
}

// Exponent e of the scale of magnitude `amax`: the smallest e >= -64 with amax <= 448 * 2^e.  448
// is 1.75 * 2^8, so with amax = 1.f * 2^x it is x - 8, and one more where 1.f > 1.75.
constexpr int kMinScaleExp = -64;
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kMinScaleExp ? kMinScaleExp : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace kv
}  // namespace cpattn

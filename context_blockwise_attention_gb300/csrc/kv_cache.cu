// Writing tokens into the paged e4m3 cache and reading them back (cp_kv_cache_write / _read).
#include "internal.h"
#include "kv_common.cuh"

namespace cpattn {

namespace {

using kv::find_seq;

constexpr int kThreads = 256;

// N consecutive elements of a row as fp32 (N * sizeof(T) is 4, 8 or 16 bytes).
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
  if constexpr (N == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = v.x, x[1] = v.y;
  }
}
__device__ __forceinline__ void unpack_bf16x2(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xffff0000u);
}
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[N]) {
  if constexpr (N == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    unpack_bf16x2(v.x, x[0], x[1]);
    unpack_bf16x2(v.y, x[2], x[3]);
  } else {
    unpack_bf16x2(__ldg(reinterpret_cast<const uint32_t*>(p)), x[0], x[1]);
  }
}

// The page that a unit of work stands for.  Sequence b owns the unit numbers from
// U(b) = floor(row_start[b] / P) + 2 b on: as many as its rows can touch pages, whatever slot they
// begin at, so that the grid's size follows from the row count alone and no prefix sum over the
// sequences is needed.
struct PageSpan {
  int64_t page;  // -1: bad
  int64_t row;   // first row of the call that goes into it
  int slot, n;   // slots [slot, slot + n)
};
__device__ __forceinline__ bool span_of(const cp_kv_rows& r, int64_t n_pages, int P, int64_t unit, int lane,
                                        PageSpan& out) {
  const int b = find_seq(r.n_seqs, unit, lane, [&](int i) { return kv::row_at(r, i) / P + 2 * static_cast<int64_t>(i); });
  const int64_t r0 = kv::row_at(r, b), r1 = kv::row_at(r, b + 1);
  const int64_t first = __ldg(r.tokens + b);
  const int64_t k = unit - (r0 / P + 2 * static_cast<int64_t>(b));
  if (r1 <= r0 || first < 0 || k < 0) return false;
  const int64_t ord = first / P + k;
  const int64_t begin = k == 0 ? first : ord * P;  // first token of the call in this page
  const int64_t end = first + (r1 - r0);
  if (begin >= end) return false;
  out.page = kv::page_at(r, n_pages, b, ord);
  out.row = r0 + (begin - first);
  out.slot = static_cast<int>(begin - ord * P);
  const int64_t room = P - out.slot, left = end - begin;
  out.n = static_cast<int>(room < left ? room : left);
  return true;
}

struct WriteParams {
  cp_kv_cache c;
  cp_kv_rows rows;
  const void* x[2];  // k, v
  int32_t* status;
  int64_t units;
};

// One warp per (page, head, K or V): it goes over the page's new rows twice, first for the largest
// magnitude and then to convert them, and over the older slots where the scale grew.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_write_warp_kernel(const WriteParams p) {
  constexpr int kN = D / 32;  // elements of a row per lane
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int hkv = p.c.hkv, P = p.c.page_size;
  const int64_t unit = w / (2 * hkv);
  if (unit >= p.units) return;
  const int sub = static_cast<int>(w - unit * (2 * hkv));
  const int which = sub & 1, head = sub >> 1;
  PageSpan s;
  if (!span_of(p.rows, p.c.n_pages, P, unit, lane, s)) return;
  if (s.page < 0) {
    if (lane == 0) kv::report(p.status, kv::kSitePage);
    return;
  }
  const T* x = static_cast<const T*>(p.x[which]) + (s.row * hkv + head) * D + lane * kN;
  const int64_t tile = s.page * hkv + head;
  uint8_t* out = static_cast<uint8_t*>(which ? p.c.v : p.c.k) + tile * P * D + lane * kN;
  float* scale = (which ? p.c.v_scale : p.c.k_scale) + tile;
  const float old = s.slot > 0 ? *scale : 0.0f;
  float amax = 0.0f;
  for (int i = 0; i < s.n; ++i) {
    float e[kN];
    load_row<kN>(x + static_cast<int64_t>(i) * hkv * D, e);
#pragma unroll
    for (int j = 0; j < kN; ++j) amax = fmaxf(amax, kv::magnitude(e[j]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int ex = kv::scale_exp(amax);
  float now = kv::pow2(ex), inv = kv::pow2(-ex);
  if (s.slot > 0) {
    if (old >= now) {
      now = old;
      inv = 1.0f / old;  // exact: a power of two
    } else {
      const float ratio = old / now;
      for (int i = 0; i < s.slot; ++i) {
        uint8_t* q = out + i * D;
        if constexpr (kN == 4) {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(q);
          const float2 a = kv::e4m3x2_to_float2(v), b = kv::e4m3x2_to_float2(v >> 16);
          *reinterpret_cast<uint32_t*>(q) =
              kv::to_e4m3x2(a.x * ratio, a.y * ratio) | (kv::to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
        } else {
          const float2 a = kv::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(q));
          *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(kv::to_e4m3x2(a.x * ratio, a.y * ratio));
        }
      }
    }
  }
  for (int i = 0; i < s.n; ++i) {
    float e[kN];
    load_row<kN>(x + static_cast<int64_t>(i) * hkv * D, e);
    uint8_t* q = out + (s.slot + i) * D;
    const uint32_t lo = kv::to_e4m3x2(e[0] * inv, e[1] * inv);
    if constexpr (kN == 4)
      *reinterpret_cast<uint32_t*>(q) = lo | (kv::to_e4m3x2(e[2] * inv, e[3] * inv) << 16);
    else
      *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(lo);
  }
  if (lane == 0 && now != old) *scale = now;
}

struct ReadParams {
  cp_kv_cache c;
  cp_kv_rows rows;
  void* x[2];
  int32_t* status;
};

// One warp per (row, head).
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
  constexpr int kN = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int hkv = p.c.hkv, P = p.c.page_size;
  const int64_t row = w / hkv;
  const int head = static_cast<int>(w - row * hkv);
  if (row >= p.rows.n_rows) return;
  const int b = find_seq(p.rows.n_seqs, row, lane, [&](int i) { return kv::row_at(p.rows, i); });
  const int64_t r0 = kv::row_at(p.rows, b), r1 = kv::row_at(p.rows, b + 1);
  const int64_t first = __ldg(p.rows.tokens + b);
  if (row < r0 || row >= r1) return;
  const int64_t token = first + (row - r0);
  const int64_t page = first < 0 ? -1 : kv::page_at(p.rows, p.c.n_pages, b, token / P);
  if (page < 0) {
    if (lane == 0) kv::report(p.status, kv::kSitePage);
    return;
  }
  const int64_t tile = page * hkv + head;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint8_t* q =
        static_cast<const uint8_t*>(which ? p.c.v : p.c.k) + (tile * P + token % P) * D + lane * kN;
    const float scale = __ldg((which ? p.c.v_scale : p.c.k_scale) + tile);
    T* out = static_cast<T*>(p.x[which]) + (row * hkv + head) * D + lane * kN;
#pragma unroll
    for (int j = 0; j < kN; j += 2) {
      const float2 f = kv::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(q + j));
      out[j] = static_cast<T>(f.x * scale);
      out[j + 1] = static_cast<T>(f.y * scale);
    }
  }
}

template <class K, class P>
cp_status launch(K kernel, const P& p, int64_t warps, const char* what, cudaStream_t s) {
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) {
    set_error("%s: too many rows", what);
    return CP_ERR_INVALID_ARG;
  }
  kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? CP_OK : cuda_fail(e, what);
}

}  // namespace

cp_status launch_kv_write(const cp_kv_cache& c, const cp_kv_rows& rows, const void* k, const void* v, bool bf16,
                          int32_t* status, cudaStream_t s) {
  WriteParams p{c, rows, {k, v}, status, rows.n_rows / c.page_size + 2 * static_cast<int64_t>(rows.n_seqs)};
  const int64_t warps = p.units * c.hkv * 2;
  const char* what = "kv_write_warp_kernel launch";
  if (c.d == 128)
    return bf16 ? launch(kv_write_warp_kernel<128, __nv_bfloat16>, p, warps, what, s)
                : launch(kv_write_warp_kernel<128, float>, p, warps, what, s);
  return bf16 ? launch(kv_write_warp_kernel<64, __nv_bfloat16>, p, warps, what, s)
              : launch(kv_write_warp_kernel<64, float>, p, warps, what, s);
}

cp_status launch_kv_read(const cp_kv_cache& c, const cp_kv_rows& rows, void* k, void* v, bool bf16, int32_t* status,
                         cudaStream_t s) {
  ReadParams p{c, rows, {k, v}, status};
  const int64_t warps = rows.n_rows * c.hkv;
  const char* what = "kv_read_kernel launch";
  if (c.d == 128)
    return bf16 ? launch(kv_read_kernel<128, __nv_bfloat16>, p, warps, what, s)
                : launch(kv_read_kernel<128, float>, p, warps, what, s);
  return bf16 ? launch(kv_read_kernel<64, __nv_bfloat16>, p, warps, what, s)
              : launch(kv_read_kernel<64, float>, p, warps, what, s);
}

}  // namespace cpattn

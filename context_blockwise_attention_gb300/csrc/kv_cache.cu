// Writing tokens into the paged e4m3 cache and reading them back (cp_kv_cache_write / _read).
#include "internal.h"
#include "kv_common.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using kv::find_seq;

constexpr int kThreads = 256;
constexpr int kReadBlocks = 5;  // blocks of the reading kernel that an SM holds

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
  int page;     // -1: bad
  int row;      // first row of the call that goes into it
  int slot, n;  // slots [slot, slot + n)
};
__device__ __forceinline__ bool span_of(const cp_kv_rows& r, int64_t n_pages, int P, uint32_t unit, int lane,
                                        PageSpan& out) {
  const int shift = 31 - __clz(P);
  auto begin = [&](int i) { return (static_cast<uint32_t>(kv::row_at(r, i)) >> shift) + 2u * i; };
  const int b = find_seq(r.n_seqs, unit, lane, [&](int i) { return static_cast<int64_t>(begin(i)); });
  const int r0 = static_cast<int>(kv::row_at(r, b)), r1 = static_cast<int>(kv::row_at(r, b + 1));
  const int first = __ldg(r.tokens + b);
  const uint32_t at = begin(b);
  if (r1 <= r0 || first < 0 || unit < at) return false;
  const int64_t ord = (first >> shift) + static_cast<int64_t>(unit - at);
  const int64_t from = unit == at ? first : ord << shift;  // first token of the call in this page
  const int64_t end = static_cast<int64_t>(first) + (r1 - r0);
  if (from >= end) return false;
  out.page = static_cast<int>(kv::page_at(r, n_pages, b, ord));
  out.row = r0 + static_cast<int>(from - first);
  out.slot = static_cast<int>(from - (ord << shift));
  const int64_t left = end - from;
  out.n = static_cast<int>(P - out.slot < left ? P - out.slot : left);
  return true;
}

// Four cached bytes at a larger scale: old scale / new scale is `ratio`.
__device__ __forceinline__ void requantise4(uint8_t* q, float ratio) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(q);
  const float2 a = kv::e4m3x2_to_float2(v), b = kv::e4m3x2_to_float2(v >> 16);
  *reinterpret_cast<uint32_t*>(q) =
      kv::to_e4m3x2(a.x * ratio, a.y * ratio) | (kv::to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

// Reports row starts and counts that break the rules.  A launch of its own, where there is a status word to report to:
// as the first block's task in the writing kernels it cost calls without one up to 16 % (other code for the copies).
__global__ void __launch_bounds__(kThreads) kv_check_rows_kernel(const __grid_constant__ cp_kv_rows r, int32_t* status) {
  ptx::wait_dependencies();
  for (int b = threadIdx.x; b < r.n_seqs; b += kThreads) {
    const int from = __ldg(r.row_start + b), to = __ldg(r.row_start + b + 1);
    if (from < 0 || to < from || to > r.n_rows) kv::report(status, kv::kSiteRows);
    else if (from < to && __ldg(r.tokens + b) < 0) kv::report(status, kv::kSiteTokens);
  }
}

struct WriteParams {
  cp_kv_cache c;
  cp_kv_rows rows;
  const void* x[2];  // k, v
  int32_t* status;
  uint32_t units;
  int32_t heads, pages;  // of a block of the tile kernel
};

// One warp per (page, head, K or V): it goes over the page's new rows twice, first for the largest
// magnitude and then to convert them, and over the older slots where the scale grew.  Bound by latency:
// one token each of 128 sequences, 8 heads: 2.7 us.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_write_warp_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kN = D / 32;  // elements of a row per lane
  const int lane = threadIdx.x & 31;
  const int hkv = p.c.hkv, P = p.c.page_size;
  const uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), unit = w / (2u * hkv);
  if (unit >= p.units) return;
  const int sub = static_cast<int>(w - unit * (2u * hkv));
  const int which = sub & 1, head = sub >> 1;
  ptx::wait_dependencies();
  PageSpan s;
  if (!span_of(p.rows, p.c.n_pages, P, unit, lane, s)) return;
  if (s.page < 0) {
    if (lane == 0) kv::report(p.status, kv::kSitePage);
    return;
  }
  const T* x = static_cast<const T*>(p.x[which]) + (static_cast<int64_t>(s.row) * hkv + head) * D + lane * kN;
  const int64_t tile = static_cast<int64_t>(s.page) * hkv + head;
  uint8_t* out = static_cast<uint8_t*>(which ? p.c.v : p.c.k) + tile * P * D + lane * kN;
  float* scale = (which ? p.c.v_scale : p.c.k_scale) + tile;
  const float old = s.slot > 0 ? *scale : 0.0f;
  float amax = 0.0f;
#pragma unroll 4
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
          requantise4(q, ratio);
        } else {
          const float2 a = kv::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(q));
          *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(kv::to_e4m3x2(a.x * ratio, a.y * ratio));
        }
      }
    }
  }
#pragma unroll 4
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

// 16 bytes of a row as fp32: 8 bf16 or 4 fp32.
template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  unpack_bf16x2(v.x, x[0], x[1]);
  unpack_bf16x2(v.y, x[2], x[3]);
  unpack_bf16x2(v.z, x[4], x[5]);
  unpack_bf16x2(v.w, x[6], x[7]);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}

// Largest counting magnitude of 16 bytes.  The maximum passes over NaN by itself; where it finds an
// infinity it is taken again without.
__device__ __forceinline__ float top_of(const uint4& v, const __nv_bfloat16*) {
  auto abs2 = [](uint32_t u) {
    u &= 0x7fff7fffu;
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  };
  const __nv_bfloat162 m = __hmax2(__hmax2(abs2(v.x), abs2(v.y)), __hmax2(abs2(v.z), abs2(v.w)));
  float top = fmaxf(__low2float(m), __high2float(m));
  if (!(top < INFINITY)) {
    float e[8];
    unpack(v, e);
    top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, kv::magnitude(e[j]));
  }
  return top;
}
__device__ __forceinline__ float top_of(const uint4& v, const float*) {
  float e[4];
  unpack(v, e);
  float top = fmaxf(fmaxf(fabsf(e[0]), fabsf(e[1])), fmaxf(fabsf(e[2]), fabsf(e[3])));
  if (!(top < INFINITY))
    top = fmaxf(fmaxf(kv::magnitude(e[0]), kv::magnitude(e[1])), fmaxf(kv::magnitude(e[2]), kv::magnitude(e[3])));
  return top;
}

// Prompts: the threads of a tile (page, head, K or V) hold its new rows in registers between the
// largest magnitude and the conversion, so that they are read once.  A block takes as many heads of
// one page at once as fit, and goes over p.heads of them, so that where the page lies is looked up
// once; where there are fewer heads than fit it takes p.pages pages (96 k and 196 k tokens of 1 x 64 bf16, pages
// of 16 and 32: 8.6 and 18 us for 37 and 75 MB, with one page a block 39 and 44).  Bound by memory: 2 or 4 bytes
// in and 1 out per number; 16-byte loads, all of a thread's in flight at once: 64 numbers a thread, 32 in small
// pages (29 k tokens of 8 x 128 bf16, pages of 64, 178 MB: 28.7 us, 6.2 TB/s, with 32 a thread 30.8; 32 k tokens,
// pages of 16: 34 us with 32, 36 with 64, 40 with 16).
template <int D, int P>
constexpr int kTileThreads = P >= 64 ? P * D / 64 : P * D / 32;
template <int D, int P, class T>
__global__ void __launch_bounds__(kThreads) kv_write_tile_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kV = kVec<T>, kTT = kTileThreads<D, P>, kTiles = kThreads / kTT;
  constexpr int kPerRow = D / kV, kRowsAtOnce = kTT / kPerRow, kPasses = P / kRowsAtOnce;
  __shared__ float tops[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = p.c.hkv;
  const int which = blockIdx.y & 1, h0 = (blockIdx.y >> 1) * p.heads;
  const int h1 = h0 + p.heads < hkv ? h0 + p.heads : hkv;
  const int at = tid % kTT, row0 = at / kPerRow, col = at % kPerRow * kV;
  const int nth = p.pages > 1 ? tid / kTT / hkv : 0;  // page of the block; the same for a whole warp
  const uint32_t unit = blockIdx.x * p.pages + nth;
  ptx::wait_dependencies();
  PageSpan s;
  bool some = nth < p.pages && unit < p.units && span_of(p.rows, p.c.n_pages, P, unit, lane, s);
  if (some && s.page < 0) {
    if (at == 0 && tid / kTT == nth * hkv) kv::report(p.status, kv::kSitePage);
    some = false;
  }
  if (!some) {
    if (p.pages == 1) return;  // the same for the whole block
    s = PageSpan{0, 0, 0, 0};
  }
  int turn = 0;
  for (int h = h0; h < h1; h += kTiles, turn ^= 1) {
    const int head = h + tid / kTT - nth * hkv;
    const bool mine = some && head < h1;
    const T* x = static_cast<const T*>(p.x[which]) + (static_cast<int64_t>(s.row) * hkv + head) * D + col;
    const int64_t tile = static_cast<int64_t>(s.page) * hkv + head;
    uint8_t* out = static_cast<uint8_t*>(which ? p.c.v : p.c.k) + tile * P * D + col;
    float* scale = (which ? p.c.v_scale : p.c.k_scale) + tile;
    const float old = mine && s.slot > 0 ? *scale : 0.0f;
    uint4 held[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = row0 + i * kRowsAtOnce;
      held[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mine && r < s.n) held[i] = __ldcs(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(r) * hkv * D));
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) amax = fmaxf(amax, top_of(held[i], x));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) tops[turn][warp] = amax;
    __syncthreads();  // two sets of maxima: the next head's do not wait for these to be read
#pragma unroll
    for (int i = 0; i < kTT / 32; ++i) amax = fmaxf(amax, tops[turn][warp / (kTT / 32) * (kTT / 32) + i]);
    if (!mine) continue;
    const int ex = kv::scale_exp(amax);
    float now = kv::pow2(ex), inv = kv::pow2(-ex);
    if (old >= now) {
      now = old;
      inv = 1.0f / old;  // exact: a power of two
    } else if (s.slot > 0) {
      const float ratio = old / now;
      for (int r = row0; r < s.slot; r += kRowsAtOnce)
#pragma unroll
        for (int j = 0; j < kV; j += 4) requantise4(out + r * D + j, ratio);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = row0 + i * kRowsAtOnce;
      if (r >= s.n) break;
      float e[kV];
      unpack(held[i], e);
      uint32_t w[kV / 4];
#pragma unroll
      for (int j = 0; j < kV; j += 4)
        w[j / 4] = kv::to_e4m3x2(e[j] * inv, e[j + 1] * inv) | (kv::to_e4m3x2(e[j + 2] * inv, e[j + 3] * inv) << 16);
      uint8_t* q = out + (s.slot + r) * D;
      if constexpr (kV == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(q) = w[0];
    }
    if (at == 0 && now != old) *scale = now;
  }
}

struct ReadParams {
  cp_kv_cache c;
  cp_kv_rows rows;
  void* x[2];
  int32_t* status;
  int32_t heads, per_block;  // heads and rows of a block
};

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A thread writes 16 bytes at a time, so that a warp's stores fill whole lines (two stores of 16 bytes to
// neighbouring places touched every sector twice), and goes over the heads of its row: where a token
// lives is looked up once.  Bound by memory: 1 byte in and 2 or 4 out per number; the loads of kAhead
// heads are in flight together.  31 k tokens of 8 x 128 to bf16 (191 MB): 33.3 us, 5.7 TB/s.
template <int D, class T>
__global__ void __launch_bounds__(kThreads, kReadBlocks) kv_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kV = kVec<T>, kCols = D / kV, kRows = kThreads / kCols, kAhead = 8;
  __shared__ int seqs[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = p.c.hkv, P = p.c.page_size, shift = 31 - __clz(P);
  const int n_rows = static_cast<int>(p.rows.n_rows);
  const int row0 = blockIdx.x * p.per_block;
  const int row_end = n_rows - row0 < p.per_block ? n_rows : row0 + p.per_block;
  const int which = blockIdx.y & 1, h0 = (blockIdx.y >> 1) * p.heads;
  const int h1 = h0 + p.heads < hkv ? h0 + p.heads : hkv;
  const int col = tid % kCols * kV;
  ptx::wait_dependencies();
  if (warp < 2) {  // the sequences of the block's first and last row
    const int b = find_seq(p.rows.n_seqs, warp == 0 ? row0 : row_end - 1, lane,
                           [&](int i) { return kv::row_at(p.rows, i); });
    if (lane == 0) seqs[warp] = b;
  }
  __syncthreads();
  const uint8_t* const cache = static_cast<const uint8_t*>(which ? p.c.v : p.c.k);
  const float* const scales = which ? p.c.v_scale : p.c.k_scale;
  for (int row = row0 + tid / kCols; row < row_end; row += kRows) {
    int b = seqs[0], z = seqs[1];
    while (b < z) {  // the last one that begins at or before the row
      const int mid = (b + z + 1) >> 1;
      if (kv::row_at(p.rows, mid) <= row) b = mid;
      else z = mid - 1;
    }
    const int r0 = static_cast<int>(kv::row_at(p.rows, b)), r1 = static_cast<int>(kv::row_at(p.rows, b + 1));
    const int first = __ldg(p.rows.tokens + b);
    if (row < r0 || row >= r1) continue;
    const int64_t token = static_cast<int64_t>(first) + (row - r0);
    const int64_t page = first < 0 ? -1 : kv::page_at(p.rows, p.c.n_pages, b, token >> shift);
    if (page < 0) {
      kv::report(p.status, kv::kSitePage);
      continue;
    }
    const uint8_t* src = cache + ((page * hkv + h0) * P + (token & (P - 1))) * D + col;
    const float* scale = scales + page * hkv;
    T* dst = static_cast<T*>(p.x[which]) + (static_cast<int64_t>(row) * hkv + h0) * D + col;
    for (int h = h0; h < h1; h += kAhead) {
      uint32_t v[kAhead][kV / 4];
      float f[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < h1) {
          const uint8_t* q = src + static_cast<int64_t>(i) * P * D;
          if constexpr (kV == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(q));
            v[i][0] = u.x, v[i][kV / 4 - 1] = u.y;
          } else {
            v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(q));
          }
          f[i] = __ldg(scale + h + i);
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < h1) {
          float x[kV];
#pragma unroll
          for (int j = 0; j < kV / 4; ++j) {
            const float2 lo = kv::e4m3x2_to_float2(v[i][j]), hi = kv::e4m3x2_to_float2(v[i][j] >> 16);
            x[4 * j] = lo.x * f[i], x[4 * j + 1] = lo.y * f[i];
            x[4 * j + 2] = hi.x * f[i], x[4 * j + 3] = hi.y * f[i];
          }
          T* to = dst + i * D;
          if constexpr (kV == 8)
            __stcs(reinterpret_cast<uint4*>(to), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                            pack_bf16x2(x[kV - 4], x[kV - 3]),
                                                            pack_bf16x2(x[kV - 2], x[kV - 1])));
          else
            __stcs(reinterpret_cast<float4*>(to), make_float4(x[0], x[1], x[2], x[3]));
        }
      src += static_cast<int64_t>(kAhead) * P * D;
      dst += kAhead * D;
    }
  }
}

// The same for up to four heads of a block, where a row alone does not keep enough loads in flight: a block
// looks up where its rows' tokens live, a thread a row, and then goes over (row, head) pairs, kAhead of a
// thread's in flight together.  60 k tokens of 1 / 2 / 3 / 4 x 128 to bf16: 8.1 / 13.2 / 22.4 / 33 us, against 21 /
// 22.6 / 26.4 / 33 the other way; 31 k tokens of 8 x 128 35.1 against 33.6.
template <int D, class T>
__global__ void __launch_bounds__(kThreads, kReadBlocks) kv_read_few_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kV = kVec<T>, kCols = D / kV, kPairs = kThreads / kCols, kAhead = 8;
  __shared__ int seqs[2];
  __shared__ int64_t place[kThreads];  // (page * hkv) * P + slot of a row, -1: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hkv = p.c.hkv, P = p.c.page_size, shift = 31 - __clz(P);
  const int n_rows = static_cast<int>(p.rows.n_rows);
  const int row0 = blockIdx.x * p.per_block;
  const int row_end = n_rows - row0 < p.per_block ? n_rows : row0 + p.per_block;
  const int which = blockIdx.y & 1, h0 = (blockIdx.y >> 1) * p.heads;
  const int heads = hkv - h0 < p.heads ? hkv - h0 : p.heads;
  const float inv_heads = 1.0f / static_cast<float>(heads);
  const int col = tid % kCols * kV;
  ptx::wait_dependencies();
  if (warp < 2) {  // the sequences of the block's first and last row
    const int b = find_seq(p.rows.n_seqs, warp == 0 ? row0 : row_end - 1, lane,
                           [&](int i) { return kv::row_at(p.rows, i); });
    if (lane == 0) seqs[warp] = b;
  }
  const uint8_t* const cache = static_cast<const uint8_t*>(which ? p.c.v : p.c.k) + col;
  const float* const scales = which ? p.c.v_scale : p.c.k_scale;
  T* const x_out = static_cast<T*>(p.x[which]) + col;
  for (int base = row0; base < row_end; base += kThreads) {
    const int n = row_end - base < kThreads ? row_end - base : kThreads;
    __syncthreads();  // the places of the rows before have been read
    if (tid < n) {
      const int row = base + tid;
      int b = seqs[0], z = seqs[1];
      while (b < z) {  // the last one that begins at or before the row
        const int mid = (b + z + 1) >> 1;
        if (kv::row_at(p.rows, mid) <= row) b = mid;
        else z = mid - 1;
      }
      const int r0 = static_cast<int>(kv::row_at(p.rows, b)), r1 = static_cast<int>(kv::row_at(p.rows, b + 1));
      const int first = __ldg(p.rows.tokens + b);
      int64_t at = -1;
      if (row >= r0 && row < r1) {
        const int64_t token = static_cast<int64_t>(first) + (row - r0);
        const int64_t page = first < 0 ? -1 : kv::page_at(p.rows, p.c.n_pages, b, token >> shift);
        if (page < 0) kv::report(p.status, kv::kSitePage);
        else at = page * hkv * P + (token & (P - 1));
      }
      place[tid] = at;
    }
    __syncthreads();
    const int pairs = n * heads;
    for (int i0 = tid / kCols; i0 < pairs; i0 += kPairs * kAhead) {
      uint32_t v[kAhead][kV / 4];
      float f[kAhead];
      int to[kAhead];  // row of the output's (row, head) pairs from (base, 0) on, -1: none
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int pair = i0 + i * kPairs;
        to[i] = -1;
        if (pair < pairs) {
          const int r = static_cast<int>((static_cast<float>(pair) + 0.5f) * inv_heads);  // exact: below 2^22
          const int h = h0 + pair - r * heads;
          const int64_t at = place[r];
          if (at >= 0) {
            to[i] = r * hkv + h;
            const uint8_t* q = cache + (at + static_cast<int64_t>(h) * P) * D;
            if constexpr (kV == 8) {
              const uint2 u = __ldg(reinterpret_cast<const uint2*>(q));
              v[i][0] = u.x, v[i][kV / 4 - 1] = u.y;
            } else {
              v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(q));
            }
            f[i] = __ldg(scales + (at >> shift) + h);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (to[i] >= 0) {
          float x[kV];
#pragma unroll
          for (int j = 0; j < kV / 4; ++j) {
            const float2 lo = kv::e4m3x2_to_float2(v[i][j]), hi = kv::e4m3x2_to_float2(v[i][j] >> 16);
            x[4 * j] = lo.x * f[i], x[4 * j + 1] = lo.y * f[i];
            x[4 * j + 2] = hi.x * f[i], x[4 * j + 3] = hi.y * f[i];
          }
          T* const o = x_out + (static_cast<int64_t>(base) * hkv + to[i]) * D;
          if constexpr (kV == 8)
            __stcs(reinterpret_cast<uint4*>(o), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                           pack_bf16x2(x[kV - 4], x[kV - 3]),
                                                           pack_bf16x2(x[kV - 2], x[kV - 1])));
          else
            __stcs(reinterpret_cast<float4*>(o), make_float4(x[0], x[1], x[2], x[3]));
        }
    }
  }
}

template <class K, class... P>
cp_status launch(K kernel, int64_t bx, int64_t by, const char* what, cudaStream_t s, const P&... p) {
  if (bx > 0x7fffffff || by > 65535) {
    set_error("%s: too many rows or heads", what);
    return CP_ERR_INVALID_ARG;
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by));
  cfg.blockDim = dim3(kThreads);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p...);
  return e == cudaSuccess ? CP_OK : cuda_fail(e, what);
}

// Heads of a block, so that `blocks` blocks a head make at least `want` blocks in all.
int32_t heads_of(int32_t hkv, int64_t blocks, int64_t want) {
  const int64_t cut = (want + blocks - 1) / blocks;
  return static_cast<int32_t>((hkv + cut - 1) / cut);
}

template <int D, int P, class T>
cp_status write_tiles(WriteParams& p, int num_sms, cudaStream_t s) {
  constexpr int kTiles = kThreads / kTileThreads<D, P>;
  int32_t heads = heads_of(p.c.hkv, 2 * p.units, 8 * num_sms);
  p.heads = (heads + kTiles - 1) / kTiles * kTiles;
  p.pages = p.c.hkv < kTiles ? kTiles / p.c.hkv : 1;
  return launch(kv_write_tile_kernel<D, P, T>, (p.units + p.pages - 1) / p.pages,
                2 * ((p.c.hkv + p.heads - 1) / p.heads), "kv_write_tile_kernel launch", s, p);
}
template <int D, class T>
cp_status write(WriteParams& p, int num_sms, cudaStream_t s) {
  // Threads that hold a tile's rows pay where there are rows for them.  A warp a tile against them, us, bf16:
  // 100 sequences, 8 x 128, pages of 128: 24 rows 6.7 / 11, 64 rows 14.4 / 13.8, 128 rows 26 / 19, 512 rows 90 / 53;
  // pages of 64: 24 rows 7.3 / 9.0, 48 rows 11.6 / 10.8, 512 rows 81 / 53; of 32: 24 rows 6.4 / 7.7, 48 rows 11.6 /
  // 9.8, 512 rows 60 / 57; of 16: 64 rows 10.5 / 11.1, 96 rows 13.1 / 12.5, 512 rows 61 / 58 (fp32, 40 sequences: 256
  // rows 16.6 / 20, 384 rows 34 / 33); 64 sequences, 32 x 64, pages of 16: 4 rows 4.5 / 4.9, 8 rows 5.6 / 5.5, 512 rows
  // 110 / 71 (fp32: 8 rows 5.7 / 6.6, 16 rows 7.8 / 8.1, 32 rows 10.6 / 9.6, and with 8 heads 8 rows 3.3 / 3.2).  They
  // also pay where their blocks are few and a warp would take a tile's rows one after the other: 8 sequences, 8 x 128,
  // pages of 128: 8 rows 3.0 / 3.2, 32 rows 5.3 / 3.4, 64 rows 9.9 / 3.5.
  const int P = p.c.page_size;
  const int64_t tiles = static_cast<int64_t>(p.units) * p.c.hkv * 2, seqs = p.rows.n_seqs;
  const int64_t blocks = tiles * P * D / (P >= 64 ? 64 : 32) / kThreads;
  const int from = P == 128 ? 64 : P >= 32 ? 48 : D == 64 ? 8 : sizeof(T) == 2 ? 96 : 384;
  const bool long_rows = p.rows.n_rows >= seqs * from;
  const bool few = p.rows.n_rows >= 8 * seqs && blocks <= 2 * num_sms;
  if (!long_rows && !few) {
    const int64_t warps = tiles;
    return launch(kv_write_warp_kernel<D, T>, (warps + kThreads / 32 - 1) / (kThreads / 32), 1,
                  "kv_write_warp_kernel launch", s, p);
  }
  switch (p.c.page_size) {
    case 16: return write_tiles<D, 16, T>(p, num_sms, s);
    case 32: return write_tiles<D, 32, T>(p, num_sms, s);
    case 64: return write_tiles<D, 64, T>(p, num_sms, s);
    default: return write_tiles<D, 128, T>(p, num_sms, s);
  }
}
template <int D, class T>
cp_status read(ReadParams& p, int num_sms, cudaStream_t s) {
  // One wave of blocks with equal shares of the rows (31 k rows of 8 x 128: 33.3 us; 35.5 with a third of a
  // second wave); where the rows are few, fewer heads a block.
  constexpr int kRows = kThreads / (D / kVec<T>);
  const int64_t most = kReadBlocks * static_cast<int64_t>(num_sms) / 2;
  const int64_t per = (p.rows.n_rows + most - 1) / most;
  p.per_block = static_cast<int32_t>(per < kRows ? kRows : per);
  const int64_t bx = (p.rows.n_rows + p.per_block - 1) / p.per_block;
  p.heads = heads_of(p.c.hkv, 2 * bx, 4 * num_sms);
  const int64_t by = 2 * ((p.c.hkv + p.heads - 1) / p.heads);
  return p.heads > 4 ? launch(kv_read_kernel<D, T>, bx, by, "kv_read_kernel launch", s, p)
                     : launch(kv_read_few_kernel<D, T>, bx, by, "kv_read_few_kernel launch", s, p);
}

}  // namespace

cp_status launch_kv_check(const cp_kv_rows& rows, int32_t* status, cudaStream_t s) {
  return launch(kv_check_rows_kernel, 1, 1, "kv_check_rows_kernel launch", s, rows, status);
}

cp_status launch_kv_write(const cp_kv_cache& c, const cp_kv_rows& rows, const void* k, const void* v, bool bf16,
                          int32_t* status, int num_sms, cudaStream_t s) {
  const int64_t units = rows.n_rows / c.page_size + 2 * static_cast<int64_t>(rows.n_seqs);
  WriteParams p{c, rows, {k, v}, status, static_cast<uint32_t>(units), 0, 1};
  if (c.d == 128) return bf16 ? write<128, __nv_bfloat16>(p, num_sms, s) : write<128, float>(p, num_sms, s);
  return bf16 ? write<64, __nv_bfloat16>(p, num_sms, s) : write<64, float>(p, num_sms, s);
}

cp_status launch_kv_read(const cp_kv_cache& c, const cp_kv_rows& rows, void* k, void* v, bool bf16, int32_t* status,
                         int num_sms, cudaStream_t s) {
  ReadParams p{c, rows, {k, v}, status, 0, 0};
  if (c.d == 128) return bf16 ? read<128, __nv_bfloat16>(p, num_sms, s) : read<128, float>(p, num_sms, s);
  return bf16 ? read<64, __nv_bfloat16>(p, num_sms, s) : read<64, float>(p, num_sms, s);
}

}  // namespace cpattn

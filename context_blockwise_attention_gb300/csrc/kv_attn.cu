// Attention of a batch's new tokens over the paged 8-bit cache (cp_kv_cache_attn).
#include "internal.h"
#include "kv_common.cuh"

namespace cpattn {

namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnParams {
  cp_kv_cache c;
  cp_kv_rows rows;
  const void* q;
  void* o;
  float* lse;
  const int32_t* q_first;
  int32_t hq, q_bf16, o_bf16;
  float scale;
  cp_posmap kv_pos;
  int32_t* status;
};

// Number of cached tokens that a row at position `pos` sees: token j stands at base + stride j.
__device__ __forceinline__ int64_t visible(int64_t tokens, bool causal, int64_t pos, const cp_posmap& m) {
  if (!causal) return tokens;
  if (pos < m.base) return 0;
  const int64_t n = (pos - m.base) / m.stride + 1;
  return n < tokens ? n : tokens;
}

// One warp per (row, query head): D / 32 dimensions a lane, one key after the other.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_attn_row_kernel(const AttnParams p) {
  constexpr int kN = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = w / p.hq;
  const int h = static_cast<int>(w - row * p.hq);
  if (row >= p.rows.n_rows) return;
  const int b = kv::find_seq(p.rows.n_seqs, row, lane, [&](int i) { return kv::row_at(p.rows, i); });
  const int64_t r0 = kv::row_at(p.rows, b), r1 = kv::row_at(p.rows, b + 1);
  if (row < r0 || row >= r1) return;
  const int P = p.c.page_size, hkv = p.c.hkv, head = h / (p.hq / hkv);
  int64_t tokens = __ldg(p.rows.tokens + b);
  const int64_t held = static_cast<int64_t>(p.rows.max_pages) * P;
  const bool over = tokens > held;
  if (over) tokens = held;
  if (over && lane == 0) kv::report(p.status, kv::kSiteTokens);
  const bool causal = p.q_first != nullptr;
  const int64_t n = visible(tokens < 0 ? 0 : tokens, causal, causal ? __ldg(p.q_first + b) + (row - r0) : 0, p.kv_pos);
  float q[kN], acc[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int64_t at = (row * p.hq + h) * D + lane * kN + j;
    q[j] = p.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[at]) : static_cast<const float*>(p.q)[at];
    acc[j] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t ord = 0; ord * P < n; ++ord) {
    int64_t page = kv::page_at(p.rows, p.c.n_pages, b, ord);
    if (over && ord == p.rows.max_pages - 1) page = -1;
    if (page < 0) {
      if (lane == 0) kv::report(p.status, kv::kSitePage);
      m = l = __int_as_float(0x7fffffff);
      for (int j = 0; j < kN; ++j) acc[j] = m;
      break;
    }
    const int64_t tile = page * hkv + head;
    const float ks = __ldg(p.c.k_scale + tile), vs = __ldg(p.c.v_scale + tile);
    const int here = static_cast<int>(n - ord * P < P ? n - ord * P : P);
    for (int t = 0; t < here; ++t) {
      const uint8_t* kp = static_cast<const uint8_t*>(p.c.k) + (tile * P + t) * D + lane * kN;
      const uint8_t* vp = static_cast<const uint8_t*>(p.c.v) + (tile * P + t) * D + lane * kN;
      float z = 0.0f, v[kN];
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        const float2 f = kv::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(kp + j));
        const float2 g = kv::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(vp + j));
        z = fmaf(q[j], f.x, fmaf(q[j + 1], f.y, z));
        v[j] = g.x;
        v[j + 1] = g.y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      z *= ks * p.scale * kLog2e;
      const float top = fmaxf(m, z);
      const float w0 = exp2f(m - top), w1 = exp2f(z - top);
      l = l * w0 + w1;
#pragma unroll
      for (int j = 0; j < kN; ++j) acc[j] = fmaf(acc[j], w0, w1 * (v[j] * vs));
      m = top;
    }
  }
  const float inv = n > 0 ? 1.0f / l : 0.0f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int64_t at = (row * p.hq + h) * D + lane * kN + j;
    if (p.o_bf16)
      static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(acc[j] * inv);
    else
      static_cast<float*>(p.o)[at] = acc[j] * inv;
  }
  if (lane == 0) p.lse[row * p.hq + h] = n > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

int64_t kv_attn_workspace(const cp_kv_attn_desc&, int) { return 0; }

cp_status launch_kv_attn(const cp_kv_attn_desc& d, float scale, int64_t, int, cudaStream_t s) {
  AttnParams p{d.cache, d.rows, d.q, d.o, d.lse, d.q_first, d.hq, d.in_dtype == CP_BF16, d.o_dtype == CP_BF16,
               scale, d.kv_pos, d.status};
  const int64_t blocks = (d.rows.n_rows * d.hq + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) {
    set_error("cp_kv_cache_attn: too many rows");
    return CP_ERR_INVALID_ARG;
  }
  if (d.cache.d == 128)
    kv_attn_row_kernel<128><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  else
    kv_attn_row_kernel<64><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "kv_attn_row_kernel launch");
}

}  // namespace cpattn

// Rotary positions with several axes (cp_rope_axes).
//
// The angle of pair i of a token is position * inv_freq[i].  The host turns inv_freq into a 64-bit
// fraction of a turn, u = round(inv_freq / 2 pi * 2^64) mod 2^64; position * u modulo 2^64 is then
// the fraction of a turn exactly, whatever the position, with three 32-bit integer products and no
// fp64 arithmetic (which this part has little of).  Its upper 32 bits, read as a signed number,
// give an angle in [-pi, pi).
#include <cuda_bf16.h>

#include "internal.h"

namespace cpattn {

namespace {

constexpr int kThreads = 256;

struct RopeParams {
  const void* in[4];
  void* out[4];
  int32_t head0[5];  // first head of each tensor among all heads, and their number
  int32_t axis0[5];  // first pair of each axis
  int64_t tokens;
  int32_t n_tensors, n_axes, d, rot, interleaved, inverse;
  const int32_t* positions;
  uint64_t turn[128];
};

// One thread per (token, head, pair or copied pair).
template <class T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  const int half = p.rot / 2, per = p.d / 2;
  const int heads = p.head0[p.n_tensors];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = i / per;
  const int64_t token = row / heads;
  if (token >= p.tokens) return;
  const int pair = static_cast<int>(i - row * per), head = static_cast<int>(row - token * heads);
  int t = 0;
  while (t + 1 < p.n_tensors && head >= p.head0[t + 1]) ++t;
  const int64_t at = (token * (p.head0[t + 1] - p.head0[t]) + (head - p.head0[t])) * p.d;
  const T* x = static_cast<const T*>(p.in[t]) + at;
  T* y = static_cast<T*>(p.out[t]) + at;
  if (pair >= half) {
    y[2 * pair] = x[2 * pair];
    y[2 * pair + 1] = x[2 * pair + 1];
    return;
  }
  int axis = 0;
  while (axis + 1 < p.n_axes && pair >= p.axis0[axis + 1]) ++axis;
  const int64_t pos = p.positions[axis * p.tokens + token];
  const uint64_t turns = static_cast<uint64_t>(pos) * p.turn[pair];
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &s, &c);
  if (p.inverse) s = -s;
  const int ia = p.interleaved ? 2 * pair : pair, ib = p.interleaved ? 2 * pair + 1 : pair + half;
  const float a = static_cast<float>(x[ia]), b = static_cast<float>(x[ib]);
  y[ia] = static_cast<T>(a * c - b * s);
  y[ib] = static_cast<T>(a * s + b * c);
}

}  // namespace

cp_status launch_rope(const RopeArgs& a, cudaStream_t s) {
  RopeParams p{};
  for (int t = 0; t < a.n_tensors; ++t) {
    p.in[t] = a.in[t];
    p.out[t] = a.out[t];
    p.head0[t + 1] = p.head0[t] + a.heads[t];
  }
  for (int x = 0; x < a.n_axes; ++x) p.axis0[x + 1] = p.axis0[x] + a.sections[x];
  p.tokens = a.tokens;
  p.n_tensors = a.n_tensors;
  p.n_axes = a.n_axes;
  p.d = a.d;
  p.rot = a.rot;
  p.interleaved = a.interleaved;
  p.inverse = a.inverse;
  p.positions = a.positions;
  for (int i = 0; i < a.rot / 2; ++i) p.turn[i] = a.turn[i];
  const int64_t n = a.tokens * p.head0[a.n_tensors] * (a.d / 2);
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) {
    set_error("cp_rope_axes: too many elements");
    return CP_ERR_INVALID_ARG;
  }
  if (a.bf16)
    rope_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  else
    rope_kernel<float><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "rope_kernel launch");
}

}  // namespace cpattn

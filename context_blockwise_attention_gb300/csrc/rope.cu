// Rotary positions with several axes (cp_rope_axes).
//
// The angle of pair i of a token is position * inv_freq[i].  The host turns inv_freq into a 64-bit
// fraction of a turn, u = inv_freq / 2 pi * 2^64 mod 2^64 less at most 2; position * u modulo 2^64 is then
// the fraction of a turn to 2^-32, whatever the position, with three 32-bit integer products and no
// fp64 arithmetic (which this part has little of).  Its upper 32 bits, read as a signed number,
// give an angle in [-pi, pi).
//
// Bound by memory: every number is read and written once.  32768 tokens x 40 heads x 128 bf16 (671 MB):
// 109 us, 6.2 TB/s; one thread a pair with its own cosine took 787.
// A block takes a few tokens, makes their cosines and sines once in shared memory (a thread makes those
// of one pair, and uses 8 for each 16 numbers), and turns all heads of all tensors with 16-byte
// accesses; a thread's first loads are under way while the table is made.  Where the heads are few the table is
// what counts: 20 k tokens of 3 x 128 bf16 9.8 us, with other pairs in every turn of a thread 16.9.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kThreads = 256;

struct RopeParams {
  const void* in[4];
  void* out[4];
  int32_t head0[5];  // first head of each tensor among all heads, and their number
  int32_t axis0[5];  // first pair of each axis
  int64_t tokens;
  int32_t n_tensors, n_axes, rot, inverse;
  int32_t words;      // 16-byte words of a head
  int32_t copies;     // groups of 8 numbers behind rot that are copied
  int32_t per_block;  // tokens of a block
  float inv_heads;
  const int32_t* positions;
  uint64_t turn[128];
};

// 8 pairs, or 16 numbers to copy, as 16-byte words: kW words of the first and of the second half.
template <class T>
constexpr int kW = 8 * static_cast<int>(sizeof(T)) / 16;

__device__ __forceinline__ void unpack(const uint4 (&v)[1], float (&x)[8]) {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4 (&v)[2], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(v[i].x), x[4 * i + 1] = __uint_as_float(v[i].y);
    x[4 * i + 2] = __uint_as_float(v[i].z), x[4 * i + 3] = __uint_as_float(v[i].w);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void pack(const float (&x)[8], uint4 (&v)[1]) {
  v[0] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void pack(const float (&x)[8], uint4 (&v)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                      __float_as_uint(x[4 * i + 3]));
}

// Units of a head: rot / 16 groups of 8 pairs, then (d - rot) / 8 groups of 8 numbers to copy (none
// in place).  Thread (unit, row): rows are the heads of the block's tokens, one token after the other.
template <class T, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kWords = kW<T>;
  extern __shared__ float4 table[];  // [token][4][rot / 16]: two (cos, sin) each
  const int half = p.rot / 2, groups = half / 8, units = groups + p.copies;
  const int heads = p.head0[p.n_tensors];
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * p.per_block;
  const int here = static_cast<int>(p.tokens - token0 < p.per_block ? p.tokens - token0 : p.per_block);
  const int tid = threadIdx.x;
  const int unit = tid % units, step = kThreads / units;
  int r = tid / units;
  const int rows = tid < step * units ? here * heads : 0;  // threads beyond the last whole row rest
  // words of the unit's two parts, in 16-byte words from the row's start
  int first, second;
  if (unit >= groups) {
    first = (p.rot + (unit - groups) * 8) * static_cast<int>(sizeof(T)) / 16;
    second = first;
  } else if (INTER) {
    first = unit * 2 * kWords;
    second = first + kWords;
  } else {
    first = unit * kWords;
    second = first + groups * kWords;
  }

  uint4 a[kWords], b[kWords];
  int token = 0, next_token = 0;
  uint4* to = nullptr;
  auto load = [&](int row, uint4 (&u)[kWords], uint4 (&v)[kWords], int& tok, uint4*& dst) {
    tok = static_cast<int>((static_cast<float>(row) + 0.5f) * p.inv_heads);  // exact: row is below 2^20
    const int head = row - tok * heads;
    int t = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i) t += i < p.n_tensors && head >= p.head0[i];
    const int64_t at = ((token0 + tok) * (p.head0[t + 1] - p.head0[t]) + (head - p.head0[t])) * p.words;
    const uint4* src = static_cast<const uint4*>(p.in[t]) + at;
    dst = static_cast<uint4*>(p.out[t]) + at;
#pragma unroll
    for (int w = 0; w < kWords; ++w) u[w] = __ldcs(src + first + w);
    if (unit < groups) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) v[w] = __ldcs(src + second + w);
    }
  };
  ptx::wait_dependencies();
  if (r < rows) load(r, a, b, token, to);
  const int side = kThreads / half;  // tokens side by side, a thread with one pair of them
  if (tid < side * half) {
    const int t0 = tid / half, pair = tid - t0 * half;
    int axis = 0;
#pragma unroll
    for (int x = 1; x < 4; ++x) axis += x < p.n_axes && pair >= p.axis0[x];
    const int32_t* const pos = p.positions + axis * p.tokens + token0;
    const uint64_t per_turn = p.turn[pair];
    float2* const at = reinterpret_cast<float2*>(table) + (pair & 7) / 2 * groups * 2 + pair / 8 * 2 + (pair & 1);
#pragma unroll 4
    for (int t = t0; t < here; t += side) {
      const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(__ldg(pos + t))) * per_turn;
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &s, &c);
      at[t * 8 * groups] = make_float2(c, p.inverse ? -s : s);
    }
  }
  __syncthreads();
  while (r < rows) {
    uint4 na[kWords], nb[kWords];
    uint4* next_to = nullptr;
    const int next = r + step;
    if (next < rows) load(next, na, nb, next_token, next_to);
    if (unit < groups) {
      float x[8], y[8];
      unpack(a, x);
      unpack(b, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 cs = table[(token * 4 + k) * groups + unit];  // pairs 2 k and 2 k + 1 of the unit
        // element of each pair: neighbours, or the same place of the two halves
        auto turn = [](float& u, float& v, float c, float s) {
          const float t = u * c - v * s;
          v = u * s + v * c;
          u = t;
        };
        if (INTER) {
          if (k < 2) {
            turn(x[4 * k], x[4 * k + 1], cs.x, cs.y);
            turn(x[4 * k + 2], x[4 * k + 3], cs.z, cs.w);
          } else {
            turn(y[4 * (k - 2)], y[4 * (k - 2) + 1], cs.x, cs.y);
            turn(y[4 * (k - 2) + 2], y[4 * (k - 2) + 3], cs.z, cs.w);
          }
        } else {
          turn(x[2 * k], y[2 * k], cs.x, cs.y);
          turn(x[2 * k + 1], y[2 * k + 1], cs.z, cs.w);
        }
      }
      pack(x, a);
      pack(y, b);
#pragma unroll
      for (int w = 0; w < kWords; ++w) __stcs(to + second + w, b[w]);
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) __stcs(to + first + w, a[w]);
    r = next;
    token = next_token;
    to = next_to;
#pragma unroll
    for (int w = 0; w < kWords; ++w) a[w] = na[w], b[w] = nb[w];
  }
}

}  // namespace

cp_status launch_rope(const RopeArgs& a, int num_sms, cudaStream_t s) {
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
  p.rot = a.rot;
  p.inverse = a.inverse;
  p.positions = a.positions;
  for (int i = 0; i < a.rot / 2; ++i) p.turn[i] = a.turn[i];
  bool in_place = true;
  for (int t = 0; t < a.n_tensors; ++t) in_place = in_place && a.in[t] == a.out[t];
  const int heads = p.head0[a.n_tensors];
  p.words = a.d * (a.bf16 ? 2 : 4) / 16;
  p.copies = in_place ? 0 : (a.d - a.rot) / 8;
  p.inv_heads = 1.0f / static_cast<float>(heads);
  // Tokens of a block: about four rows a thread, but no fewer than four blocks an SM, and 16 KB of table.
  const int units = a.rot / 16 + p.copies, rows = kThreads / units;
  int64_t per = (4 * rows + heads - 1) / heads;
  const int64_t spread = a.tokens / (4 * num_sms);
  if (per > spread) per = spread;
  if (per > 16384 / (4 * a.rot)) per = 16384 / (4 * a.rot);
  if (per < 1) per = 1;
  p.per_block = static_cast<int32_t>(per);
  const int64_t blocks = (a.tokens + per - 1) / per;
  if (blocks > 0x7fffffff) {
    set_error("cp_rope_axes: too many tokens");
    return CP_ERR_INVALID_ARG;
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(per) * a.rot * 4;
  const cudaError_t e =
      a.bf16 ? (a.interleaved ? cudaLaunchKernelEx(&cfg, rope_kernel<__nv_bfloat16, true>, p)
                              : cudaLaunchKernelEx(&cfg, rope_kernel<__nv_bfloat16, false>, p))
             : (a.interleaved ? cudaLaunchKernelEx(&cfg, rope_kernel<float, true>, p)
                              : cudaLaunchKernelEx(&cfg, rope_kernel<float, false>, p));
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "rope_kernel launch");
}

}  // namespace cpattn

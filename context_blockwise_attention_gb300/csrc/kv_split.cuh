// What the attention kernels over the paged caches share: the arguments, the numbering of the work, its
// equal shares, and the reading and writing of rows.  An item is a (sequence, KV head, block of RT query
// rows); its unit of work is a granule of 4096 / D keys.
#pragma once

#include "internal.h"
#include "kv_common.cuh"
#include "ptx.cuh"

namespace cpattn {
namespace kvattn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kFull = 0xffffffffu;

template <int D>
constexpr int kKeysOf = 4096 / D;  // keys of a granule

struct Params {
  const float* scale[2];   // 8-bit cache: scales of K, V
  const uint8_t* tile[2];  // 4-bit cache: rows of K, V
  cp_kv_rows rows;
  int64_t n_pages;
  const void* q;
  void* o;
  float* lse;
  const int32_t* q_first;
  int32_t hq, hkv, group, page, page_log2;
  int32_t q_bf16, o_bf16, stall;
  float scale_log2;
  cp_posmap kv_pos;
  int32_t* status;
  int64_t timeout_ns;
  int64_t few;     // workers that may have less than four numbers
  int32_t setup;   // what an item costs besides its granules, in granules
  int32_t cluster; // SOLO 2: blocks of an item, 2 to 8
  float* part_o;   // [workers][2][RT][D]
  float2* part_ml; // [workers][2][RT]: m (base 2), l
  float* aside;    // [workers][RT][D]: accumulators put aside
};

// What a sequence asks for.
struct Seq {
  int64_t r0;      // first row
  int64_t pos0;    // position of its first row
  int32_t rows;
  int32_t tokens;  // cached tokens; of those behind the page table one, which has a bad page, stands for all
  int32_t keys;    // tokens that its last row sees
  int32_t gpi;     // granules of an item
  int32_t blocks;  // blocks of RT query rows; 0 where no row sees a token
  bool over;       // more tokens than the table has pages for
};

// Number of tokens that a row at position `pos` sees: token j stands at base + stride * j.
__device__ __forceinline__ int32_t visible(const Params& p, int32_t tokens, int64_t pos) {
  if (p.q_first == nullptr) return tokens;
  const int64_t off = pos - p.kv_pos.base;  // below 2^32
  if (off < 0) return 0;
  const uint32_t n = static_cast<uint32_t>(off) / static_cast<uint32_t>(p.kv_pos.stride);
  return n < static_cast<uint32_t>(tokens) ? static_cast<int32_t>(n) + 1 : tokens;
}

template <int D, int RT>
__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  Seq s;
  s.r0 = kv::row_at(p.rows, b);
  const int64_t r1 = kv::row_at(p.rows, b + 1);
  s.rows = r1 > s.r0 ? static_cast<int32_t>(r1 - s.r0) : 0;
  int64_t t = __ldg(p.rows.tokens + b);
  const int64_t room = static_cast<int64_t>(p.rows.max_pages) << p.page_log2;
  s.over = t > room;
  if (s.over) t = room + 1;
  s.tokens = t < 0 ? 0 : static_cast<int32_t>(t);
  s.pos0 = p.q_first != nullptr ? __ldg(p.q_first + b) : 0;
  s.keys = s.rows > 0 ? visible(p, s.tokens, s.pos0 + s.rows - 1) : 0;
  s.gpi = (s.keys + kKeysOf<D> - 1) / kKeysOf<D>;
  s.blocks = s.keys > 0 ? (s.rows * p.group + RT - 1) / RT : 0;
  return s;
}
__device__ __forceinline__ int64_t numbers(const Params& p, const Seq& s) {
  return static_cast<int64_t>(s.blocks) * p.hkv * (s.gpi + p.setup);
}

// Shares of W numbers among n workers: worker w has [share(w), share(w + 1)).
__device__ __forceinline__ int64_t share(int64_t W, int64_t n, int64_t w) { return W * w / n; }
__device__ __forceinline__ int64_t worker_of(int64_t W, int64_t n, int64_t x) { return ((x + 1) * n - 1) / W; }
// Of `most` workers those that get a share: where an item would have more than some 128 partials, workers
// of at least four numbers (1 x 131072 / 40000 / 4096 tokens, 8/1, 4/2, 8/1 heads: 22.7 / 16.7 / 9.1 us; always as
// many as there are: 29.7 / 19.4 / 9.0; always four numbers: 22.8 / 16.7 / 12.8).
__device__ __forceinline__ int64_t workers(const Params& p, int64_t W, int64_t most) {
  const int64_t few = W < p.few ? W : p.few, some = W / 4 > few ? W / 4 : few;
  return some < most ? some : most;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t to_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 from_f16x2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Four consecutive query elements as fp32.
__device__ __forceinline__ void load4(const Params& p, int64_t at, float (&x)[4]) {
  if (p.q_bf16) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + at));
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
    const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
}

__device__ __forceinline__ void store_row4(const Params& p, int64_t at, float a, float b, float c, float d) {
  if (p.o_bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    uint2 pk;
    pk.x = *reinterpret_cast<const uint32_t*>(&x);
    pk.y = *reinterpret_cast<const uint32_t*>(&y);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at) = pk;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) = make_float4(a, b, c, d);
  }
}

// A lane's consecutive part of a row.
__device__ __forceinline__ void store_lane(const Params& p, int64_t at, const float (&x)[4]) {
  store_row4(p, at, x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_lane(const Params& p, int64_t at, const float (&x)[2]) {
  if (p.o_bf16)
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.o) + at) = __floats2bfloat162_rn(x[0], x[1]);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at) = make_float2(x[0], x[1]);
}

// Sums of of(b) before each sequence b, in shared memory: plan[0 .. n].
template <int THREADS, class F>
__device__ __forceinline__ void make_plan_of(int n, int64_t* plan, int64_t* scratch, F of) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t before = 0;
  for (int base = 0; base < n; base += THREADS) {
    const int b = base + tid;
    int64_t x = b < n ? of(b) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t add = before, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) add += scratch[i];
      all += scratch[i];
    }
    if (b < n) plan[b + 1] = add + x;
    before += all;
    __syncthreads();
  }
  if (tid == 0) plan[0] = 0;
  __syncthreads();
}

// Numbers before each sequence, in shared memory: plan[0 .. n_seqs].
template <int D, int RT, int THREADS>
__device__ __forceinline__ void make_plan(const Params& p, int64_t* plan, int64_t* scratch) {
  make_plan_of<THREADS>(p.rows.n_seqs, plan, scratch, [&](int b) {
    const Seq s = seq_of<D, RT>(p, b);
    if (s.over && s.rows > 0 && blockIdx.x == 0) kv::report(p.status, kv::kSiteTokens);
    return numbers(p, s);
  });
}

// A place in the numbering of granules.
struct Cursor {
  int b, head, block, g;
  int gpi, blocks;
};

// Moves to the first sequence behind c.b that has items.
template <int D, int RT>
__device__ __forceinline__ void next_seq(const Params& p, Cursor& c, Seq& s) {
  do {
    ++c.b;
    if (c.b >= p.rows.n_seqs) return;
    s = seq_of<D, RT>(p, c.b);
  } while (s.blocks == 0);
  c.head = c.block = c.g = 0;
  c.gpi = s.gpi;
  c.blocks = s.blocks;
}

// How a call is answered: by the query rows that a sequence has on average.
struct Plan {
  int nt, qp, pp;
  int rows;      // RT
  int warps;     // of a block
  bool solo;     // one block or cluster of blocks per (sequence, KV head), no workspace
  int cluster;
  double most;
  int64_t grid;
  int64_t ml_off, o_off, aside_off, bytes;
};

// Sums the partials of the items that several workers shared, and answers the rows that see nothing.  Launched behind
// the attention kernel of `workers` workers, as its programmatic dependent.  RT is 8, 16 or, at
// D = 128, 24.
template <int D, int RT>
cp_status launch_sum(const Params& p, int64_t workers, int64_t items, int num_sms, cudaStream_t s);

}  // namespace kvattn
}  // namespace cpattn

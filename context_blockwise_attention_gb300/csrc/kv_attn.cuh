// Attention of a batch's new tokens over the paged 8-bit cache (cp_kv_cache_attn): the kernels and their
// launches.  kv_attn.cu chooses among them; kv_attn_d64.cu and kv_attn_d128.cu compile them.
//
// Per (sequence, KV head) the g = hq / hkv query heads of the sequence's rows are one block of
// query rows that share keys and values:
//   s_ij = log2 e * scale * ks(page of j) * (q_i . k8_j),  p_ij = 2^(s_ij - m_i),
//   O_i = sum_j p_ij vs(page of j) v8_j / l_i,             LSE_i = ln 2 (m_i + log2 l_i),  l_i = sum_j p_ij.
// Bound: every cached byte is read once for 2 g rows' worth of products per byte, so it is memory
// bound for up to a few dozen rows; the design is about keeping loads in flight and splitting the
// keys evenly, not about the tensor rate.
//
// Work split.  The unit is a granule of 4096 / D keys (8 KB of cache) of one item (sequence, KV head,
// block of RT query rows); granules are numbered item after item, each item beginning with kSetup
// numbers that stand for the time its start and end take.  Every warp of the grid is a worker on its
// own, with an equal share of consecutive numbers, whatever the sequences' lengths: no barrier
// between warps, and a worker's copies run ahead across item borders.  An item that lies within one
// share is finished there; of the others each worker leaves a partial (O unnormalised, m, l), at most
// two per worker (the item its share begins inside of and the one it ends in), and a second kernel,
// launched as a programmatic dependent, combines them in the order of the workers.  That kernel also
// answers the rows of sequences without visible tokens, which are no items.
//
// Few short rows (SOLO): one block, or a cluster of up to 8, per (sequence, KV head); their warps share the
// granules, and the partials meet in shared memory, a block's first and then the cluster's: one launch and no
// workspace.
//
// Products.  mma.sync m16n8k16 with f16 operands: e4m3 -> f16 is exact and one instruction for two
// values, and the 128-row tiles of tcgen05 would be mostly empty with 8 to 32 query rows.  Both
// products are taken transposed, S^T = K Q^T and O^T = V^T P^T: keys and head dimensions fill the 16
// rows of an operand tile, query rows its 8 columns, so that 8 rows waste nothing and O takes
// D / 4 registers; P^T gets from the accumulator's layout into the operand's by one 8x8 transpose
// for 8 keys.  The orders of keys and dimensions inside the products are free as long as both
// operands agree; they are chosen so that every lane reads 16 consecutive bytes of a key or value
// row, without bank conflicts under the 128-byte swizzle that the copies apply.
//
// Precision.  A query row is scaled by a power of two to at most 2^15; as f16 a bf16 row is then
// exact (over 2^28 of range), an fp32 row is split into a high and a low part, 22 bits.  An operand of P is a
// contribution, p_ij vs, in one f16 part for a bf16 output (off by 2^-11 at most, against the output's 2^-8) and in
// two for an fp32 one.  f16 ends at 2^-24, so the row's largest contribution is held at 2^15 to 2^16: m_i is
//   max_j (s_ij + log2 vs(page of j)) - base,
// a whole number, with one `base` for an item's pages, and p_ij vs 2^(15 - base) is the operand.  So a contribution
// is off by 2^-40 of the row's largest besides, which only columns show in which the heavy tokens hold zeros; pages
// whose scales differ by 2^40 lose nothing to one another; and what a row does not see has no part in its bits.  (With
// the largest scale at 2^15 instead, a light or unseen token of a page 2^40 larger left nothing of the others.)  Sums,
// maxima and the accumulators are fp32.
//
// Measured (GB300, calls back to back in a graph): 64 x 256-8192 tokens, 32/8 heads, D = 128, bf16: 85-86 us
// for 471 MB, 5.5 TB/s; 8 x 90000-131072, 64/8, D = 64, fp32 partials: 147-149 us for 910 MB, 6.1 TB/s (copy:
// 6.8); 16 x 2-6 rows over 1000-20000 tokens, 32/8, D = 128: 104 us; one token over 1000, 32/8, D = 128: 8.2 us; 4 x
// 2000: 9.3 us (tables for 8192 tokens at most).  What is left of the long calls is 6 us until the first data are there
// for all, SMs that end up to a tenth later than others, and 4 us of the second kernel.
#pragma once

#include "internal.h"
#include "kv_common.cuh"
#include "ptx.cuh"
#include "sync.cuh"

namespace cpattn {
namespace kvattn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kPExp = 15;            // P operands are below 2^(kPExp + kTop) = 65490 and f16's largest is 65504
constexpr float kTop = 0.999f;       // largest s + log2 vs - base - m
constexpr float kNear = 40.0f;       // largest |log2 vs - base| but for base = kFarBase
constexpr int kFarBase = 40;
constexpr float kNoBase = -10000.0f;
constexpr int kSetup = 1;            // what an item costs besides its granules
constexpr unsigned kFull = 0xffffffffu;

template <int D>
constexpr int kKeysOf = 4096 / D;  // keys of a granule

// QP, PP: f16 parts of a query element and of a weight.  NT: tiles of 8 query rows.
template <int D, int NT, int QP, int PP>
struct Shape {
  // More warps hide more latency; registers (O takes NT D / 4) and shared memory bound their number.
  static constexpr bool kHeavy = NT * D >= 256 || NT * QP >= 4;
  static constexpr int kWarps = kHeavy ? 8 : 12;
  static constexpr int kRows = NT * 8;  // RT
  // The tensor cores' fp32 sums are truncated, an error that grows with the length of a sum: 5e-6 of O after
  // 64 granules of rows over 1e5 tokens, 1e-6 after 8.  So the accumulators are added to others every
  // kFlush granules: in registers where there are some left (kHold), else in the workspace (every 8
  // granules that took 5 %).  bf16 outputs can wait longer.
  static constexpr bool kHold = PP == 2 && D == 64 && NT == 1;
  static constexpr int kFlush = PP == 1 ? 64 : kHold ? 4 : D == 128 ? 16 : 8;
  static constexpr int kKeys = kKeysOf<D>;
  static constexpr int kSteps = kKeys / 16;          // steps of 16 keys
  static constexpr int kHalf = kKeys * D;            // bytes of K (or V) of a granule
  static constexpr int kStage = 2 * kHalf;
  static constexpr bool kQSmem = D == 128 && NT * QP >= 4;  // query operands in shared memory
  static constexpr int kStages = kHeavy && !kQSmem ? 3 : 2;
  static constexpr int kQBytes = kQSmem ? NT * QP * (D / 16) * 256 : 0;
  static constexpr int kWarpBytes = kStages * kStage + kQBytes;
  // behind the warps' parts (1024-byte aligned for the swizzle): scales, barriers, control, plan
  static constexpr int kScaleOff = kWarps * kWarpBytes;               // [warp][stage][8] fp32
  static constexpr int kBarOff = kScaleOff + kWarps * kStages * 32;   // [warp][stage] + stall
  static constexpr int kCtlOff = kBarOff + (kWarps * kStages + 1) * 8;
  static constexpr int kScanOff = (kCtlOff + 8 + 15) / 16 * 16;       // [warp] 8 bytes
  static constexpr int kPlanOff = kScanOff + 16 * 8;
};

struct Params {
  const float* scale[2];  // K, V
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
  return static_cast<int64_t>(s.blocks) * p.hkv * (s.gpi + kSetup);
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

// Numbers before each sequence, in shared memory: plan[0 .. n_seqs].
template <int D, int RT, int THREADS>
__device__ __forceinline__ void make_plan(const Params& p, int64_t* plan, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.rows.n_seqs;
  int64_t before = 0;
  for (int base = 0; base < n; base += THREADS) {
    const int b = base + tid;
    int64_t x = 0;
    if (b < n) {
      const Seq s = seq_of<D, RT>(p, b);
      x = numbers(p, s);
      if (s.over && s.rows > 0 && blockIdx.x == 0) kv::report(p.status, kv::kSiteTokens);
    }
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

// SOLO: 0 split, 1 one block an item, 2 a cluster of p.cluster blocks an item.  Three kernels, as the code of one
// in another's cost it 2 to 7 %.
template <int D, int NT, int QP, int PP, int SOLO>
__global__ void __launch_bounds__(Shape<D, NT, QP, PP>::kWarps * 32, 1)
    kv_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v) {
  using S = Shape<D, NT, QP, PP>;
  constexpr int RT = S::kRows;
  constexpr int kMt = D / 16;  // 16-row tiles of O^T; also steps of 16 dimensions of S
  constexpr int kCols = D / 8; // columns of O that a lane holds, for two query rows
  constexpr int kSt = S::kStages, kSteps = S::kSteps, kKeys = S::kKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  int64_t* const plan = reinterpret_cast<int64_t*>(smem + S::kPlanOff);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + S::kCtlOff);
  const uint32_t base = ptx::smem_u32(smem);
  const uint32_t ring = base + warp * S::kWarpBytes;
  const uint32_t q_smem = ring + kSt * S::kStage;
  const uint32_t scales = base + S::kScaleOff + warp * kSt * 32;
  const uint32_t bars = base + S::kBarOff + warp * kSt * 8;
  const uint32_t stall_bar = base + S::kBarOff + S::kWarps * kSt * 8;

  if (lane == 0) {
    // one arrival for the copies' bytes, and one for each lane that copies a scale
    for (int i = 0; i < kSt; ++i) ptx::mbar_init(bars + i * 8, 1 + 2 * kSteps);
    if (warp == 0) {
      ptx::mbar_init(stall_bar, 1);
      *abort_flag = 0;
      ptx::tma_prefetch_desc(&map_k);
      ptx::tma_prefetch_desc(&map_v);
    }
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  ptx::wait_dependencies();  // launched early: what was in the stream before is complete from here on
  const int n_seqs = p.rows.n_seqs;
  const sync::Ctl ctl{abort_flag, p.status, p.timeout_ns};
  const int64_t worker = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;  // neighbours on different SMs
  Cursor c;  // where the products are
  Seq seq;
  int64_t left;  // numbers of the share from the cursor on
  bool inside;   // the share begins inside of an item
  const bool stalled = p.stall && blockIdx.x == 0 && warp == 0;  // test only
  // SOLO: rank of the block among those of its item, and the warp and number of warps among all of them
  const int cluster = SOLO == 2 ? p.cluster : 1;
  const int rank = SOLO == 2 ? blockIdx.x % cluster : 0;
  const int solo_warp = rank * S::kWarps + warp, solo_warps = cluster * S::kWarps;
  if constexpr (SOLO) {
    const int item = blockIdx.x / cluster;
    c.b = item / p.hkv;
    c.head = item - c.b * p.hkv;
    seq = seq_of<D, RT>(p, c.b);
    if (seq.over && seq.rows > 0 && tid == 0) kv::report(p.status, kv::kSiteTokens);
    if (seq.blocks == 0) {  // nothing to see
      for (int rho = solo_warp; rho < seq.rows * p.group; rho += solo_warps) {
        const int t = rho / p.group;
        const int64_t out = (seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group);
        const float zero[D / 32] = {};
        store_lane(p, out * D + lane * (D / 32), zero);
        if (lane == 0) p.lse[out] = -INFINITY;
      }
      return;
    }
    __syncthreads();  // the abort flag is set up
    c.block = 0;
    c.gpi = seq.gpi;
    c.blocks = seq.blocks;
    c.g = seq.gpi * solo_warp / solo_warps;
    left = seq.gpi * (solo_warp + 1) / solo_warps - c.g;
    inside = false;
  } else {
    make_plan<D, RT, S::kWarps * 32>(p, plan, reinterpret_cast<int64_t*>(smem + S::kScanOff));
    ptx::launch_dependents();
    if (stalled) {
      sync::wait_warp(stall_bar, 0, ctl, kv::kSiteWait);
      return;
    }
    const int64_t W = plan[n_seqs];
    const int64_t n_workers = workers(p, W, static_cast<int64_t>(gridDim.x) * S::kWarps);
    if (worker >= n_workers) return;
    const int64_t lo = share(W, n_workers, worker), hi = share(W, n_workers, worker + 1);
    left = hi - lo;
    int a = 0, z = n_seqs - 1;  // the last sequence whose numbers begin at or before lo
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (plan[mid] <= lo) a = mid;
      else z = mid - 1;
    }
    c.b = a;
    seq = seq_of<D, RT>(p, a);
    const int64_t off = lo - plan[a];
    const int64_t item = off / (seq.gpi + kSetup);
    const int at = static_cast<int>(off - item * (seq.gpi + kSetup));
    inside = at >= kSetup;
    c.g = inside ? at - kSetup : 0;
    if (!inside) left -= kSetup - at;
    c.head = static_cast<int>(item / seq.blocks);
    c.block = static_cast<int>(item - static_cast<int64_t>(c.head) * seq.blocks);
    c.gpi = seq.gpi;
    c.blocks = seq.blocks;
    if (left <= 0) return;
  }
  bool ok = true;
  if (stalled) {  // the block's other warps still meet it
    ok = sync::wait_warp(stall_bar, 0, ctl, kv::kSiteWait);
    left = 0;
  }
  const int g_first = c.g, solo_left = static_cast<int>(left);  // of a block of rows, where SOLO
  Cursor f = c;  // where the copies are
  int64_t to_issue = left;
  int f_keys = seq.keys;
  int window = -32;        // lane i holds page window + i of sequence f.b, -1 behind its keys
  int pages = -1;

  auto page_of = [&](int ord) -> int {
    if (static_cast<unsigned>(ord - window) >= 32u) {
      window = ord;
      // entries that hold no token are the caller's to change at any time: they are not read
      pages = -1;
      if ((ord + lane) << p.page_log2 < f_keys)
        pages = static_cast<int>(kv::page_at(p.rows, p.n_pages, f.b, ord + lane));
    }
    return __shfl_sync(kFull, pages, ord - window);
  };
  // Starts the copies of one page's part of K and V (`lines` lines of the maps from `page` on).
  auto copy = [&](int page, int slot, uint32_t dst, uint32_t bar) {
    const int row = (page * p.hkv + f.head) * p.page + slot;  // below 2^31: checked on the host
    const int line = D == 128 ? row : row >> 1;
    ptx::tma_load_2d(dst, &map_k, 0, line, bar);
    ptx::tma_load_2d(dst + S::kHalf, &map_v, 0, line, bar);
  };
  // Copies the scale of K (even lane) or V (odd lane), or stands in for it: where there is no
  // token the smallest scale, for a bad page NaN, which reaches the rows that see it.
  auto copy_scale = [&](int page, bool need, uint32_t to) {
    if (page >= 0) ptx::cp_async4(to, p.scale[lane & 1] + (page * p.hkv + f.head));
    else asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(need ? 0x7fffffffu : 0x1f800000u) : "memory");
  };

  // Starts the copies of the next granule into stage `st`.
  auto issue = [&](int st) {
    const uint32_t bar = bars + st * 8, dst = ring + st * S::kStage;
    const int key0 = f.g * kKeys;
    const int mine = key0 + (lane >> 1) * 16;  // lane 2 i + w copies the scale of step i of K (w = 0) or V (w = 1)
    int my_page = -1;
    bool bad = false;
    if (p.page >= kKeys) {
      const int page = page_of(key0 >> p.page_log2);
      bad = page < 0;
      my_page = page;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(bar, bad ? 0 : S::kStage);
        if (!bad) copy(page, key0 & (p.page - 1), dst, bar);
      }
    } else {  // several pages, as far as there are tokens
      const int part = p.page * D;
      uint32_t tx = 0;
      int page[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int k = key0 + i * p.page;
        page[i] = -1;
        if (i * p.page < kKeys && k < f_keys) {
          page[i] = page_of(k >> p.page_log2);
          if (page[i] >= 0) tx += 2 * part;
          else bad = true;
          if (mine >= k && mine < k + p.page) my_page = page[i];
        }
      }
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(bar, tx);
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          if (page[i] >= 0) copy(page[i], 0, dst + i * part, bar);
      }
    }
    if (lane < 2 * kSteps) {
      copy_scale(my_page, mine < f_keys, scales + st * 32 + lane * 4);
      ptx::cp_async_arrive(bar);
    }
    if (bad && lane == 0) kv::report(p.status, kv::kSitePage);
    --to_issue;
    if (++f.g == f.gpi && to_issue > kSetup) {
      to_issue -= kSetup;
      f.g = 0;
      if (++f.block == f.blocks) {
        f.block = 0;
        if (++f.head == p.hkv) {
          Seq s{};
          next_seq<D, RT>(p, f, s);
          f_keys = s.keys;
          window = -32;
        }
      }
    } else if (f.g == f.gpi) {
      to_issue = 0;
    }
  };

  // lane's offsets inside a stage.  128-byte lines; 16-byte chunk x of line y sits at x ^ (y & 7).
  // A step of 16 keys has two groups u = 0, 1 of 8, group u being rows 8 u .. 8 u + 7 of the operand.
  // D = 128: a line is a key; row c of group u is key 8 u + c.  Lane (gid, tig) reads dimensions
  //   32 tig .. + 31 of key c = gid, and dimensions 16 gid .. + 15 of the values of c = 2 tig, 2 tig + 1.
  // D = 64: a line is two keys; row c of group u is key 4 (c >> 1) + 2 u + (c & 1), so that the four
  //   values of a lane, 4 tig .. 4 tig + 3, are two lines that no other tig shares a bank with.
  uint32_t k_off[2], v_off[4];
  if (D == 128) {
#pragma unroll
    for (int j = 0; j < 2; ++j) k_off[j] = gid * 128 + (((2 * tig + j) ^ gid) << 4);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int c0 = 2 * tig + (x & 1);
      v_off[x] = S::kHalf + (c0 + 8 * (x >> 1)) * 128 + ((gid ^ c0) << 4);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int line = 2 * (gid >> 1) + u;
      k_off[u] = line * 128 + ((((gid & 1) * 4 + tig) ^ line) << 4);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int line = 2 * tig + (x >> 1);
      v_off[x] = S::kHalf + line * 128 + ((((x & 1) * 4 + (gid >> 1)) ^ line) << 4) + (gid & 1) * 8;
    }
  }
  // key of row c of group u in a step
  auto key_at = [](int u, int c0) { return D == 128 ? 8 * u + c0 : 4 * (c0 >> 1) + 2 * u + (c0 & 1); };

  uint32_t qf[S::kQSmem ? 1 : NT * QP][S::kQSmem ? 1 : kMt][2];
  // of the lane's two query rows 2 tig, 2 tig + 1 in each tile
  float fac[NT][2], m[NT][2], l[NT][2];
  int lim[NT][2];
  float acc[NT][kMt][4];
  float b_off = kNoBase;  // -127 - base, a whole number
  float b_unit = 0.0f;    // 2^(kPExp - base)
  bool second = false;    // the granule at hand wants a second pass, see granule
  int lim_min = 0, lim_max = 0;
  int live = NT;         // tiles that have rows
  int row_q = 0;         // first query row (token row * group + head in group) of the block
  float* const aside = p.aside + worker * (RT * D);
  float m_aside[NT][2] = {};  // what the values put aside refer to
  bool flushed = false;
  int since = 0;         // granules since then
  constexpr bool kHold = S::kHold;
  float held[kHold ? kMt : 1][4];  // of the one tile

  auto begin_item = [&]() {
    row_q = c.block * RT;
    const int n_rows = seq.rows * p.group;
    live = min(NT, (n_rows - row_q + 7) / 8);
    int lmin = 0x7fffffff, lmax = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // the lane's part of query row gid of the tile
      const int rho = row_q + n * 8 + gid;
      const bool live = rho < n_rows;
      const int t = live ? rho / p.group : 0;
      const int64_t at = ((seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group)) * D + tig * (D / 4);
      int lm = live ? visible(p, seq.tokens, seq.pos0 + t) : -1;
      if (live) {
        lmin = min(lmin, lm);
        lmax = max(lmax, lm);
      }
      float x[kMt][4];
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < kMt; ++j) {
        if (live) load4(p, at + j * 4, x[j]);
        else x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[j][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // 2^e <= top < 2^(e + 1) goes to [2^14, 2^15); rows of (almost) zeros keep a finite factor
      const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
      const float up = kv::pow2(14 - e), f = p.scale_log2 * kv::pow2(e - 14);
#pragma unroll
      for (int j = 0; j < kMt; ++j) {
        uint32_t h[2], w[2];
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const float a = x[j][2 * e2] * up, b = x[j][2 * e2 + 1] * up;
          h[e2] = to_f16x2(a, b);
          const float2 back = from_f16x2(h[e2]);
          w[e2] = to_f16x2(a - back.x, b - back.y);
        }
        if constexpr (S::kQSmem) {
          const uint32_t to = q_smem + ((n * QP * kMt + j) * 32 + lane) * 8;
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(h[0]), "r"(h[1]) : "memory");
          if (QP == 2)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to + kMt * 256), "r"(w[0]), "r"(w[1]) : "memory");
        } else {
          qf[n * QP][j][0] = h[0], qf[n * QP][j][1] = h[1];
          if (QP == 2) qf[n * QP + QP - 1][j][0] = w[0], qf[n * QP + QP - 1][j][1] = w[1];
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        fac[n][r] = __shfl_sync(kFull, f, (2 * tig + r) * 4);
        lim[n][r] = __shfl_sync(kFull, lm, (2 * tig + r) * 4);
        m[n][r] = -INFINITY;
        l[n][r] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kMt; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.0f;
    }
    lim_min = __reduce_min_sync(kFull, lmin);
    lim_max = __reduce_max_sync(kFull, lmax);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (lim[n][r] < 0) lim[n][r] = lim_max;  // rows of nobody must not make the tile a masked one
    b_off = kNoBase;
    flushed = false;
    since = 0;
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < kMt; ++j) held[j][0] = held[j][1] = held[j][2] = held[j][3] = 0.0f;
    }
  };

  // Where some row of the block does not see all keys of the granule: values that no row sees count as zero,
  // since 0 * NaN would not vanish, and NaN among values that only some of the rows see go to those rows'
  // accumulators and are taken out.  Rolled up, as a granule's other code has to stay in the instruction cache.
  auto mask_values = [&](uint32_t tile) {
    constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks;  // 16-byte chunks of a key, keys of a pass
    const int key0 = c.g * kKeys;
    auto value_at = [&](int k, int chunk) {  // address of a chunk of key key0 + k
      const int line = D == 128 ? k : k >> 1;
      return tile + S::kHalf + line * 128 + ((((D == 128 ? 0 : (k & 1) * 4) + chunk) ^ (line & 7)) << 4);
    };
    const int first = max(lim_min - key0, 0);  // below kKeys
    bool odd = false;
#pragma unroll 1
    for (int k0 = first & ~(kAtOnce - 1); k0 < kKeys; k0 += kAtOnce) {
      const int k = k0 + lane / kChunks;
      const uint32_t at = value_at(k, lane % kChunks);
      if (key0 + k >= lim_max) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
      } else if (k >= first) {
        const uint4 v = ptx::lds128u(at);
        const uint32_t nan = __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                             __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
        odd |= nan != 0u;
      }
    }
    if (__any_sync(kFull, odd)) {
#pragma unroll 1
      for (int k = first; k < kKeys && key0 + k < lim_max; ++k) {
        const uint32_t at = D == 128 ? value_at(k, gid) : value_at(k, gid >> 1) + (gid & 1) * 8;
        uint32_t v[kCols / 4];
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          const uint2 x = ptx::lds64(at + 8 * i);
          v[2 * i] = x.x, v[2 * i + 1] = x.y;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const uint32_t nan = __vcmpeq4(v[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 4 * i), "r"(v[i] & ~nan) : "memory");
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if ((nan >> (8 * e) & 1u) && key0 + k < lim[n][r])
                  acc[n][2 * i + (e >> 1)][2 * (e & 1) + r] = __int_as_float(0x7fffffff);
        }
      }
    }
    ptx::fence_proxy_async_smem();  // before the next copies into the stage
    __syncwarp();
  };

  // Another base.  A weight p_ij = 2^(s_ij - m_i) is as far from 1 as its page's scale from base, and fp32 holds
  // 2^-126 to 2^127.  With base within 2^40 of all scales the heaviest weight is above 2^-41, far above what is lost.
  // Otherwise base is kFarBase: a cache's scales are 2^-64 to 2^120, so the heaviest is between 2^-81 and 2^105
  // whatever the scales are, and what is lost is below 2^-45 of it.
  auto rebase = [&](int to) {
    const float off = -127.0f - static_cast<float>(to);
    if (b_off != kNoBase) {
      const int by = static_cast<int>(b_off - off);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          m[n][r] -= static_cast<float>(by);
          m_aside[n][r] -= static_cast<float>(by);
          l[n][r] *= kv::pow2(by);
        }
    }
    b_off = off;
    b_unit = kv::pow2(kPExp - to);
  };

  // One granule; masked: some of its keys are not seen by some row.  Masks and tiles without rows are uniform
  // branches and predicates, not variants: with four variants a warp's items of a few granules ran at the
  // speed of the instruction cache (62 x 16 items of some 3 granules, up to 60 rows, D = 64: 86 us, more than half
  // of the stalls; 55 with one path, and 16-row items of 8192 tokens 102 against 106).
  auto granule = [&](int st, bool masked) {
    const uint32_t tile = ring + st * S::kStage;
    const int key0 = c.g * kKeys;
    const bool both = NT == 1 || live > 1;
    auto product = [&](int n, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
      if (n == 0) ptx::mma_f16(d, a, b0, b1);
      else ptx::mma_f16_if(d, a, b0, b1, both);
    };
    float ks[kSteps], vs[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; i += 2) {
      const uint4 v = ptx::lds128u(scales + st * 32 + i * 8);
      ks[i] = __uint_as_float(v.x), vs[i] = __uint_as_float(v.y);
      ks[i + 1] = __uint_as_float(v.z), vs[i + 1] = __uint_as_float(v.w);
    }
    if (masked) {
      mask_values(tile);
      // a value scale that is not finite comes in by the scores, which rows that do not see it leave out
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (!(fabsf(vs[i]) < INFINITY)) ks[i] = __int_as_float(0x7fffffff), vs[i] = 1.0f;
      // steps that no row sees have no part in the choice of base (some row sees the first)
#pragma unroll
      for (int i = 1; i < kSteps; ++i)
        if (key0 + 16 * i >= lim_max) vs[i] = vs[0];
    }
    // log2 of the steps' V scales, rounded up, less base
    auto exponent = [](float x) { return static_cast<int>((__float_as_uint(x) + 0x7fffffu) & 0x7f800000u); };
    float ve[kSteps];
    bool far = false;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      ve[i] = fmaf(static_cast<float>(exponent(vs[i])), 0x1p-23f, b_off);
      far |= fabsf(ve[i]) > kNear;
    }
    unsigned skip = 0u;  // steps that are left out
    if (far) {
      if (b_off == kNoBase) rebase(max((exponent(vs[0]) >> 23) - 127, -64));
      unsigned away = 0u;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        away |= (fabsf(fmaf(static_cast<float>(exponent(vs[i])), 0x1p-23f, b_off)) > kNear ? 1u : 0u) << i;
      // Where some rows do not see the far pages these are taken in a pass of their own, after the others, so that those
      // rows keep their bits: no later key is one that they see.
      if (b_off == -127.0f - kFarBase || away == 0u) {
      } else if (masked && !second) {
        skip = away;
        second = true;
      } else {
        skip = second ? ~away : 0u;
        second = false;
        rebase(kFarBase);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        ve[i] = fmaxf(fmaf(static_cast<float>(exponent(vs[i])), 0x1p-23f, b_off), 63.0f + b_off);
    }
    // S^T: s[n][i][2 u + r] is key key_at(u, gid) of step i for query row 2 tig + r of tile n
    float s[NT][kSteps][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint32_t kw[2][kMt];  // word j of the lane's part of a key: dimensions of step j
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (D == 128) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 v = ptx::lds128u(tile + (2 * i + u) * 1024 + k_off[j]);
            kw[u][4 * j] = v.x, kw[u][4 * j + 1] = v.y, kw[u][4 * j + 2] = v.z, kw[u][4 * j + 3] = v.w;
          }
        } else {
          const uint4 v = ptx::lds128u(tile + i * 1024 + k_off[u]);
          kw[u][0] = v.x, kw[u][1] = v.y, kw[u][2] = v.z, kw[u][3] = v.w;
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][i][0] = s[n][i][1] = s[n][i][2] = s[n][i][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < kMt; ++j) {
        const uint32_t a[4] = {kv::e4m3x2_to_f16x2(kw[0][j]), kv::e4m3x2_to_f16x2(kw[1][j]),
                               kv::e4m3x2_to_f16x2(kw[0][j] >> 16), kv::e4m3x2_to_f16x2(kw[1][j] >> 16)};
#pragma unroll
        for (int n = 0; n < NT * QP; ++n) {
          if constexpr (S::kQSmem) {
            const uint2 b = ptx::lds64(q_smem + ((n * kMt + j) * 32 + lane) * 8);
            product(n / QP, s[n / QP][i], a, b.x, b.y);
          } else {
            product(n / QP, s[n / QP][i], a, qf[n][j][0], qf[n][j][1]);
          }
        }
      }
    }
    // Maxima.  s keeps the products; a score is s * f2 (f2 > 0), and only masked tiles, where an unseen
    // page's scale may be anything, hold scores themselves.  m moves by whole numbers: rescaling is exact, and rare.
    float down[NT][2], f2[NT][2][kSteps];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < kSteps; ++i) f2[n][r][i] = fac[n][r] * ks[i];
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float& z = s[n][i][2 * u + r];
              z = (skip >> i & 1u) || key0 + 16 * i + key_at(u, gid) >= lim[n][r] ? -INFINITY : z * f2[n][r][i];
            }
            f2[n][r][i] = 1.0f;
          }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          top = fmaxf(top, fmaf(fmaxf(s[n][i][r], s[n][i][2 + r]), f2[n][r][i], ve[i]));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
        const bool up = top - m[n][r] > kTop;  // false where both are -inf
        grew |= up;
        const float now = up ? floorf(top + (1.0f - kTop)) : m[n][r];
        down[n][r] = up ? m[n][r] - now : 0.0f;
        m[n][r] = now;
      }
    if (__any_sync(kFull, grew)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float c0 = ex2(down[n][0]), c1 = ex2(down[n][1]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // in two steps: between scales far apart m moves by up to 184
          const float half = floorf(0.5f * fmaxf(down[n][r], -300.0f));
          l[n][r] = l[n][r] * ex2(half) * ex2(fmaxf(down[n][r], -300.0f) - half);
        }
#pragma unroll
        for (int j = 0; j < kMt; ++j) {
          acc[n][j][0] *= c0;
          acc[n][j][1] *= c1;
          acc[n][j][2] *= c0;
          acc[n][j][3] *= c1;
          if constexpr (kHold) {
            held[j][0] *= c0;
            held[j][1] *= c1;
            held[j][2] *= c0;
            held[j][3] *= c1;
          }
        }
      }
    }
    // Weights as operands: pb[n][part][i][u], keys 2 tig, 2 tig + 1 of group u for query row gid
    uint32_t pb[NT][PP][kSteps][2];
    float vf[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) vf[i] = vs[i] * b_unit;
    if (skip != 0u) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (skip >> i & 1u) vf[i] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float ref[2] = {m[n][0] == -INFINITY ? 0.0f : m[n][0], m[n][1] == -INFINITY ? 0.0f : m[n][1]};
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float pv[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float w = ex2(fmaf(s[n][i][2 * u + r], f2[n][r][i], -ref[r]));
            l[n][r] += w;
            pv[r] = w * vf[i];
          }
          const uint32_t h = to_f16x2(pv[0], pv[1]);
          pb[n][0][i][u] = ptx::transpose8x8(h);
          if constexpr (PP == 2) {
            const float2 back = from_f16x2(h);
            pb[n][1][i][u] = ptx::transpose8x8(to_f16x2(pv[0] - back.x, pv[1] - back.y));
          }
        }
    }
    // O^T += V^T P^T: rows gid and gid + 8 of tile w are columns kCols gid + 2 w and + 1 of O
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (D == 128) {
          const uint4 v = ptx::lds128u(tile + i * 2048 + v_off[x]);
          vw[x][0] = v.x, vw[x][1] = v.y, vw[x][D / 32 - 2] = v.z, vw[x][D / 32 - 1] = v.w;
        } else {
          const uint2 v = ptx::lds64(tile + i * 1024 + v_off[x]);
          vw[x][0] = v.x, vw[x][1] = v.y;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // columns 4 w + 2 half, + 1: bytes of two keys side by side
          const uint32_t a = __byte_perm(vw[0][w], vw[1][w], half ? 0x7362 : 0x5140);
          const uint32_t b = __byte_perm(vw[2][w], vw[3][w], half ? 0x7362 : 0x5140);
          const uint32_t av[4] = {kv::e4m3x2_to_f16x2(a), kv::e4m3x2_to_f16x2(a >> 16), kv::e4m3x2_to_f16x2(b),
                                  kv::e4m3x2_to_f16x2(b >> 16)};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < PP; ++part)
              product(n, acc[n][2 * w + half], av, pb[n][part][i][0], pb[n][part][i][1]);
        }
    }
  };

  // Columns 4 j .. 4 j + 3 of the lane's part of query row 2 tig + r of tile n: the accumulators, with
  // what was put aside (`from`) at weight `keep`.
  auto four = [&](int n, int r, int j, const float* from, float keep, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = acc[n][2 * j + (e >> 1)][2 * (e & 1) + r];
      if constexpr (kHold) x[e] += held[2 * j + (e >> 1)][2 * (e & 1) + r];
    }
    if (flushed) {
      const float4 y = *reinterpret_cast<const float4*>(from + 4 * j);
      x[0] = fmaf(y.x, keep, x[0]), x[1] = fmaf(y.y, keep, x[1]);
      x[2] = fmaf(y.z, keep, x[2]), x[3] = fmaf(y.w, keep, x[3]);
    }
  };

  // Weight of what was put aside of a row (zeros where it had seen nothing).
  auto keep_of = [&](int n, int r) {
    return flushed && m_aside[n][r] != -INFINITY ? ex2(m_aside[n][r] - m[n][r]) : 0.0f;
  };

  // Puts the accumulators aside: adds them to the others and clears them.
  auto to_workspace = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float* const at = aside + (n * 8 + 2 * tig + r) * D + gid * kCols;
        const float keep = keep_of(n, r);
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j) {
          float x[4];
          four(n, r, j, at, keep, x);
          *reinterpret_cast<float4*>(at + 4 * j) = make_float4(x[0], x[1], x[2], x[3]);
        }
        m_aside[n][r] = m[n][r];
      }
#pragma unroll
      for (int j = 0; j < kMt; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.0f;
    }
    flushed = true;
  };
  auto flush = [&]() {
    since = 0;
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < kMt; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          held[j][e] += acc[0][j][e];
          acc[0][j][e] = 0.0f;
        }
    } else {
      to_workspace();
    }
  };

  // Leaves the rows of an item: the answer where the item was this worker's alone, else a partial at
  // part_o [RT][D], part_ml [RT], with l between 1 and 2.
  auto end_item = [&](bool whole, float* part_o, float2* part_ml) {
    const int n_rows = seq.rows * p.group;
    const int base = static_cast<int>(-127.0f - b_off);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[n][r];
        sum += __shfl_xor_sync(kFull, sum, 4);
        sum += __shfl_xor_sync(kFull, sum, 8);
        sum += __shfl_xor_sync(kFull, sum, 16);
        const int local = n * 8 + 2 * tig + r;
        const int rho = row_q + local;
        if (rho >= n_rows) continue;
        const float keep = keep_of(n, r);
        const int up = min(max(static_cast<int>(__float_as_uint(sum) >> 23 & 255u) - 127, -100), 126);
        const float norm = sum * kv::pow2(-up), ref = m[n][r] + static_cast<float>(up);
        const float back = kv::pow2(min(max(base - kPExp - up, -126), 127));
        const float f = whole ? (sum == 0.0f ? 0.0f : back / norm) : back;
        float* const part = part_o + local * D + gid * kCols;
        const int t = rho / p.group;
        const int64_t out = (seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group);
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j) {
          float x[4];
          four(n, r, j, aside + local * D + gid * kCols, keep, x);
          if (whole) store_row4(p, out * D + gid * kCols + 4 * j, x[0] * f, x[1] * f, x[2] * f, x[3] * f);
          else *reinterpret_cast<float4*>(part + 4 * j) = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
        }
        if (gid == 0) {
          if (whole) p.lse[out] = sum == 0.0f ? -INFINITY : (ref + log2f(norm)) * kLn2;
          else part_ml[local] = make_float2(sum == 0.0f ? -INFINITY : ref, norm);
        }
      }
  };

  // A stage is mostly there already: the clock that bounds the wait is read only where it is not.
  auto wait = [&](uint32_t bar, uint32_t par) {
    return __all_sync(kFull, ptx::mbar_try_wait(bar, par)) || sync::wait_warp(bar, par, ctl, kv::kSiteWait);
  };
  int st = 0, in_flight = 0;
  uint32_t parity = 0;
  bool from_start = c.g == 0;  // the item at hand is ours from its first granule on
  while (true) {  // once; for each block of rows where SOLO
    for (int i = 0; i < kSt; ++i)
      if (to_issue > 0) {
        issue(st + i < kSt ? st + i : st + i - kSt);
        ++in_flight;
      }
    begin_item();
    while (left > 0) {
      if (!wait(bars + st * 8, parity)) {
        ok = false;
        break;
      }
      const int key0 = c.g * kKeys;
      if (key0 < lim_max) {
        granule(st, key0 + kKeys > lim_min);
        if (second) continue;
      }
      __syncwarp();
      if (to_issue > 0) issue(st);
      else --in_flight;
      if (++st == kSt) {
        st = 0;
        parity ^= 1u;
      }
      --left;
      ++c.g;
      if (c.g == c.gpi || left == 0) {
        if (SOLO) break;
        const int64_t slot = worker * 2 + (inside ? 0 : 1);
        end_item(from_start && c.g == c.gpi, p.part_o + slot * (RT * D), p.part_ml + slot * RT);
        left -= kSetup;  // of the next item
        if (left <= 0) break;
        c.g = 0;
        from_start = true;
        inside = false;
        if (++c.block == c.blocks) {
          c.block = 0;
          if (++c.head == p.hkv) next_seq<D, RT>(p, c, seq);
        }
        begin_item();
      } else if (++since == S::kFlush && (kHold || !SOLO)) {  // 16 granules need no more
        flush();
      }
    }
    if (!SOLO) break;
    // The warps' partials meet where their stages were; a warp of no granules leaves an empty one.
    static_assert(S::kStages * S::kStage >= RT * (D * 4 + 8), "a warp's partial fits its stages");
    float* const mine = reinterpret_cast<float*>(smem + warp * S::kWarpBytes);
    __syncwarp();
    end_item(false, mine, reinterpret_cast<float2*>(mine + RT * D));
    __syncthreads();
    auto finish = [&](int rho, float top, float sum, float (&x)[D / 32]) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[j] *= inv;
      const int t = rho / p.group;
      const int64_t out = (seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group);
      store_lane(p, out * D + lane * (D / 32), x);
      if (lane == 0) p.lse[out] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };
    for (int i = warp; i < RT; i += S::kWarps) {
      const int rho = row_q + i;
      if (rho >= seq.rows * p.group) break;
      float top = -INFINITY;
      for (int w = 0; w < S::kWarps; ++w)
        top = fmaxf(top, reinterpret_cast<const float2*>(smem + w * S::kWarpBytes + RT * D * 4)[i].x);
      const float ref = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f, x[D / 32];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[j] = 0.0f;
      for (int w = 0; w < S::kWarps; ++w) {
        const float2 ml = reinterpret_cast<const float2*>(smem + w * S::kWarpBytes + RT * D * 4)[i];
        const float wt = ex2(ml.x - ref);
        sum = fmaf(wt, ml.y, sum);
        const float* const from = reinterpret_cast<const float*>(smem + w * S::kWarpBytes) + i * D + lane * (D / 32);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) x[j] = fmaf(wt, from[j], x[j]);
      }
      if constexpr (SOLO == 1) {
        finish(rho, top, sum, x);
      } else {  // the block's partial takes the place of its first warp's
        __syncwarp();
#pragma unroll
        for (int j = 0; j < D / 32; ++j) reinterpret_cast<float*>(smem)[i * D + lane * (D / 32) + j] = x[j];
        if (lane == 0) reinterpret_cast<float2*>(smem + RT * D * 4)[i] = make_float2(top, sum);
      }
    }
    int stop = 0;
    if constexpr (SOLO == 2) {
      ptx::cluster_sync();
      for (int i = rank + cluster * warp; i < RT; i += solo_warps) {
        const int rho = row_q + i;
        if (rho >= seq.rows * p.group) break;
        float top = -INFINITY, sum = 0.0f;
        if (lane < cluster) {
          const uint32_t at = ptx::cluster_addr(base + RT * D * 4 + i * 8, lane);
          top = ptx::ld_cluster(at);
          sum = ptx::ld_cluster(at + 4);
        }
        const float mine = top;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        top = __shfl_sync(kFull, top, 0);
        const float wt = ex2(mine - (top == -INFINITY ? 0.0f : top));
        sum *= wt;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        sum = __shfl_sync(kFull, sum, 0);
        float x[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) x[j] = 0.0f;
#pragma unroll 4
        for (int r = 0; r < cluster; ++r) {
          const float w = __shfl_sync(kFull, wt, r);
          const uint32_t at = ptx::cluster_addr(base + (i * D + lane * (D / 32)) * 4, r);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) x[j] = fmaf(w, ptx::ld_cluster(at + 4 * j), x[j]);
        }
        finish(rho, top, sum, x);
      }
      // a wait that ran out in one block ends them all, since they read one another's memory
      if (lane < cluster)
        stop = __float_as_int(ptx::ld_cluster(ptx::cluster_addr(base + S::kCtlOff, lane)));
      stop = __any_sync(kFull, stop != 0);
    }
    ptx::fence_proxy_async_smem();  // the next block's copies write where the partials were
    if constexpr (SOLO == 2) ptx::cluster_sync();
    else __syncthreads();
    if (++c.block == c.blocks || (SOLO == 2 ? stop != 0 : *abort_flag != 0)) break;
    f.block = c.block;
    f.g = c.g = g_first;
    left = to_issue = solo_left;
  }
  if (!ok) {
    // copies in flight must not outlive the block: those of this granule and, where there was more to
    // copy, of the next
    for (int i = 0; i < in_flight; ++i) {
      sync::wait_drain(bars + st * 8, parity, p.timeout_ns);
      if (++st == kSt) {
        st = 0;
        parity ^= 1u;
      }
    }
  }
}

// Sum the partials of the items that several workers shared, and answer the rows that see nothing.  What
// depends on the shapes alone is worked out before the wait for the first kernel, while its last blocks
// still run.
constexpr int kSumThreads = 256;

// The partials of an output row: one of each worker from w0 on, the first in slot slot0.
struct Parts {
  int64_t w0;
  int slot0, local;  // local: row of the item
  int n;             // 0: the row sees nothing; -1: nothing to write here
};
template <int D, int RT>
__device__ __forceinline__ Parts parts_of(const Params& p, const int64_t* plan, int64_t n_workers, int64_t row, int h,
                                          int b) {
  Parts r{0, 0, 0, -1};
  const int64_t W = plan[p.rows.n_seqs];
  const Seq seq = seq_of<D, RT>(p, b);
  if (row < seq.r0 || row >= seq.r0 + seq.rows) return r;
  r.n = 0;
  if (seq.blocks == 0) return r;
  const int head = h / p.group;
  const int rho = static_cast<int>(row - seq.r0) * p.group + (h - head * p.group);
  const int block = rho / RT;
  r.local = rho - block * RT;
  const int64_t from = plan[b] + (static_cast<int64_t>(head) * seq.blocks + block) * (seq.gpi + kSetup) + kSetup;
  r.w0 = worker_of(W, n_workers, from);
  const int64_t w1 = worker_of(W, n_workers, from + seq.gpi - 1);
  r.slot0 = share(W, n_workers, r.w0) < from ? 1 : 0;       // the later ones begin inside of the item
  r.n = r.w0 == w1 ? -1 : static_cast<int>(w1 - r.w0) + 1;  // one: finished by its worker
  return r;
}

// WPR warps for each (row, query head), each going over every WPR-th partial.  Most rows of short items were
// finished by their worker: a warp of its own looks 32 of its rows up side by side (58 x 32 items of up to 52
// rows and one granule: 36 us the whole call, against 56 one row after the other).
template <int D, int RT, int WPR>
__global__ void __launch_bounds__(kSumThreads, 4)
    kv_attn_combine_kernel(const __grid_constant__ Params p, int64_t most) {
  constexpr int kN = D / 32, kPer = kSumThreads / 32 / WPR;  // rows of a block at a time
  extern __shared__ int64_t plan[];
  __shared__ int64_t scratch[kSumThreads / 32];
  __shared__ float sh_o[WPR > 1 ? WPR : 1][D];
  __shared__ float2 sh_ml[WPR];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % WPR;
  const int64_t outs = p.rows.n_rows * p.hq;
  make_plan<D, RT, kSumThreads>(p, plan, scratch);
  const int64_t n = workers(p, plan[p.rows.n_seqs], most);
  bool waited = false;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kPer;
  constexpr int kScan = WPR == 1 ? 32 : 1;
  for (int64_t id0 = static_cast<int64_t>(blockIdx.x) * kPer + warp / WPR; id0 < outs; id0 += kScan * stride) {
    Parts mine{0, 0, 0, -1};
    unsigned todo;
    if constexpr (WPR == 1) {
      const int64_t my_id = id0 + lane * stride;
      if (my_id < outs) {
        const int64_t row = my_id / p.hq;
        int b = 0, z = p.rows.n_seqs - 1;  // the last sequence that begins at or before the row
        while (b < z) {
          const int mid = (b + z + 1) >> 1;
          if (kv::row_at(p.rows, mid) <= row) b = mid;
          else z = mid - 1;
        }
        mine = parts_of<D, RT>(p, plan, n, row, static_cast<int>(my_id - row * p.hq), b);
      }
      todo = __ballot_sync(kFull, mine.n >= 0);
    } else {
      const int64_t row = id0 / p.hq;
      const int b = kv::find_seq(p.rows.n_seqs, row, lane, [&](int i) { return kv::row_at(p.rows, i); });
      mine = parts_of<D, RT>(p, plan, n, row, static_cast<int>(id0 - row * p.hq), b);
      todo = mine.n >= 0 ? 1u : 0u;  // the same for the whole block
    }
    if (!waited) ptx::wait_dependencies();
    waited = true;
    while (todo != 0u) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1u;
      const int64_t id = id0 + src * stride;
      Parts r = mine;
      if constexpr (WPR == 1) {
        r.w0 = __shfl_sync(kFull, mine.w0, src);
        r.slot0 = __shfl_sync(kFull, mine.slot0, src);
        r.local = __shfl_sync(kFull, mine.local, src);
        r.n = __shfl_sync(kFull, mine.n, src);
      }
      const int parts = r.n;
      auto place = [&](int i) { return ((r.w0 + i) * 2 + (i == 0 ? r.slot0 : 0)) * RT + r.local; };
      float top = -INFINITY, sum = 0.0f;
      float acc[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
      for (int base = sub; base < parts; base += 32 * WPR) {
        const int mine = base + lane * WPR;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (mine < parts) ml = p.part_ml[place(mine)];
        float t = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, o));
        const float now = fmaxf(top, t);
        const float ref = now == -INFINITY ? 0.0f : now;
        const float old = ex2(top - ref);
        const float wt = ex2(ml.x - ref);
        float z = ml.y * wt;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
        sum = sum * old + z;
#pragma unroll
        for (int j = 0; j < kN; ++j) acc[j] *= old;
        top = now;
        const int many = (parts - 1 - base) / WPR + 1;
        const int count = many < 32 ? many : 32;
        for (int i0 = 0; i0 < count; i0 += 4) {
          float v[4][kN];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (i0 + u < count) {
              const float* src = p.part_o + place(base + (i0 + u) * WPR) * D + lane * kN;
              if constexpr (kN == 4) {
                const float4 x = *reinterpret_cast<const float4*>(src);
                v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][kN - 1] = x.w;
              } else {
                const float2 x = *reinterpret_cast<const float2*>(src);
                v[u][0] = x.x, v[u][1] = x.y;
              }
            }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float wi = __shfl_sync(kFull, wt, (i0 + u) & 31);
            if (i0 + u < count) {
#pragma unroll
              for (int j = 0; j < kN; ++j) acc[j] = fmaf(wi, v[u][j], acc[j]);
            }
          }
        }
      }
      if constexpr (WPR > 1) {
        __syncthreads();  // the row before has been read
#pragma unroll
        for (int j = 0; j < kN; ++j) sh_o[warp][lane * kN + j] = acc[j];
        if (lane == 0) sh_ml[warp] = make_float2(top, sum);
        __syncthreads();
        if (warp == 0) {
          float all = -INFINITY;
          for (int w = 0; w < WPR; ++w) all = fmaxf(all, sh_ml[w].x);
          const float ref = all == -INFINITY ? 0.0f : all;
          sum = 0.0f;
#pragma unroll
          for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
          for (int w = 0; w < WPR; ++w) {
            const float wt = ex2(sh_ml[w].x - ref);
            sum = fmaf(wt, sh_ml[w].y, sum);
#pragma unroll
            for (int j = 0; j < kN; ++j) acc[j] = fmaf(wt, sh_o[w][lane * kN + j], acc[j]);
          }
          top = all;
        }
      }
      if (sub == 0) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int j = 0; j < kN; ++j) acc[j] *= inv;
        store_lane(p, id * D + lane * kN, acc);
        if (lane == 0) p.lse[id] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
    }
  }
  // A block without rows waits too: the kernel behind this one may begin once this grid is through,
  // and must not meet the blocks of the one before.
  if (!waited) ptx::wait_dependencies();
}

// A block for each 32 columns of a (row, query head): eight lanes, four columns each, to a partial, so that 32
// partials are summed side by side and 256 reads are on their way.  For one row of 1800 partials, as one long
// sequence leaves them, a block of eight warps for a row's whole length took 27 us.
template <int D, int RT>
__global__ void __launch_bounds__(kSumThreads, 4)
    kv_attn_combine_columns_kernel(const __grid_constant__ Params p, int64_t most) {
  constexpr int kWarps = kSumThreads / 32, kSide = kSumThreads / 8, kSlices = D / 32;
  extern __shared__ int64_t plan[];
  __shared__ int64_t scratch[kWarps];
  __shared__ float sh_m[kWarps], sh_l[kWarps];
  __shared__ float4 sh_o[kWarps][8];
  float* const weight = reinterpret_cast<float*>(plan + p.rows.n_seqs + 1);  // [most]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t ids = p.rows.n_rows * p.hq * kSlices;
  make_plan<D, RT, kSumThreads>(p, plan, scratch);
  const int64_t n = workers(p, plan[p.rows.n_seqs], most);
  bool waited = false;
  for (int64_t id = blockIdx.x; id < ids; id += gridDim.x) {
    const int64_t out = id / kSlices;
    const int col = static_cast<int>(id % kSlices) * 32;
    const int64_t row = out / p.hq;
    const int b = kv::find_seq(p.rows.n_seqs, row, lane, [&](int i) { return kv::row_at(p.rows, i); });
    const Parts r = parts_of<D, RT>(p, plan, n, row, static_cast<int>(out - row * p.hq), b);
    if (!waited) ptx::wait_dependencies();
    waited = true;
    if (r.n < 0) continue;  // the same for the whole block
    auto place = [&](int i) { return ((r.w0 + i) * 2 + (i == 0 ? r.slot0 : 0)) * RT + r.local; };
    float top = -INFINITY;
    for (int i = tid; i < r.n; i += kSumThreads) {
      const float m = p.part_ml[place(i)].x;
      weight[i] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (lane == 0) sh_m[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int i = tid; i < r.n; i += kSumThreads) {
      const float wt = ex2(weight[i] - ref);
      weight[i] = wt;
      sum = fmaf(wt, p.part_ml[place(i)].y, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) sh_l[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh_l[w];
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* const from = p.part_o + col + (tid & 7) * 4;
    constexpr int kAhead = 8;
    for (int i0 = tid >> 3; i0 < r.n; i0 += kSide * kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u * kSide < r.n) v[u] = *reinterpret_cast<const float4*>(from + place(i0 + u * kSide) * D);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u * kSide < r.n) {
          const float wt = weight[i0 + u * kSide];
          acc.x = fmaf(wt, v[u].x, acc.x), acc.y = fmaf(wt, v[u].y, acc.y);
          acc.z = fmaf(wt, v[u].z, acc.z), acc.w = fmaf(wt, v[u].w, acc.w);
        }
    }
#pragma unroll
    for (int o = 16; o >= 8; o >>= 1) {
      acc.x += __shfl_xor_sync(kFull, acc.x, o), acc.y += __shfl_xor_sync(kFull, acc.y, o);
      acc.z += __shfl_xor_sync(kFull, acc.z, o), acc.w += __shfl_xor_sync(kFull, acc.w, o);
    }
    if (lane < 8) sh_o[warp][lane] = acc;
    __syncthreads();
    if (tid < 8) {
      acc = sh_o[0][tid];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 x = sh_o[w][tid];
        acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      store_row4(p, out * D + col + tid * 4, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (col == 0 && tid == 0) p.lse[out] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
  if (!waited) ptx::wait_dependencies();  // as above
}

// The variant for a call: by the query rows that a sequence has on average.
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
template <int D, int NT, int QP, int PP>
cp_status run(const Params& p, const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv, int64_t items,
              int num_sms, cudaStream_t s) {
  using S = Shape<D, NT, QP, PP>;
  constexpr int most_smem = 1024 + S::kPlanOff + (CP_KV_MAX_SEQS + 1) * 8;
  static_assert(most_smem <= 232448, "shared memory of a block");
  const int smem = 1024 + S::kPlanOff + (p.rows.n_seqs + 1) * 8;
  const auto kernel = !pl.solo           ? kv_attn_kernel<D, NT, QP, PP, 0>
                      : pl.cluster == 1 ? kv_attn_kernel<D, NT, QP, PP, 1>
                                        : kv_attn_kernel<D, NT, QP, PP, 2>;
  // The limit is the function's, not the call's: always the same, for other host threads launch the kernel too.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
  if (e != cudaSuccess) return cuda_fail(e, "kv_attn_kernel attribute");
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(pl.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pl.solo && pl.cluster > 1 ? 2 : 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(pl.grid));
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p, mk, mv)) != cudaSuccess) return cuda_fail(e, "kv_attn_kernel launch");
  if (pl.solo) return CP_OK;
  // Eight warps an output row while there are few rows (320 rows of 8 partials: 8 us against 14), or many
  // partials to a row; else one (2176 rows of 5 partials: 104 us the whole call, against 116 with eight; 45 x 0-103
  // tokens, 1-4 rows of 128/32 heads 22 and 75).
  const int64_t workers = pl.grid * S::kWarps, parts = workers / (items < 1 ? 1 : items), outs = p.rows.n_rows * p.hq;
  const bool wide = parts > 16 || outs <= 1024;
  const int64_t resident = 4 * static_cast<int64_t>(num_sms);
  // A block for 32 columns of a row where these are one wave and have many partials to read (1 x 120000 tokens,
  // 5/1 heads: 23 us against 31; 1 x 8000, 32/8, split: 13.6 against 14.3; 4 x 30000: the same).  Two waves of them are
  // slower (1 x 30000 with 32 rows, 32/8: 39 against 36).
  const bool columns = outs * (D / 32) <= resident && parts > 32;
  const int64_t blocks = columns ? outs * (D / 32) : wide ? outs : (outs + 7) / 8;
  cfg.dynamicSmemBytes = (p.rows.n_seqs + 1) * 8 + (columns ? workers * 4 : 0);
  cfg.blockDim = dim3(kSumThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < resident ? blocks : resident));
  const auto sum = columns ? kv_attn_combine_columns_kernel<D, S::kRows>
                   : wide  ? kv_attn_combine_kernel<D, S::kRows, 8>
                           : kv_attn_combine_kernel<D, S::kRows, 1>;
  e = cudaLaunchKernelEx(&cfg, sum, p, workers);
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "kv_attn_combine_kernel launch");
}

template <int D>
cp_status run_d(const Params& p, const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv, int64_t items,
                int num_sms, cudaStream_t s) {
  if (pl.pp == 1)
    return pl.nt == 1 ? run<D, 1, 1, 1>(p, pl, mk, mv, items, num_sms, s)
                      : run<D, 2, 1, 1>(p, pl, mk, mv, items, num_sms, s);
  if (pl.qp == 1)
    return pl.nt == 1 ? run<D, 1, 1, 2>(p, pl, mk, mv, items, num_sms, s)
                      : run<D, 2, 1, 2>(p, pl, mk, mv, items, num_sms, s);
  return pl.nt == 1 ? run<D, 1, 2, 2>(p, pl, mk, mv, items, num_sms, s)
                    : run<D, 2, 2, 2>(p, pl, mk, mv, items, num_sms, s);
}

}  // namespace kvattn
}  // namespace cpattn

// Attention of a batch's new tokens over the paged 8-bit cache (cp_kv_cache_attn).
//
// Per (sequence, KV head) the g = hq / hkv query heads of the sequence's rows are one block of
// query rows that share keys and values:
//   s_ij = scale * ks(page of j) * (q_i . k8_j),  p_ij = 2^(s_ij log2 e - m_i),
//   O_i = sum_j p_ij vs(page of j) v8_j / l_i,    LSE_i = ln 2 (m_i + log2 l_i),  l_i = sum_j p_ij.
// Bound: every cached byte is read once for 2 g rows' worth of products per byte, so it is memory
// bound for up to a few dozen rows; the design is about keeping loads in flight and splitting the
// keys evenly, not about the tensor rate.
//
// Work split.  The unit is a granule of 32 keys of one item (sequence, KV head, block of RT query
// rows); granules are numbered item after item.  Every warp of the grid is a worker on its own,
// with an equal share of consecutive granules, whatever the sequences' lengths: no barrier between
// warps, and a worker's copies run ahead across item borders.  An item that lies within one share is
// finished there; of the others each worker leaves a partial (O unnormalised, m, l), at most two per
// worker (the item its share begins in and the one it ends in), and a second kernel, launched as
// a programmatic dependent, combines them in the order of the workers.
//
// Products.  mma.sync m16n8k16 with f16 operands: e4m3 -> f16 is exact and one instruction for two
// values, and with 8 to 32 query rows the 128-row tiles of tcgen05 would be mostly empty.  Rows of
// S are query rows, so that the accumulator layout of S is the operand layout of P.  The orders of
// keys and dimensions inside the products are free as long as both operands agree; they are chosen
// so that every lane reads 16 consecutive bytes of a key or value row, without bank conflicts under
// the 128-byte swizzle that the copies apply.
//
// Precision.  A query row is scaled by a power of two to at most 2^15 and split into f16 parts, high
// and low; P likewise (times 2^15).  With up to 8 rows (kTwo) the unused upper half of the 16-row
// operand holds the low parts: 22 bits at no cost.  With more rows and bf16 in and out, one f16
// part is enough: bf16 queries are exact, and P's 2^-12 is far below the output's 2^-9.  Sums,
// maxima and the accumulators are fp32.
#include "internal.h"
#include "kv_common.cuh"
#include "ptx.cuh"
#include "sync.cuh"

namespace cpattn {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kPScale = 32768.0f;  // largest P operand
constexpr int kKeys = 32;            // keys of a granule
constexpr unsigned kFull = 0xffffffffu;

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

template <int D, int NT, bool TWO>
struct Shape {
  static constexpr int kWarps = 8;
  static constexpr int kRows = NT * (TWO ? 8 : 16);  // RT
  static constexpr int kStages = D == 128 ? (NT == 1 ? 3 : 2) : 4;
  static constexpr int kHalf = kKeys * D;            // bytes of K (or V) of a granule
  static constexpr int kStage = 2 * kHalf;
  static constexpr bool kQSmem = NT > 1;             // query operands in shared memory
  static constexpr int kQBytes = kQSmem ? NT * (D / 16) * 512 : 0;
  static constexpr int kWarpBytes = kStages * kStage + kQBytes;
  // behind the warps' parts (1024-byte aligned for the swizzle): scales, barriers, control, plan
  static constexpr int kScaleOff = kWarps * kWarpBytes;               // [warp][stage][4] fp32
  static constexpr int kBarOff = kScaleOff + kWarps * kStages * 16;   // [warp][stage] + stall
  static constexpr int kCtlOff = kBarOff + (kWarps * kStages + 1) * 8;
  static constexpr int kPlanOff = (kCtlOff + 8 + 15) / 16 * 16 + 16 * 16;  // 16 x 8 B scan scratch before it
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
  int64_t* plan;   // [n_seqs + 1] granules before each sequence (workspace)
  float* part_o;   // [workers][2][RT][D]
  float2* part_ml; // [workers][2][RT]: m (base 2), l
};

// What a sequence asks for.
struct Seq {
  int64_t r0;      // first row
  int64_t pos0;    // position of its first row
  int32_t rows;
  int32_t tokens;  // cached tokens, as far as the page table reaches
  int32_t keys;    // tokens that its last row sees
  int32_t gpi;     // granules of an item, at least 1
  int32_t blocks;  // blocks of RT query rows
  bool over;       // more tokens than the table has pages for
};

// Number of tokens that a row at position `pos` sees: token j stands at base + stride * j.
__device__ __forceinline__ int32_t visible(const Params& p, int32_t tokens, int64_t pos) {
  if (p.q_first == nullptr) return tokens;
  const int64_t off = pos - p.kv_pos.base;
  if (off < 0) return 0;
  const int64_t n = off / p.kv_pos.stride + 1;
  return n < tokens ? static_cast<int32_t>(n) : tokens;
}

template <int RT>
__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  Seq s;
  s.r0 = kv::row_at(p.rows, b);
  const int64_t r1 = kv::row_at(p.rows, b + 1);
  s.rows = r1 > s.r0 ? static_cast<int32_t>(r1 - s.r0) : 0;
  int64_t t = __ldg(p.rows.tokens + b);
  const int64_t room = static_cast<int64_t>(p.rows.max_pages) << p.page_log2;
  s.over = t > room;
  if (s.over) t = room;
  s.tokens = t < 0 ? 0 : static_cast<int32_t>(t);
  s.pos0 = p.q_first != nullptr ? __ldg(p.q_first + b) : 0;
  s.keys = s.rows > 0 ? visible(p, s.tokens, s.pos0 + s.rows - 1) : 0;
  s.gpi = s.keys > kKeys ? (s.keys + kKeys - 1) / kKeys : 1;
  s.blocks = static_cast<int32_t>((static_cast<int64_t>(s.rows) * p.group + RT - 1) / RT);
  return s;
}
__device__ __forceinline__ int64_t granules(const Params& p, const Seq& s) {
  return static_cast<int64_t>(s.blocks) * p.hkv * s.gpi;
}

// Shares of W granules among n workers: worker w has [share(w), share(w + 1)).
__device__ __forceinline__ int64_t share(int64_t W, int64_t n, int64_t w) { return W * w / n; }
__device__ __forceinline__ int64_t worker_of(int64_t W, int64_t n, int64_t x) { return ((x + 1) * n - 1) / W; }
__device__ __forceinline__ int64_t workers(int64_t W, int64_t most) { return W < most ? W : most; }

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

// Granules before each sequence, in shared memory: plan[0 .. n_seqs].
template <int RT, int THREADS>
__device__ __forceinline__ void make_plan(const Params& p, int64_t* plan, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.rows.n_seqs;
  int64_t before = 0;
  for (int base = 0; base < n; base += THREADS) {
    const int b = base + tid;
    int64_t x = 0;
    if (b < n) {
      const Seq s = seq_of<RT>(p, b);
      x = granules(p, s);
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

// Moves to the first sequence at or behind c.b + 1 that has rows.
template <int RT>
__device__ __forceinline__ void next_seq(const Params& p, Cursor& c, Seq& s) {
  do {
    ++c.b;
    if (c.b >= p.rows.n_seqs) return;
    s = seq_of<RT>(p, c.b);
  } while (s.blocks == 0);
  c.head = c.block = c.g = 0;
  c.gpi = s.gpi;
  c.blocks = s.blocks;
}

template <int D, int NT, bool TWO>
__global__ void __launch_bounds__(Shape<D, NT, TWO>::kWarps * 32, 1)
    kv_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v) {
  using S = Shape<D, NT, TWO>;
  constexpr int RT = S::kRows;
  constexpr int kNd = D / 8;          // 8-column tiles of O; also the columns of a lane's V chunk
  constexpr int kRl = TWO ? 1 : 2;    // query rows of a lane per row tile
  constexpr int kSt = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  int64_t* const plan = reinterpret_cast<int64_t*>(smem + S::kPlanOff);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + S::kCtlOff);
  const uint32_t base = ptx::smem_u32(smem);
  const uint32_t ring = base + warp * S::kWarpBytes;
  const uint32_t q_smem = ring + kSt * S::kStage;
  const uint32_t scales = base + S::kScaleOff + warp * kSt * 16;
  const uint32_t bars = base + S::kBarOff + warp * kSt * 8;
  const uint32_t stall_bar = base + S::kBarOff + S::kWarps * kSt * 8;

  if (lane == 0) {
    // one arrival for the copies' bytes, four for the lanes that copy the scales
    for (int i = 0; i < kSt; ++i) ptx::mbar_init(bars + i * 8, 5);
    if (warp == 0) {
      ptx::mbar_init(stall_bar, 1);
      *abort_flag = 0;
      ptx::tma_prefetch_desc(&map_k);
      ptx::tma_prefetch_desc(&map_v);
    }
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  make_plan<RT, S::kWarps * 32>(p, plan, reinterpret_cast<int64_t*>(smem + S::kPlanOff - 16 * 16));
  const int n_seqs = p.rows.n_seqs;
  if (blockIdx.x == 0)
    for (int i = tid; i <= n_seqs; i += S::kWarps * 32) p.plan[i] = plan[i];
  ptx::launch_dependents();
  const sync::Ctl ctl{abort_flag, p.status, p.timeout_ns};
  if (p.stall && blockIdx.x == 0 && warp == 0) {
    sync::wait_warp(stall_bar, 0, ctl, kv::kSiteWait);
    return;
  }

  const int64_t W = plan[n_seqs];
  const int64_t n_workers = workers(W, static_cast<int64_t>(gridDim.x) * S::kWarps);
  const int64_t worker = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;  // neighbours on different SMs
  if (worker >= n_workers) return;
  const int64_t lo = share(W, n_workers, worker), hi = share(W, n_workers, worker + 1);
  int64_t left = hi - lo, to_issue = left;

  Cursor c;  // where the products are
  Seq seq;
  {
    int a = 0, z = n_seqs - 1;  // the last sequence whose granules begin at or before lo
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (plan[mid] <= lo) a = mid;
      else z = mid - 1;
    }
    c.b = a;
    seq = seq_of<RT>(p, a);
    const int64_t off = lo - plan[a];
    const int64_t item = off / seq.gpi;
    c.g = static_cast<int>(off - item * seq.gpi);
    c.head = static_cast<int>(item / seq.blocks);
    c.block = static_cast<int>(item - static_cast<int64_t>(c.head) * seq.blocks);
    c.gpi = seq.gpi;
    c.blocks = seq.blocks;
  }
  Cursor f = c;  // where the copies are
  int f_keys = seq.keys;
  bool f_over = seq.over;
  int64_t page_first = -1;  // lane i holds the (page_first + i)-th page of sequence f.b
  int pages = -1;

  auto page_of = [&](int64_t ord) -> int64_t {
    if (page_first < 0 || ord < page_first || ord >= page_first + 32) {
      page_first = ord;
      const int64_t mine = ord + lane;
      int64_t id = kv::page_at(p.rows, p.n_pages, f.b, mine);
      if (f_over && mine == p.rows.max_pages - 1) id = -1;
      pages = id < 0 ? -1 : static_cast<int>(id);
    }
    return __shfl_sync(kFull, pages, static_cast<int>(ord - page_first));
  };

  // Starts the copies of the next granule into stage `st`.
  auto issue = [&](int st) {
    const uint32_t bar = bars + st * 8, dst = ring + st * S::kStage;
    const int key0 = f.g * kKeys;
    const int parts = p.page < kKeys ? 2 : 1;       // pages of 16 tokens: two to a granule
    const int part_bytes = S::kHalf / parts;
    int64_t page[2] = {-1, -1};
    bool want[2];
    uint32_t tx = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = key0 + i * 16;
      want[i] = i < parts && k < f_keys;
      if (want[i]) {
        page[i] = page_of(static_cast<int64_t>(k) >> p.page_log2);
        if (page[i] >= 0) tx += 2 * part_bytes;
        else if (lane == 0) kv::report(p.status, kv::kSitePage);
      }
    }
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(bar, tx);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (want[i] && page[i] >= 0) {
          const int64_t row = (page[i] * p.hkv + f.head) * p.page + ((key0 + i * 16) & (p.page - 1));
          const int line = static_cast<int>(D == 128 ? row : row >> 1);
          ptx::tma_load_2d(dst + i * part_bytes, &map_k, 0, line, bar);
          ptx::tma_load_2d(dst + S::kHalf + i * part_bytes, &map_v, 0, line, bar);
        }
    }
    if (lane < 4) {  // lane 2 i + w: scale of part i of K (w = 0) or V (w = 1)
      const int i = parts == 2 ? lane >> 1 : 0;
      const int64_t pg = i ? page[1] : page[0];
      const bool need = i ? want[1] : want[0];
      const uint32_t to = scales + st * 16 + lane * 4;
      if (need && pg >= 0)
        ptx::cp_async4(to, p.scale[lane & 1] + pg * p.hkv + f.head);
      else  // no token: the smallest scale; a bad page: NaN, which reaches the rows that see it
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(need ? 0x7fffffffu : 0x1f800000u) : "memory");
      ptx::cp_async_arrive(bar);
    }
    --to_issue;
    if (++f.g == f.gpi) {
      f.g = 0;
      if (++f.block == f.blocks) {
        f.block = 0;
        if (++f.head == p.hkv && to_issue > 0) {
          Seq s{};
          next_seq<RT>(p, f, s);
          f_keys = s.keys;
          f_over = s.over;
          page_first = -1;
        }
      }
    }
  };

  for (int i = 0; i < kSt; ++i)
    if (to_issue > 0) issue(i);

  // lane's offsets inside a stage.  128-byte lines; 16-byte chunk x of line y sits at x ^ (y & 7).
  // D = 128: a line is a key.  Key tile t holds keys 8 t + g; lane (gid, tig) reads dimensions
  //   32 tig .. + 31 of key 8 t + gid, and dimensions 16 gid .. + 15 of four values a step of 16.
  // D = 64: a line is two keys.  Column (2 x + y) of key tile 2 i + u is key 16 i + 4 x + 2 u + y, so
  //   that the four values of a lane are 16 i + 4 tig + (0 .. 3), two lines.
  uint32_t k_off[2], v_off[4];
  if (D == 128) {
#pragma unroll
    for (int j = 0; j < 2; ++j) k_off[j] = gid * 128 + (((2 * tig + j) ^ gid) << 4);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = 2 * tig + (x & 1);
      v_off[x] = S::kHalf + (r + 8 * (x >> 1)) * 128 + ((gid ^ r) << 4);
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
  // first of the two keys of a lane in key tile t
  auto key_of = [&](int t) { return D == 128 ? 8 * t + 2 * tig : 16 * (t >> 1) + 4 * tig + 2 * (t & 1); };

  uint32_t qf[S::kQSmem ? 1 : NT][S::kQSmem ? 1 : D / 16][4];
  float fac[NT][kRl], m[NT][kRl], l[NT][kRl];
  int lim[NT][kRl];
  float acc[NT][kNd][4];
  float v_ref = 1e-37f;  // largest V scale so far: P is held relative to it
  int lim_min = 0, lim_max = 0;
  int64_t row_q = 0;  // first query row (token row * group + head in group) of the block

  auto begin_item = [&]() {
    row_q = static_cast<int64_t>(c.block) * RT;
    const int64_t n_rows = static_cast<int64_t>(seq.rows) * p.group;
    int lmin = 0x7fffffff, lmax = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < kRl; ++r) {
        const int64_t rho = row_q + n * (TWO ? 8 : 16) + r * 8 + gid;
        const bool live = rho < n_rows;
        const int64_t t = live ? rho / p.group : 0;
        const int64_t at = ((seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group)) * D + tig * (D / 4);
        lim[n][r] = live ? visible(p, seq.tokens, seq.pos0 + t) : -1;
        if (live) {
          lmin = min(lmin, lim[n][r]);
          lmax = max(lmax, lim[n][r]);
        }
        float x[D / 16][4];
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          if (live) load4(p, at + s * 4, x[s]);
          else x[s][0] = x[s][1] = x[s][2] = x[s][3] = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[s][e]));
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // 2^e <= top < 2^(e + 1) goes to [2^14, 2^15); rows of (almost) zeros keep a finite factor
        const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
        const float up = kv::pow2(14 - e);
        fac[n][r] = p.scale_log2 * kv::pow2(e - 14);
        m[n][r] = -INFINITY;
        l[n][r] = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          uint32_t h[2], w[2];
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const float a = x[s][2 * e2] * up, b = x[s][2 * e2 + 1] * up;
            h[e2] = to_f16x2(a, b);
            if (TWO) {
              const float2 back = from_f16x2(h[e2]);
              w[e2] = to_f16x2(a - back.x, b - back.y);
            }
          }
          if constexpr (S::kQSmem) {
            const uint32_t to = q_smem + ((n * (D / 16) + s) * 32 + lane) * 16;
            if constexpr (TWO) {
              ptx::sts128(to, h[0], w[0], h[1], w[1]);
            } else {
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + r * 4), "r"(h[0]) : "memory");
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 8 + r * 4), "r"(h[1]) : "memory");
            }
          } else if constexpr (TWO) {
            qf[n][s][0] = h[0], qf[n][s][1] = w[0], qf[n][s][2] = h[1], qf[n][s][3] = w[1];
          } else {
            qf[n][s][r] = h[0], qf[n][s][2 + r] = h[1];
          }
        }
      }
    lim_min = __reduce_min_sync(kFull, lmin);
    lim_max = __reduce_max_sync(kFull, lmax);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < kRl; ++r)
        if (lim[n][r] < 0) lim[n][r] = lim_max;  // rows of nobody must not make the tile a masked one
#pragma unroll
      for (int j = 0; j < kNd; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.0f;
    }
    v_ref = 1e-37f;
  };

  // One granule; kMask: some of its keys are not seen by some row.
  auto granule = [&](int st, auto mask_tag) {
    constexpr bool kMask = decltype(mask_tag)::value;
    const uint32_t tile = ring + st * S::kStage;
    const int key0 = c.g * kKeys;
    const uint4 sc4 = ptx::lds128u(scales + st * 16);
    const float ks[2] = {__uint_as_float(sc4.x), __uint_as_float(sc4.z)};
    const float vs[2] = {__uint_as_float(sc4.y), __uint_as_float(sc4.w)};
    float s[NT][4][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t) s[n][t][0] = s[n][t][1] = s[n][t][2] = s[n][t][3] = 0.0f;
    {
      // words of K: step j of 16 dimensions is the lane's j-th word of a key
      uint32_t kw[4][D / 16];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (D == 128) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 v = ptx::lds128u(tile + t * 1024 + k_off[j]);
            kw[t][4 * j] = v.x, kw[t][4 * j + 1] = v.y, kw[t][4 * j + 2] = v.z, kw[t][4 * j + 3] = v.w;
          }
        } else {
          const uint4 v = ptx::lds128u(tile + (t >> 1) * 1024 + k_off[t & 1]);
          kw[t][0] = v.x, kw[t][1] = v.y, kw[t][2] = v.z, kw[t][3] = v.w;
        }
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t a[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (S::kQSmem) {
            const uint4 v = ptx::lds128u(q_smem + ((n * (D / 16) + j) * 32 + lane) * 16);
            a[n][0] = v.x, a[n][1] = v.y, a[n][2] = v.z, a[n][3] = v.w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[n][e] = qf[n][j][e];
          }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t b0 = kv::e4m3x2_to_f16x2(kw[t][j]), b1 = kv::e4m3x2_to_f16x2(kw[t][j] >> 16);
#pragma unroll
          for (int n = 0; n < NT; ++n) ptx::mma_f16(s[n][t], a[n], b0, b1);
        }
      }
    }
    // scores, maxima
    float corr[NT][kRl];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < kRl; ++r) {
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float f2 = fac[n][r] * ks[t >> 1];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float z = TWO ? s[n][t][e] + s[n][t][2 + e] : s[n][t][2 * r + e];
            z *= f2;
            if (kMask && key0 + key_of(t) + e >= lim[n][r]) z = -INFINITY;
            s[n][t][2 * r + e] = z;
            top = fmaxf(top, z);
          }
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        const bool up = top > m[n][r];
        grew |= up;
        const float now = up ? top : m[n][r];
        corr[n][r] = now == -INFINITY ? 1.0f : ex2(m[n][r] - now);
        m[n][r] = now;
      }
    const float v_top = fmaxf(v_ref, fmaxf(vs[0], vs[1]));
    if (__any_sync(kFull, grew || v_top > v_ref)) {
      const float rr = v_ref / v_top;
      v_ref = v_top;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < kRl; ++r) l[n][r] *= corr[n][r];
        const float c0 = corr[n][0] * rr, c1 = corr[n][kRl - 1] * rr;
#pragma unroll
        for (int j = 0; j < kNd; ++j) {
          acc[n][j][0] *= c0;
          acc[n][j][1] *= c0;
          acc[n][j][2] *= c1;
          acc[n][j][3] *= c1;
        }
      }
    }
    // weights and their operands
    uint32_t pa[NT][2][4];
    const float inv_ref = kPScale / v_ref;
    const float vf[2] = {vs[0] * inv_ref, vs[1] * inv_ref};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < kRl; ++r) {
        const float ref = m[n][r] == -INFINITY ? 0.0f : m[n][r];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float a = ex2(s[n][t][2 * r] - ref), b = ex2(s[n][t][2 * r + 1] - ref);
          l[n][r] += a + b;
          float av = a * vf[t >> 1], bv = b * vf[t >> 1];
          if (kMask) {  // an unseen page's scale may be NaN
            if (s[n][t][2 * r] == -INFINITY) av = 0.0f;
            if (s[n][t][2 * r + 1] == -INFINITY) bv = 0.0f;
          }
          const uint32_t h = to_f16x2(av, bv);
          // operand register: row gid (+ 8) of the even or odd key tile of a step
          if constexpr (TWO) {
            const float2 back = from_f16x2(h);
            pa[n][t >> 1][2 * (t & 1)] = h;
            pa[n][t >> 1][2 * (t & 1) + 1] = to_f16x2(av - back.x, bv - back.y);
          } else {
            pa[n][t >> 1][2 * (t & 1) + r] = h;
          }
        }
      }
    // O += P V
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t vw[4][D / 32];
      bool odd = false;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (D == 128) {
          const uint4 v = ptx::lds128u(tile + i * 2048 + v_off[x]);
          vw[x][0] = v.x, vw[x][1] = v.y, vw[x][D / 32 - 2] = v.z, vw[x][D / 32 - 1] = v.w;
        } else {
          const uint2 v = ptx::lds64(tile + i * 1024 + v_off[x]);
          vw[x][0] = v.x, vw[x][1] = v.y;
        }
        if (kMask) {
          // what no row sees counts as zero: 0 * NaN would not vanish
          const int key = key0 + 16 * i + (D == 128 ? 2 * tig + (x & 1) + 8 * (x >> 1) : 4 * tig + x);
          if (key >= lim_max) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vw[x][w] = 0u;
          } else if (key >= lim_min) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) odd |= __vcmpeq4(vw[x][w] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
          }
        }
      }
      if (kMask && __any_sync(kFull, odd)) {
        // NaN among values that only some of the rows see: those rows get NaN by a product of the
        // rows' visibility with the places of the NaN, and the NaN are taken out of V.
        uint32_t va[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = key0 + key_of(2 * i + u);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int lm = r < kRl ? lim[n][r < kRl ? r : 0] : 0;
              va[n][2 * u + r] = (k < lm ? 0x3c00u : 0u) | (k + 1 < lm ? 0x3c000000u : 0u);
            }
          }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t at[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t nan = __vcmpeq4(vw[x][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            at[x] = nan & 0x38383838u;  // e4m3 one
            vw[x][w] &= ~nan;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t sel = (e & 1) * 0x11u + (e >> 1) * 0x22u;
            const uint32_t b0 = kv::e4m3x2_to_f16x2(__byte_perm(at[0], at[1], 0x40u + sel));
            const uint32_t b1 = kv::e4m3x2_to_f16x2(__byte_perm(at[2], at[3], 0x40u + sel));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              ptx::mma_f16(hit, va[n], b0, b1);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (hit[k] > 0.0f) acc[n][4 * w + e][k] = __int_as_float(0x7fffffff);
            }
          }
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        // bytes of two keys side by side: columns 4 w, 4 w + 1 and 4 w + 2, 4 w + 3
        const uint32_t a01 = __byte_perm(vw[0][w], vw[1][w], 0x5140), b01 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
        const uint32_t a23 = __byte_perm(vw[0][w], vw[1][w], 0x7362), b23 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
        const uint32_t b0[4] = {kv::e4m3x2_to_f16x2(a01), kv::e4m3x2_to_f16x2(a01 >> 16), kv::e4m3x2_to_f16x2(a23),
                                kv::e4m3x2_to_f16x2(a23 >> 16)};
        const uint32_t b1[4] = {kv::e4m3x2_to_f16x2(b01), kv::e4m3x2_to_f16x2(b01 >> 16), kv::e4m3x2_to_f16x2(b23),
                                kv::e4m3x2_to_f16x2(b23 >> 16)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int n = 0; n < NT; ++n) ptx::mma_f16(acc[n][4 * w + e], pa[n][i], b0[e], b1[e]);
      }
    }
  };

  // The lane's part of a row: columns tig * D / 4 .. + D / 4 - 1, the first half from the even
  // column of the accumulators, the second from the odd one.
  auto end_item = [&](bool whole, int slot) {
    const int64_t n_rows = static_cast<int64_t>(seq.rows) * p.group;
    const float back = v_ref * (1.0f / kPScale);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < kRl; ++r) {
        float sum = l[n][r];
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        const int local = n * (TWO ? 8 : 16) + r * 8 + gid;
        const int64_t rho = row_q + local;
        if (rho >= n_rows) continue;
        const float f2 = whole ? (sum == 0.0f ? 0.0f : back / sum) : back;
        float* const part =
            p.part_o + ((worker * 2 + slot) * RT + local) * D + tig * (D / 4);
        const int64_t t = rho / p.group;
        const int64_t out = (seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
#pragma unroll
          for (int j = 0; j < kNd; j += 4) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = (TWO ? acc[n][j + e][odd] + acc[n][j + e][2 + odd] : acc[n][j + e][2 * r + odd]) * f2;
            const int col = odd * kNd + j;
            if (whole) store_row4(p, out * D + tig * (D / 4) + col, x[0], x[1], x[2], x[3]);
            else *reinterpret_cast<float4*>(part + col) = make_float4(x[0], x[1], x[2], x[3]);
          }
        if (tig == 0) {
          if (whole) p.lse[out] = sum == 0.0f ? -INFINITY : (m[n][r] + log2f(sum)) * kLn2;
          else p.part_ml[(worker * 2 + slot) * RT + local] = make_float2(m[n][r], sum);
        }
      }
  };

  int st = 0;
  uint32_t parity = 0;
  bool first = true;       // the item at hand is the one the share begins in
  int item_from = c.g;     // first granule of it that is ours
  bool ok = true;
  begin_item();
  while (left > 0) {
    if (!sync::wait_warp(bars + st * 8, parity, ctl, kv::kSiteWait)) {
      ok = false;
      break;
    }
    const int key0 = c.g * kKeys;
    if (key0 + kKeys <= lim_min) granule(st, No{});
    else if (key0 < lim_max) granule(st, Yes{});
    __syncwarp();
    if (to_issue > 0) issue(st);
    if (++st == kSt) {
      st = 0;
      parity ^= 1u;
    }
    --left;
    ++c.g;
    if (c.g == c.gpi || left == 0) {
      const bool whole = item_from == 0 && c.g == c.gpi;
      end_item(whole, first || item_from != 0 ? 0 : 1);
      if (left > 0) {
        c.g = 0;
        item_from = 0;
        // the first item keeps slot 0 even where the share begins at its first granule
        first = false;
        if (++c.block == c.blocks) {
          c.block = 0;
          if (++c.head == p.hkv) next_seq<RT>(p, c, seq);
        }
        begin_item();
      }
    }
  }
  if (!ok) {
    // copies in flight must not outlive the block: `left` granules are waited for, as many as stages
    for (int i = 0; i < kSt && i < left; ++i) {
      sync::wait_drain(bars + st * 8, parity, p.timeout_ns);
      if (++st == kSt) {
        st = 0;
        parity ^= 1u;
      }
    }
  }
}

struct CombineParams {
  Params p;
  int64_t most;  // workers of the first kernel
};

// WPR warps per (row, query head): each goes over every WPR-th partial.
template <int D, int RT, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 256 : WPR * 32) kv_attn_combine_kernel(const __grid_constant__ CombineParams cp) {
  const Params& p = cp.p;
  constexpr int kN = D / 32;
  __shared__ float sh_o[WPR][D];
  __shared__ float2 sh_ml[WPR];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t id = WPR == 1 ? static_cast<int64_t>(blockIdx.x) * 8 + warp : static_cast<int64_t>(blockIdx.x);
  const int64_t row = id / p.hq;
  const int h = static_cast<int>(id - row * p.hq);
  if (row >= p.rows.n_rows) return;
  const int b = kv::find_seq(p.rows.n_seqs, row, lane, [&](int i) { return kv::row_at(p.rows, i); });
  const Seq seq = seq_of<RT>(p, b);
  if (row < seq.r0 || row >= seq.r0 + seq.rows) return;
  const int head = h / p.group;
  const int64_t rho = (row - seq.r0) * p.group + (h - head * p.group);
  const int64_t block = rho / RT;
  const int local = static_cast<int>(rho - block * RT);
  ptx::wait_dependencies();
  const int64_t W = p.plan[p.rows.n_seqs], n = workers(W, cp.most);
  const int64_t from = p.plan[b] + (head * static_cast<int64_t>(seq.blocks) + block) * seq.gpi;
  const int64_t w0 = worker_of(W, n, from), w1 = worker_of(W, n, from + seq.gpi - 1);
  if (w0 == w1) return;  // finished by its worker
  auto place = [&](int64_t w) { return (w * 2 + (share(W, n, w) < from ? 1 : 0)) * RT + local; };

  const int sub = WPR == 1 ? 0 : warp;
  float top = -INFINITY, sum = 0.0f;
  float acc[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
  for (int64_t base = w0 + sub; base <= w1; base += 32 * WPR) {
    const int64_t mine = base + static_cast<int64_t>(lane) * WPR;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (mine <= w1) ml = p.part_ml[place(mine)];
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
    const int64_t many = (w1 - base) / WPR + 1;
    const int count = many < 32 ? static_cast<int>(many) : 32;
#pragma unroll 8
    for (int i = 0; i < count; ++i) {
      const float wi = __shfl_sync(kFull, wt, i);
      const float* src = p.part_o + place(base + static_cast<int64_t>(i) * WPR) * D + lane * kN;
      if constexpr (kN == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(wi, v.x, acc[0]), acc[1] = fmaf(wi, v.y, acc[1]);
        acc[2] = fmaf(wi, v.z, acc[2]), acc[kN - 1] = fmaf(wi, v.w, acc[kN - 1]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(wi, v.x, acc[0]), acc[1] = fmaf(wi, v.y, acc[1]);
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int j = 0; j < kN; ++j) sh_o[warp][lane * kN + j] = acc[j];
    if (lane == 0) sh_ml[warp] = make_float2(top, sum);
    __syncthreads();
    if (warp != 0) return;
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
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t out = row * p.hq + h;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int64_t at = out * D + lane * kN + j;
    if (p.o_bf16) static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(acc[j] * inv);
    else static_cast<float*>(p.o)[at] = acc[j] * inv;
  }
  if (lane == 0) p.lse[out] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The variant for a call: by the query rows that a sequence has on average.
struct Plan {
  int nt;
  bool two;
  int rows;      // RT
  int64_t grid;
  int64_t plan_off, ml_off, o_off, bytes;
};
Plan plan_of(const cp_kv_attn_desc& d, int sms) {
  Plan r;
  const int64_t group = d.hq / d.cache.hkv, seqs = d.rows.n_seqs > 0 ? d.rows.n_seqs : 1;
  const int64_t per = (d.rows.n_rows + seqs - 1) / seqs * group;
  const bool narrow = d.in_dtype == CP_BF16 && d.o_dtype == CP_BF16;
  r.two = per <= 8 || !narrow;
  r.nt = per <= (r.two ? 8 : 16) ? 1 : 2;
  r.rows = r.nt * (r.two ? 8 : 16);
  const int64_t most = ((static_cast<int64_t>(d.rows.max_pages) * d.cache.page_size + kKeys - 1) / kKeys) * d.cache.hkv *
                       (seqs + d.rows.n_rows * group / r.rows);
  r.grid = most < sms ? (most < 1 ? 1 : most) : sms;
  const int64_t slots = r.grid * 8 * 2 * r.rows;
  r.plan_off = 0;
  r.ml_off = (seqs + 1) * 8;
  r.o_off = (r.ml_off + slots * 8 + 255) / 256 * 256;
  r.bytes = r.o_off + slots * d.cache.d * 4;
  return r;
}

template <int D, int NT, bool TWO>
cp_status run(const Params& p, const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv, int64_t items,
              cudaStream_t s) {
  using S = Shape<D, NT, TWO>;
  const int smem = 1024 + S::kPlanOff + (p.rows.n_seqs + 1) * 8;
  cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<D, NT, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "kv_attn_kernel attribute");
  kv_attn_kernel<D, NT, TWO><<<static_cast<unsigned>(pl.grid), S::kWarps * 32, smem, s>>>(p, mk, mv);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "kv_attn_kernel launch");
  CombineParams cp{p, pl.grid * S::kWarps};
  // with few items each is cut into many partials: more warps for each output row
  const int64_t parts = cp.most / (items < 1 ? 1 : items), outs = p.rows.n_rows * p.hq;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  if (parts > 16) {
    cfg.gridDim = dim3(static_cast<unsigned>(outs));
    cfg.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&cfg, kv_attn_combine_kernel<D, S::kRows, 8>, cp);
  } else {
    cfg.gridDim = dim3(static_cast<unsigned>((outs + 7) / 8));
    cfg.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&cfg, kv_attn_combine_kernel<D, S::kRows, 1>, cp);
  }
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "kv_attn_combine_kernel launch");
}

template <int D>
cp_status run_d(const Params& p, const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv, int64_t items,
                cudaStream_t s) {
  if (pl.two) return pl.nt == 1 ? run<D, 1, true>(p, pl, mk, mv, items, s) : run<D, 2, true>(p, pl, mk, mv, items, s);
  return pl.nt == 1 ? run<D, 1, false>(p, pl, mk, mv, items, s) : run<D, 2, false>(p, pl, mk, mv, items, s);
}

}  // namespace

int64_t kv_attn_workspace(const cp_kv_attn_desc& d, int num_sms) { return plan_of(d, num_sms).bytes; }

cp_status launch_kv_attn(const cp_kv_attn_desc& d, float scale, int64_t timeout_ns, int num_sms, cudaStream_t s) {
  const Plan pl = plan_of(d, num_sms);
  const cp_kv_cache& c = d.cache;
  const int64_t lines = c.n_pages * c.hkv * c.page_size * c.d / 128;
  const int box = (c.page_size < kKeys ? c.page_size : kKeys) * c.d / 128;
  CUtensorMap mk, mv;
  if (!encode_map_bytes(&mk, c.k, lines, box) || !encode_map_bytes(&mv, c.v, lines, box)) {
    set_error("cp_kv_cache_attn: tensor map encoding failed");
    return CP_ERR_CUDA;
  }
  if (d.rows.n_rows * d.hq > 0x7fffffff) {
    set_error("cp_kv_cache_attn: too many rows");
    return CP_ERR_INVALID_ARG;
  }
  uint8_t* const ws = static_cast<uint8_t*>(d.workspace);
  Params p{};
  p.scale[0] = c.k_scale;
  p.scale[1] = c.v_scale;
  p.rows = d.rows;
  p.n_pages = c.n_pages;
  p.q = d.q;
  p.o = d.o;
  p.lse = d.lse;
  p.q_first = d.q_first;
  p.hq = d.hq;
  p.hkv = c.hkv;
  p.group = d.hq / c.hkv;
  p.page = c.page_size;
  p.page_log2 = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.q_bf16 = d.in_dtype == CP_BF16;
  p.o_bf16 = d.o_dtype == CP_BF16;
  p.stall = (d.flags & CP_FLAG_TEST_STALL) != 0;
  p.scale_log2 = scale * kLog2e;
  p.kv_pos = d.kv_pos;
  p.status = d.status;
  p.timeout_ns = timeout_ns;
  p.plan = reinterpret_cast<int64_t*>(ws + pl.plan_off);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + pl.o_off);
  const int64_t seqs = d.rows.n_seqs;
  const int64_t items = (seqs + d.rows.n_rows * p.group / pl.rows) * c.hkv;
  return c.d == 128 ? run_d<128>(p, pl, mk, mv, items, s) : run_d<64>(p, pl, mk, mv, items, s);
}

}  // namespace cpattn

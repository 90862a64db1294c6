// Attention of a batch's new tokens over the paged 4-bit cache (cp_kv4_cache_attn): the kernels and their launches.
// kv4_attn.cu chooses among them; kv4_attn_d64.cu and kv4_attn_d128.cu compile them.
//
// Per (sequence, KV head) the g = hq / hkv query heads of the sequence's rows are one block of query rows:
//   s_ij = log2 e * scale * (q_i . k_j),  p_ij = 2^(s_ij - m_i),  O_i = sum_j p_ij v_j / l_i,
//   LSE_i = ln 2 (m_i + log2 l_i),        l_i = sum_j p_ij,
// k_j and v_j being e2m1 numbers times a scale for each 16 of them, which f16 holds exactly.
//
// Work split.  As over the 8-bit cache (kv_split.cuh, kv_attn.cuh): granules of 4096 / D keys, equal shares of
// consecutive ones for every warp, which copies ahead into a ring of its own; partials joined by a second kernel
// (kv_sum.cu).  For few short rows (SOLO) a block or a cluster of blocks an item.  Two granules share a stage of the ring,
// its wait and its copies: the upkeep of single ones was a quarter of the instructions (83 -> 74 us on the batch below, as it was then).
//
// Products.  mma.sync m16n8k16 with f16 operands, transposed, S^T = K Q^T and O^T = V^T P^T, so that 8 query rows fill an
// operand.  e2m1 becomes f16 by one instruction for two numbers and is multiplied by its scale in pairs, which is exact
// (kv4_common.cuh): 2 + 2 instructions for 4 numbers of K and as many, and a half more to put two keys' nibbles side by
// side, of V.  The 4-bit and 8-bit tensor products take no operands of these scales and precision: queries and weights
// would have to be rounded to 4 or 8 bits.
//
// Precision.  A query row is scaled by a power of two to at most 2^15; as f16 a bf16 row is then exact (over 2^28 of range),
// an fp32 row is split into a high and a low part, 22 bits.  Weights are held relative to a whole number m_i that is at
// most kSlack below the row's largest score, times 2^12: one f16 part for a bf16 output (off by 2^-11 at most, against the
// output's 2^-8), two for an fp32 one.  f16 ends at 2^-24, so a weight is off by 2^-37 of the row's largest besides.
// Sums, maxima and the accumulators are fp32; l is a sum of granules' sums, since single weights vanish next to a heavy token's
// (8 x 90000-131072 tokens, 64/8, D = 64, over 16 draws: 4.1e-7 to 1.4e-6 relative to the exact outputs key by key, 3.8e-7 to
// 4.2e-7 so, in 0.5 us more).
//
// Bound.  Each cached byte is used for twice as many products as in the 8-bit cache, and conversions and scales are half
// of some 580 instructions for a granule and tile of rows: the SMs issue at 57 % of their rate and the ALU pipe is busy for
// 49 % of the time, beside memory at two thirds of its rate.  Measured (GB300, in a graph): 64 x 256-8192 tokens, 32/8
// heads, D = 128, bf16: 70 us for 328 MB, 4.7 TB/s (the 8-bit cache: 86): copies begin at 4 us, the first data are there
// at 8, the warps end at 53 to 65 and the second kernel at 69; 6 TB/s between.  8 x 90000-131072, 64/8, D = 64, fp32
// partials: 115 us for 513 MB, 4.4 TB/s; 16 x 2-6 rows over 1000-20000, 32/8, D = 128: 98 us; one token over 1000: 8 us.
// Slower: K and V in slots of their own with 16 warps (73, 118 and 122 us: they spill or hold less in flight).
#pragma once

#include "kv4_tile.cuh"

namespace cpattn {
namespace kvattn {

// What an item costs besides its granules: its end and the next one's begin take a warp 3 to 5 us, a granule of the two
// long cases below 1.3.  At 1 the warps with many short items ended last, 8 us behind the others; 1 / 2 / 3 / 4, us: the
// batch 73.7 / 69.5 / 69.5 / 69.6, 16 x 2-6 rows 99.6 / 100.2 / 97.0 / 96.0, 26 other calls in the mean 13.9 at each.
constexpr int kSetup = 3;
constexpr int kPExp = 12;          // P operands are at most 2^(kPExp + kSlack) = 32768 and f16's largest is 65504
constexpr float kPUnit = 4096.0f;  // 2^kPExp
constexpr float kSlack = 3.0f;     // largest s - m
// m goes by scores that are rounded to fp32 and weights by fma(product, factor, -m), which is not: they differ by 2^-4 at most
// where |m| is below kLarge, but by 8 from 2^27 on.  So from kLarge on m is set 2 to 4 fp32 steps below the score, the exponent
// stays at or above 0 for the largest, and ends at kMost, below which f16 holds the weight: scores of a large magnitude that
// are some steps of fp32 apart, which is less than they are off, count as equal.  (Ending the exponents costs 1 to 1.6 % of the
// batch and the 16 sequences above and 0 to 1 % of other calls; a path of their own for such rows, with rounded scores, 2 to 4 %.)
constexpr float kLarge = 1048576.0f;
constexpr float kMost = 3.9f;
__device__ __forceinline__ float at_most(float x, float most) {  // NaN stays
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(most));
  return y;
}

// QP, PP: f16 parts of a query element and of a weight.  NT: tiles of 8 query rows.
template <int D, int NT, int QP, int PP>
struct Shape4 {
  // More warps hide more latency; registers (O takes NT D / 4) bound their number (10 warps of two tiles spill: 122 us where
  // 8 take 110).
  static constexpr bool kHeavy = NT * D >= 256 || NT * QP >= 4;
  static constexpr int kWarps = kHeavy ? 8 : 12;
  static constexpr int kRows = NT * 8;  // RT
  // The tensor cores' fp32 sums are truncated, an error that grows with the length of a sum: the accumulators are added
  // to others every kFlush granules, in registers where there are some left (kHold), else in the workspace.  Every 2 or 4
  // with kHold, on the 8 long sequences above, when l was a sum of keys: 4.2e-7 to 7.0e-7 or 5.5e-7 to 7.5e-7 relative to
  // the exact outputs, and 0.3 us between them.
  static constexpr bool kHold = PP == 2 && D == 64 && NT == 1;
  static constexpr int kFlush = PP == 1 ? 64 : kHold ? 2 : D == 128 ? 16 : 8;
  static constexpr int kKeys = Granule<D>::kKeys;
  static constexpr int kSteps = Granule<D>::kSteps;
  static constexpr int kRow = Granule<D>::kRow;
  static constexpr int kHalf = Granule<D>::kHalf;
  static constexpr int kStage = 2 * Granule<D>::kPair;  // keys, values
  static constexpr bool kQSmem = D == 128 && NT >= 2;  // query operands in shared memory
  static constexpr int kStages = kWarps == 8 && !kQSmem ? 3 : 2;
  static constexpr int kQBytes = kQSmem ? NT * QP * (D / 16) * 256 : 0;
  static constexpr int kWarpBytes = kStages * kStage + kQBytes;
  // behind the warps' parts: barriers, control.  The plan is looked at before the first copies and lies where they go.
  static constexpr int kBarOff = kWarps * kWarpBytes;  // [warp][stage] + stall
  static constexpr int kCtlOff = kBarOff + (kWarps * kStages + 1) * 8;
  static constexpr int kScanOff = (kCtlOff + 8 + 15) / 16 * 16;  // [warp] 8 bytes
  static constexpr int kBytes = kScanOff + 16 * 8;
  static_assert(kBarOff >= (CP_KV_MAX_SEQS + 1) * 8, "the plan fits the rings");
};

// SOLO: 0 split, 1 one block an item, 2 a cluster of p.cluster blocks an item.
template <int D, int NT, int QP, int PP, int SOLO>
__global__ void __launch_bounds__(Shape4<D, NT, QP, PP>::kWarps * 32, 1)
    kv4_attn_kernel(const __grid_constant__ Params p) {
  using S = Shape4<D, NT, QP, PP>;
  constexpr int RT = S::kRows;
  constexpr int kMt = D / 16;  // 16-row tiles of O^T; also steps of 16 dimensions of S
  constexpr int kCols = D / 8; // columns of O that a lane holds, for two query rows
  constexpr int kSt = S::kStages, kSteps = S::kSteps, kKeys = S::kKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((128u - (ptx::smem_u32(smem_raw) & 127u)) & 127u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  int64_t* const plan = reinterpret_cast<int64_t*>(smem);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + S::kCtlOff);
  const uint32_t base = ptx::smem_u32(smem);
  const uint32_t ring = base + warp * S::kWarpBytes;
  const uint32_t q_smem = ring + kSt * S::kStage;
  const uint32_t bars = base + S::kBarOff + warp * kSt * 8;
  const uint32_t stall_bar = base + S::kBarOff + S::kWarps * kSt * 8;

  if (lane == 0) {
    for (int i = 0; i < kSt; ++i) ptx::mbar_init(bars + i * 8, 1);
    if (warp == 0) {
      ptx::mbar_init(stall_bar, 1);
      *abort_flag = 0;
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
  int left;      // numbers of the share from the cursor on; at most 1e12 / (8 * 152) where the grid is full
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
    const int64_t W = plan[n_seqs];
    const int64_t n_workers = workers(p, W, static_cast<int64_t>(gridDim.x) * S::kWarps);
    const bool idle = worker >= n_workers || stalled;
    left = 0;
    inside = false;
    if (!idle) {
      const int64_t lo = share(W, n_workers, worker), hi = share(W, n_workers, worker + 1);
      left = static_cast<int>(hi - lo);
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
    }
    ptx::fence_proxy_async_smem();
    __syncthreads();  // the plan has been read: the copies may begin
    if (stalled) sync::wait_warp(stall_bar, 0, ctl, kv::kSiteWait);
    if (left <= 0) return;
  }
  bool ok = true;
  if (stalled) {  // the block's other warps still meet it
    ok = sync::wait_warp(stall_bar, 0, ctl, kv::kSiteWait);
    left = 0;
  }
  const int g_first = c.g, solo_left = left;  // of a block of rows, where SOLO
  Cursor f = c;         // where the copies are
  int to_issue = left;
  Feed<D, 2> feed{c.b, c.head, seq.keys, -32, -1};

  // Starts the copies of the next granules into stage `st`.
  auto issue = [&](int st) {
    const int n = together(f.g, min(f.gpi, f.g + to_issue));
    feed.stage(p, lane, f.g, n, ring + st * S::kStage, bars + st * 8);
    to_issue -= n;
    f.g += n;
    if (f.g == f.gpi) {
      to_issue -= kSetup;
      if (to_issue > 0) {
        f.g = 0;
        if (++f.block == f.blocks) {
          f.block = 0;
          if (++f.head == p.hkv) {
            Seq s{};
            next_seq<D, RT>(p, f, s);
            feed.b = f.b;
            feed.keys = s.keys;
            feed.window = -32;
          }
          feed.head = f.head;
        }
      }
    }
  };

  uint32_t qf[S::kQSmem ? 1 : NT * QP][S::kQSmem ? 1 : kMt][2];
  // of the lane's two query rows 2 tig, 2 tig + 1 in each tile
  float fac[NT][2], m[NT][2], l[NT][2];
  int lim[NT][2];
  float acc[NT][kMt][4];
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
      const int64_t at = ((seq.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group)) * D;
      int lm = live ? visible(p, seq.tokens, seq.pos0 + t) : -1;
      if (live) {
        lmin = min(lmin, lm);
        lmax = max(lmax, lm);
      }
      float f;
      if constexpr (S::kQSmem) {
        uint32_t x[QP][kMt][2];
        f = query_operands<D, QP>(p, at, live, tig, x);
#pragma unroll
        for (int part = 0; part < QP; ++part)
#pragma unroll
          for (int j = 0; j < kMt; ++j)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_smem + (((n * QP + part) * kMt + j) * 32 + lane) * 8),
                         "r"(x[part][j][0]), "r"(x[part][j][1])
                         : "memory");
      } else {
        f = query_operands<D, QP>(p, at, live, tig, &qf[n * QP]);
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
    flushed = false;
    since = 0;
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < kMt; ++j) held[j][0] = held[j][1] = held[j][2] = held[j][3] = 0.0f;
    }
  };

  // Where some row of the block does not see all keys of the granule: values that no row sees count as zero, by
  // their scales (0 * NaN would not vanish), and NaN among values that only some of the rows see go to those rows'
  // accumulators and are taken out.
  auto mask_values = [&](uint32_t tile, int key0) {
    const int first = max(lim_min - key0, 0);  // below kKeys
    bool odd = false;
#pragma unroll
    for (int k = lane; k < kKeys; k += 32) {
      const uint32_t at = tile + k * S::kRow + D / 2;
      uint32_t v[D / 64];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        if (key0 + k >= lim_max) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 4 * j), "r"(0) : "memory");
        v[j] = lds32(at + 4 * j);
        if (k >= first) odd |= __vcmpgeu4(v[j], 0xf8f8f8f8u) != 0u;
      }
    }
    __syncwarp();
    if (__any_sync(kFull, odd)) {
#pragma unroll 1
      for (int k = first; k < kKeys && key0 + k < lim_max; ++k) {
        const uint32_t at = tile + k * S::kRow + D / 2 + (D == 128 ? gid : gid >> 1);
        const bool nan = lds8(at) >= 0xf8u;
        __syncwarp();
        if (nan) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(0)) : "memory");
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (nan && key0 + k < lim[n][r]) {
#pragma unroll
              for (int j = 0; j < kMt; ++j) acc[n][j][r] = acc[n][j][2 + r] = __int_as_float(0x7fffffff);
            }
      }
    }
    ptx::fence_proxy_async_smem();  // before the next copies into the stage
    __syncwarp();
  };

  // One granule; masked: some of its keys are not seen by some row.  Masks and tiles without rows are uniform
  // branches and predicates, not variants: with four variants a warp's items of a few granules ran at the
  // speed of the instruction cache (62 x 16 items of some 3 granules, up to 60 rows, D = 64: 86 us, more than half
  // of the stalls; 55 with one path, and 16-row items of 8192 tokens 102 against 106).
  auto granule = [&](uint32_t tile, int key0) {
    const bool masked = key0 + kKeys > lim_min;
    const uint32_t values = tile + Granule<D>::kPair;
    auto product = [&](int n, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
      // tiles without rows are left out where that is cheaper than asking (D = 64: 1 to 4 %; at D = 128 asking costs 2 %)
      if (n == 0 || D == 128) ptx::mma_f16(d, a, b0, b1);
      else ptx::mma_f16_if(d, a, b0, b1, live > n);
    };
    if (masked) mask_values(values, key0);
    // S^T: s[n][i][2 u + r] is key key_at(i, u, gid) for query row 2 tig + r of tile n.  The low parts of fp32 queries are
    // summed on their own: as part of the larger sums each of their truncated additions would cost as much as one of those
    // (7 x 0-8191 tokens, 32/32, D = 128: 1.8e-6 relative to the exact outputs, 1.4e-6 so, in the same time).
    float s[NT][kSteps][4];
#pragma unroll
    for (int i = 0; i < kSteps; i += 2) {
      float z[QP][NT][2][4];
#pragma unroll
      for (int part = 0; part < QP; ++part)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[part][n][0][e] = z[part][n][1][e] = 0.0f;
      key_operands<D>(tile, i, gid, tig, [&](int j, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
#pragma unroll
        for (int part = 0; part < QP; ++part)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (S::kQSmem) {
              const uint2 q = ptx::lds64(q_smem + (((n * QP + part) * kMt + j) * 32 + lane) * 8);
              product(n, z[part][n][0], a, q.x, q.y);
              product(n, z[part][n][1], b, q.x, q.y);
            } else {
              product(n, z[part][n][0], a, qf[n * QP + part][j][0], qf[n * QP + part][j][1]);
              product(n, z[part][n][1], b, qf[n * QP + part][j][0], qf[n * QP + part][j][1]);
            }
          }
      });
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][i + h][e] = QP == 2 ? z[0][n][h][e] + z[QP - 1][n][h][e] : z[0][n][h][e];
    }
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (key0 + key_at<D>(i, u, gid) >= lim[n][r]) s[n][i][2 * u + r] = -INFINITY;
    }
    // Maxima.  s and top keep the products; a score is s * fac (fac > 0).  m is a whole number, so rescaling is exact, and it
    // moves only where a score is more than kSlack above it: mostly a comparison by every lane on its own is enough.
    bool grew = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[n][r] = fmaxf(s[n][0][r], s[n][0][2 + r]);
#pragma unroll
        for (int i = 1; i < kSteps; ++i) top[n][r] = fmaxf(top[n][r], fmaxf(s[n][i][r], s[n][i][2 + r]));
        grew |= fmaf(top[n][r], fac[n][r], -m[n][r]) > kSlack;  // false where both are -inf
      }
    if (__any_sync(kFull, grew)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float c[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = top[n][r] * fac[n][r];
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
          x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
          // an infinite score makes m infinite and its row NaN
          const float low = fabsf(x) >= kLarge && x < INFINITY ? fmaf(fabsf(x), -0x1p-22f, x) : x;
          const float now = x > m[n][r] + kSlack ? fmaxf(floorf(low), m[n][r]) : m[n][r];
          c[r] = now > m[n][r] ? ex2(m[n][r] - now) : 1.0f;
          m[n][r] = now;
          l[n][r] *= c[r];
        }
#pragma unroll
        for (int j = 0; j < kMt; ++j) {
          acc[n][j][0] *= c[0];
          acc[n][j][1] *= c[1];
          acc[n][j][2] *= c[0];
          acc[n][j][3] *= c[1];
          if constexpr (kHold) {
            held[j][0] *= c[0];
            held[j][1] *= c[1];
            held[j][2] *= c[0];
            held[j][3] *= c[1];
          }
        }
      }
    }
    // Weights as operands, times 2^kPExp: pb[n][part][i][u], keys 2 tig, 2 tig + 1 of group u for query row gid.  The power
    // of two is not part of the exponent's argument, whose rounding would be that of a number of 12.
    uint32_t pb[NT][PP][kSteps][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // two rows at a time
      const uint64_t ref = ptx::f2_pack(m[n][0] == -INFINITY ? 0.0f : -m[n][0], m[n][1] == -INFINITY ? 0.0f : -m[n][1]);
      const uint64_t both = ptx::f2_pack(fac[n][0], fac[n][1]), unit = ptx::f2_pack(kPUnit, kPUnit);
      // the granule's weights are summed on their own: next to a large l most of them would be less than half a step
      uint64_t sum = 0;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float w[2];
          ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[n][i][2 * u], s[n][i][2 * u + 1]), both, ref), w[0], w[1]);
          const uint64_t w2 = ptx::f2_pack(ex2(at_most(w[0], kMost)), ex2(at_most(w[1], kMost))), x2 = ptx::f2_mul(w2, unit);
          sum = i == 0 && u == 0 ? w2 : ptx::f2_add(sum, w2);
          float a, b;
          ptx::f2_unpack(x2, a, b);
          const uint32_t h = to_f16x2(a, b);
          pb[n][0][i][u] = ptx::transpose8x8(h);
          if constexpr (PP == 2) {
            const float2 back = from_f16x2(h);
            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(back.x, back.y), ptx::f2_pack(-1.0f, -1.0f), x2), a, b);
            pb[n][1][i][u] = ptx::transpose8x8(to_f16x2(a, b));
          }
        }
      ptx::f2_unpack(ptx::f2_add(ptx::f2_pack(l[n][0], l[n][1]), sum), l[n][0], l[n][1]);
    }
    // O^T += V^T P^T: rows gid and gid + 8 of tile w are columns kCols gid + 2 w and + 1 of O
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      value_operands<D>(values, i, gid, tig, [&](int w, const uint32_t (&a)[4][4]) {
#pragma unroll
        for (int part = 0; part < PP; ++part)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) product(n, acc[n][w + j], a[j], pb[n][part][i][0], pb[n][part][i][1]);
      });
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
  // part_o [RT][D], part_ml [RT], with l between 1 and 2 where |m| is below kLarge.
  auto end_item = [&](bool whole, float* part_o, float2* part_ml) {
    const int n_rows = seq.rows * p.group;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[n][r];
        sum += __shfl_xor_sync(kFull, sum, 4);
        sum += __shfl_xor_sync(kFull, sum, 8);
        sum += __shfl_xor_sync(kFull, sum, 16);
        if (m[n][r] == INFINITY) sum = __int_as_float(0x7fffffff);  // a finite product that is no finite score leaves 0
        const int local = n * 8 + 2 * tig + r;
        const int rho = row_q + local;
        if (rho >= n_rows) continue;
        const float keep = keep_of(n, r);
        // the exponent of l goes to m, but for an m that might not hold it
        const int up =
            fabsf(m[n][r]) >= kLarge ? 0 : min(max(static_cast<int>(__float_as_uint(sum) >> 23 & 255u) - 127, -100), 126);
        const float norm = sum * kv::pow2(-up), ref = m[n][r] + static_cast<float>(up);
        const float back = kv::pow2(-kPExp - up);
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
      const int n = together(c.g, min(c.gpi, c.g + left));
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int key0 = (c.g + i) * kKeys;
        if (key0 < lim_max) granule(ring + st * S::kStage + i * S::kHalf, key0);
      }
      __syncwarp();
      if (to_issue > 0) issue(st);
      else --in_flight;
      if (++st == kSt) {
        st = 0;
        parity ^= 1u;
      }
      left -= n;
      c.g += n;
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
      } else if ((since += n) >= S::kFlush && (kHold || !SOLO)) {  // 16 granules need no more
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

template <int D, int NT, int QP, int PP>
cp_status run4(const Params& p, const Plan& pl, int64_t items, int num_sms, cudaStream_t s) {
  using S = Shape4<D, NT, QP, PP>;
  constexpr int smem = 128 + S::kBytes;
  static_assert(smem <= 232448, "shared memory of a block");
  const auto kernel = !pl.solo           ? kv4_attn_kernel<D, NT, QP, PP, 0>
                      : pl.cluster == 1 ? kv4_attn_kernel<D, NT, QP, PP, 1>
                                        : kv4_attn_kernel<D, NT, QP, PP, 2>;
  // The limit is the function's, not the call's: always the same, for other host threads launch the kernel too.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "kv4_attn_kernel attribute");
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
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess) return cuda_fail(e, "kv4_attn_kernel launch");
  if (pl.solo) return CP_OK;
  return launch_sum<D, S::kRows>(p, pl.grid * S::kWarps, items, num_sms, s);
}

template <int D>
cp_status run4_d(const Params& p, const Plan& pl, int64_t items, int num_sms, cudaStream_t s) {
  if constexpr (D == 128)
    if (pl.nt == 3) return run4<D, 3, 1, 1>(p, pl, items, num_sms, s);
  if (pl.pp == 1)
    return pl.nt == 1 ? run4<D, 1, 1, 1>(p, pl, items, num_sms, s) : run4<D, 2, 1, 1>(p, pl, items, num_sms, s);
  if (pl.qp == 1)
    return pl.nt == 1 ? run4<D, 1, 1, 2>(p, pl, items, num_sms, s) : run4<D, 2, 1, 2>(p, pl, items, num_sms, s);
  return pl.nt == 1 ? run4<D, 1, 2, 2>(p, pl, items, num_sms, s) : run4<D, 2, 2, 2>(p, pl, items, num_sms, s);
}

}  // namespace kvattn
}  // namespace cpattn

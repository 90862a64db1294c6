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

#include "kv_split.cuh"
#include "sync.cuh"

namespace cpattn {
namespace kvattn {

constexpr int kSetup = 1;            // what an item costs besides its granules
constexpr int kPExp = 15;            // P operands are below 2^(kPExp + kTop) = 65490 and f16's largest is 65504
constexpr float kTop = 0.999f;       // largest s + log2 vs - base - m
constexpr float kNear = 40.0f;       // largest |log2 vs - base| but for base = kFarBase
constexpr int kFarBase = 40;
constexpr float kNoBase = -10000.0f;

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
      float sum[2];  // of the granule: next to a large l most weights would be less than half a step
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float pv[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float w = ex2(fmaf(s[n][i][2 * u + r], f2[n][r][i], -ref[r]));
            sum[r] = i == 0 && u == 0 ? w : sum[r] + w;
            pv[r] = w * vf[i];
          }
          const uint32_t h = to_f16x2(pv[0], pv[1]);
          pb[n][0][i][u] = ptx::transpose8x8(h);
          if constexpr (PP == 2) {
            const float2 back = from_f16x2(h);
            pb[n][1][i][u] = ptx::transpose8x8(to_f16x2(pv[0] - back.x, pv[1] - back.y));
          }
        }
      l[n][0] += sum[0];
      l[n][1] += sum[1];
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
  return launch_sum<D, S::kRows>(p, pl.grid * S::kWarps, items, num_sms, s);
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

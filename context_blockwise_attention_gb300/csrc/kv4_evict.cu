// Eviction from the paged 4-bit cache by gathered weight (cp_kv4_cache_evict).
//
// Of a sequence's n tokens the last `recent` stay, and of the others the z = keep - recent with the largest weight
// (summed over the KV heads).  Slots below z keep what stays there; the holes among them are filled, in order, by the
// tokens that stay from z on, and the recent tokens follow at z.  So only as many rows move as are evicted from the
// first z slots, and the recent ones: a batch that exceeds its budget of 4096 by 128 tokens moves 5 % of its cache, where
// closing ranks would move all of it.
//
// First kernel, a block or a cluster of blocks a sequence: every token's sum becomes a whole number of the same order and
// is kept in shared memory (in the workspace where it does not fit); the z-th largest is found by its bits, 11, 11 and 10
// at a time, from histograms that the blocks add up through distributed shared memory; of equal tokens the first stay.
// The weights are read once; the rest is latency, of some ten barriers: of 11 us for 4224 tokens and one block 5 until the
// sums are there, 3 for the three histograms, 2 for the marks; of 18 us for 65536 tokens and 8 blocks the histograms take 4.
// Second kernel: some blocks take the recent tokens of a (sequence, head), which move towards the front by n - keep and
// may overwrite slots that fills came from, in batches that are read before they are written; a warp a token the other
// fills, whose sources and holes do not overlap with anything.  A kernel for each of the two took 2 and 3 us more on the
// cases below, keys and values in the same blocks 1 and 3 us more.
// Measured (GB300, in a graph, with 4 us for copying the weights first): 64 x 4000-4224 tokens to 4096, 8 heads, D = 128:
// 26.5 us (floor 2.7; latency of two kernels); 8 x 20000-65536 to 4096, D = 64: 47.5 us (floor 6.6; filling takes 20, for
// rows of 36 bytes cost the 64 or 96 of the sectors that they touch).
#include <type_traits>

#include "internal.h"
#include "kv4_common.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostInSmem = 40960;  // tokens of a block
constexpr int kAtOnce = 4;          // tokens of a thread whose weights are on their way together
constexpr int kMostCluster = 8;
constexpr int kMoveThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

struct Sequence {  // what the first kernel tells the second
  int32_t n, z, fills, recent;  // recent: rows that move to z; 0 where nothing is evicted
};

struct EvictParams {
  cp_kv4_cache c;
  float* weight;
  const int32_t* tokens;
  const int32_t* table;
  int32_t n_seqs, max_pages, keep, recent, page_log2;
  int32_t* kept;
  int32_t* new_tokens;
  int32_t* status;
  Sequence* seqs;      // workspace: [n_seqs]
  int32_t* holes;      // [n_seqs, keep]; none where keep is as much as the page table has room for
  uint32_t* store;     // [n_seqs, cluster] of room + 3 room / 32 words, where shared memory is too small; else null
  int32_t cluster, room;  // room: tokens of a block, a multiple of 32
  int32_t ordered;     // blocks of the second kernel that move recent tokens
  int32_t per_seq;     // blocks of a sequence that move fills
};

__device__ __forceinline__ int page_of(const EvictParams& p, int b, int token) {
  return __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + (token >> p.page_log2));
}
// Row of a token among the cache's rows for head 0, which are below 2^31.
__device__ __forceinline__ int row_in(const EvictParams& p, int page, int token) {
  return (page * p.c.hkv << p.page_log2) + (token & ((1 << p.page_log2) - 1));
}
__device__ __forceinline__ int row_of(const EvictParams& p, int b, int token) {
  return row_in(p, page_of(p, b, token), token);
}

// A sum of n weights: the rounding errors of the additions are summed apart (Knuth's two-sum) and added at the end.  They are
// rounded too, so before its last rounding the sum is off by (n 2^-24)^2 of itself at most (Ogita, Rump and Oishi's bound;
// 2^-42 for 8 heads): the order of the heads decides only where a sum is that near to the middle between two of fp32.
struct Sum {
  float s = 0.0f, err = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(s, x), y = __fsub_rn(t, s);
    err = __fadd_rn(err, __fadd_rn(__fsub_rn(s, __fsub_rn(t, y)), __fsub_rn(x, y)));
    s = t;
  }
  __device__ __forceinline__ float value() const {
    return fabsf(s) < INFINITY && fabsf(err) < INFINITY ? __fadd_rn(s, err) : s;
  }
};
// Whole numbers in the order of the weights; NaN is below all of them.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Exclusive sums over the block's threads; `all`: of the whole block.
__device__ __forceinline__ int scan(int x, int* scratch, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int in = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, in, o);
    if (lane >= o) in += y;
  }
  __syncthreads();  // scratch has been read
  if (lane == 31) scratch[warp] = in;
  __syncthreads();
  static_assert(kWarps == 32, "a lane reads a warp's sum");
  const int of = scratch[lane];
  all = __reduce_add_sync(kFull, of);
  return static_cast<int>(__reduce_add_sync(kFull, lane < warp ? of : 0)) + in - x;
}

// What `x` is in all blocks of the cluster: the loads are on their way together.
__device__ __forceinline__ void ld_all(const int* x, int cluster, int (&of)[kMostCluster]) {
  const uint32_t at = ptx::smem_u32(x);
#pragma unroll
  for (int r = 0; r < kMostCluster; ++r) {
    of[r] = 0;
    if (r < cluster) of[r] = __float_as_int(ptx::ld_cluster(ptx::cluster_addr(at, r)));
  }
}

// Bit k of a word of tokens: the first `count` of them.
__device__ __forceinline__ uint32_t first_bits(int count) {
  return count <= 0 ? 0u : count >= 32 ? kFull : (1u << count) - 1u;
}

__global__ void __launch_bounds__(kThreads) kv4_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ int hist[3][kBins], totals[kBins];
  __shared__ int scratch[kWarps];
  __shared__ int found[2];   // bin, and how many are in the ones above it
  __shared__ int counts[4];  // this block's: bad, holes, movers
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cluster = p.cluster, b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const auto meet = [&]() {
    if (cluster > 1) ptx::cluster_sync();
    else __syncthreads();
  };
  ptx::wait_dependencies();
  ptx::launch_dependents();
  const int held = p.tokens[b];  // no read-only load: the answer may take its place
  const int n = held < 0 ? 0 : held;
  const bool over = n > static_cast<int64_t>(p.max_pages) << p.page_log2;
  int32_t* const kept = p.kept + static_cast<int64_t>(b) * p.keep;
  // A sequence that stays as it is.
  const auto leave = [&]() {
    // unsigned: keep may be the largest signed number
    for (uint32_t i = rank * kThreads + tid; i < static_cast<uint32_t>(p.keep); i += cluster * kThreads)
      kept[i] = i < static_cast<uint32_t>(n) ? static_cast<int32_t>(i) : -1;
    if (rank == 0 && tid == 0) {
      p.new_tokens[b] = n;
      p.seqs[b] = Sequence{n, 0, 0, 0};
    }
  };
  if (rank == 0 && tid == 0 && (held < 0 || over)) kv::report(p.status, kv::kSiteTokens);
  if (n <= p.keep || over) {  // the same for the whole cluster
    leave();
    return;
  }
  const int old = n - p.recent, z = p.keep - p.recent;
  const int chunk = ((old + cluster - 1) / cluster + 31) / 32 * 32;  // at most room
  const int from = min(rank * chunk, old), mine = min(chunk, old - from), words = (mine + 31) / 32;
  uint32_t* const key = p.store != nullptr ? p.store + static_cast<int64_t>(blockIdx.x) * (p.room + p.room / 32 * 3) : smem;
  uint32_t* const stay = key + p.room;
  int* const hole_rank = reinterpret_cast<int*>(stay + p.room / 32);
  int* const mover_rank = hole_rank + p.room / 32;

  for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  if (tid == 0) counts[0] = 0;
  __syncthreads();
  // Pages of all tokens, the recent ones too, have to be there before anything is changed.
  int bad = 0;
  for (int base = tid; base < mine; base += kAtOnce * kThreads) {
    int row[kAtOnce];
    Sum sum[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int i = base + j * kThreads;
      row[j] = -1;
      if (i < mine) {
        const int page = page_of(p, b, from + i);
        if (page < 0 || page >= p.c.n_pages) bad = 1;
        else row[j] = row_in(p, page, from + i);
      }
    }
#pragma unroll 8
    for (int h = 0; h < p.c.hkv; ++h) {
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (row[j] >= 0) sum[j].add(p.weight[row[j] + (h << p.page_log2)]);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int i = base + j * kThreads;
      if (i < mine) {
        const uint32_t k = order_of(sum[j].value());
        key[i] = k;
        atomicAdd(&hist[0][k >> 21], 1);
      }
    }
  }
  for (int i = old + rank * kThreads + tid; i < n; i += cluster * kThreads) {
    const int page = page_of(p, b, i);
    bad |= page < 0 || page >= p.c.n_pages;
  }
  if (bad) counts[0] = 1;
  meet();  // the first histograms are there too
  bad = counts[0];
  int of[kMostCluster];
  if (cluster > 1) {
    ld_all(&counts[0], cluster, of);
#pragma unroll
    for (int r = 0; r < kMostCluster; ++r) bad |= of[r];
  }
  if (bad) {
    if (cluster > 1) ptx::cluster_sync();  // a block that has ended can be asked no more
    if (rank == 0 && tid == 0) kv::report(p.status, kv::kSitePage);
    leave();
    return;
  }

  // The z-th largest: bits found so far, and how many of the tokens that begin with them stay.
  uint32_t bits = 0;
  int want = z, ties_before = 0;
  if (z > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
      if (pass > 0) {
        const uint32_t above = bits >> (pass == 1 ? 21 : 10);
        for (int i = tid; i < mine; i += kThreads) {
          const uint32_t k = key[i];
          if (k >> (pass == 1 ? 21 : 10) == above) atomicAdd(&hist[pass][k >> shift & (bins - 1)], 1);
        }
      }
      if (pass > 0) meet();
      // A block adds up its part of the bins for all: with every block reading all bins of all others the three passes took
      // 9 us, 4 this way (8 blocks).
      const int part_log2 = 31 - __clz(bins / cluster);
      if (cluster > 1) {
        for (int i = tid; i >> part_log2 == 0; i += kThreads) {
          const int bin = (rank << part_log2) + i;
          ld_all(&hist[pass][bin], cluster, of);
          int total = 0;
#pragma unroll
          for (int r = 0; r < kMostCluster; ++r) total += of[r];
          totals[bin] = total;
        }
        ptx::cluster_sync();
      }
      constexpr int kPer = kBins / kThreads;
      int count[kPer], sum = 0;
      const int per = bins / kThreads;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {  // from the last bin on
        count[j] = 0;
        if (j < per) {
          const int bin = bins - 1 - (tid * per + j);
          if (cluster > 1)
            count[j] = __float_as_int(ptx::ld_cluster(ptx::cluster_addr(ptx::smem_u32(&totals[bin]), bin >> part_log2)));
          else
            count[j] = hist[pass][bin];
        }
        sum += count[j];
      }
      int all, before = scan(sum, scratch, all);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (before < want && want <= before + count[j]) {  // one thread's, one bin's
          found[0] = bins - 1 - (tid * per + j);
          found[1] = before;
        }
        before += count[j];
      }
      __syncthreads();
      bits |= static_cast<uint32_t>(found[0]) << shift;
      want -= found[1];
      __syncthreads();
    }
    // equal tokens of the blocks before
    if (cluster > 1) {
      ld_all(&hist[2][bits & 1023u], rank, of);
#pragma unroll
      for (int r = 0; r < kMostCluster; ++r) ties_before += of[r];
    }
  }

  // What stays, 32 tokens a word; the first `want` of the tokens that equal the z-th largest.
  if (z > 0)
    for (int w = warp; w < words; w += kWarps) {
      const int i = 32 * w + lane;
      const uint32_t k = i < mine ? key[i] : 0u;
      const uint32_t more = __ballot_sync(kFull, i < mine && k > bits), same = __ballot_sync(kFull, i < mine && k == bits);
      if (lane == 0) stay[w] = more, hole_rank[w] = static_cast<int>(same);
    }
  __syncthreads();
  int holes = 0, movers = 0, ties = ties_before;
  for (int base = 0; base < words; base += kThreads) {
    const int w = base + tid;
    uint32_t more = 0, same = 0;
    if (w < words && z > 0) more = stay[w], same = static_cast<uint32_t>(hole_rank[w]);
    int all;
    int left = want - (ties + scan(__popc(same), scratch, all));
    ties += all;
    while (same != 0u && left > 0) {
      more |= same & (0u - same);
      same &= same - 1u;
      --left;
    }
    const uint32_t low = first_bits(z - (from + 32 * w)), in = first_bits(mine - 32 * w);
    const int h = w < words ? __popc(~more & low & in) : 0, m = w < words ? __popc(more & ~low) : 0;
    const int before_h = scan(h, scratch, all);
    if (w < words) {
      stay[w] = more;
      hole_rank[w] = holes + before_h;
    }
    holes += all;
    const int before_m = scan(m, scratch, all);
    if (w < words) mover_rank[w] = movers + before_m;
    movers += all;
  }
  if (tid == 0) counts[1] = holes, counts[2] = movers;
  meet();
  int holes_before = 0, movers_before = 0, fills = holes;
  if (cluster > 1) {
    fills = 0;
    int of_movers[kMostCluster];
    ld_all(&counts[1], cluster, of);
    ld_all(&counts[2], rank, of_movers);
#pragma unroll
    for (int r = 0; r < kMostCluster; ++r) {
      if (r < rank) holes_before += of[r];
      movers_before += of_movers[r];
      fills += of[r];
    }
  }
  int32_t* const list = p.holes + static_cast<int64_t>(b) * p.keep;
  for (int w = warp; w < words; w += kWarps) {
    const int at = from + 32 * w + lane;
    const uint32_t s = stay[w];
    const uint32_t hole = ~s & first_bits(z - (from + 32 * w)) & first_bits(mine - 32 * w);
    if (at < z && (s >> lane & 1u)) kept[at] = at;
    if (hole >> lane & 1u) list[holes_before + hole_rank[w] + __popc(hole & ((1u << lane) - 1u))] = at;
  }
  meet();  // the holes of all blocks; and none is asked for its counts after this
  for (int w = warp; w < words; w += kWarps) {
    const int at = from + 32 * w + lane;
    const uint32_t mover = stay[w] & ~first_bits(z - (from + 32 * w));
    if (mover >> lane & 1u) kept[__ldcg(list + movers_before + mover_rank[w] + __popc(mover & ((1u << lane) - 1u)))] = at;
  }
  for (int i = rank * kThreads + tid; i < p.recent; i += cluster * kThreads) kept[z + i] = old + i;
  if (rank == 0 && tid == 0) {
    p.new_tokens[b] = p.keep;
    p.seqs[b] = Sequence{n, z, fills, p.recent};
  }
}

// Rows move in nine pieces, of 8 bytes at D = 128 and 4 at D = 64.
template <int D>
using Piece = typename std::conditional<D == 128, uint2, uint32_t>::type;

// The recent tokens of a (sequence, head), their keys or their values and weights, and in front of them the fills that come
// from slots which they overwrite: those are among the first fills, as these are in the order of their sources.  A thread
// takes piece t % 10 of token t / 10.  Batch after batch, each read before it is written: a target is never the source of
// a later batch, since the recent ones' are in front of their sources and the fills' in front of z.
template <int D>
__device__ __forceinline__ void move_in_order(const EvictParams& p, int b, int head, bool values) {
  constexpr int kTokens = kMoveThreads / 10, kAhead = 4;
  const Sequence s = p.seqs[b];
  if (s.recent == 0) return;
  const int32_t* const kept = p.kept + static_cast<int64_t>(b) * p.keep;
  const int32_t* const list = p.holes + static_cast<int64_t>(b) * p.keep;
  const int fills = min(s.fills, s.recent), by = s.n - p.keep, mine = threadIdx.x / 10, e = threadIdx.x % 10;
  const bool weight = e == 9;
  uint8_t* const base = weight ? reinterpret_cast<uint8_t*>(p.weight)
                               : static_cast<uint8_t*>(values ? p.c.v : p.c.k) + e * static_cast<int>(sizeof(Piece<D>));
  const int64_t stride = weight ? 4 : kv4::kRow<D>, tokens = static_cast<int64_t>(fills) + s.recent;
  for (int64_t first = 0; first < tokens; first += kTokens * kAhead) {
    Piece<D> x[kAhead];
    uint8_t* to[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = first + j * kTokens + mine;
      to[j] = nullptr;
      if (i < tokens && mine < kTokens && (values || !weight)) {
        const int slot = i < fills ? __ldg(list + i) : s.z + static_cast<int>(i - fills);
        const int source = i < fills ? __ldg(kept + slot) : slot + by;
        if (i < fills && source >= p.keep) continue;  // another block's
        to[j] = base + (row_of(p, b, slot) + (head << p.page_log2)) * stride;
        const uint8_t* const from = base + (row_of(p, b, source) + (head << p.page_log2)) * stride;
        if (weight) *reinterpret_cast<uint32_t*>(&x[j]) = *reinterpret_cast<const uint32_t*>(from);
        else x[j] = *reinterpret_cast<const Piece<D>*>(from);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (to[j] != nullptr) {
        if (weight) *reinterpret_cast<uint32_t*>(to[j]) = *reinterpret_cast<const uint32_t*>(&x[j]);
        else *reinterpret_cast<Piece<D>*>(to[j]) = x[j];
      }
  }
}

// The first blocks take the recent tokens of a (sequence, head) each, the others the fills that come from behind them, a
// warp a token: lanes 0 to 8 move pieces of K, 9 to 17 of V, lane 18 the weight, of kHeads heads at a time.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 4) kv4_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kHeads = 8;
  ptx::wait_dependencies();
  ptx::launch_dependents();
  const int block = static_cast<int>(blockIdx.x) - p.ordered, lane = threadIdx.x & 31;
  if (block < 0) {
    const int pair = blockIdx.x >> 1;
    move_in_order<D>(p, pair / p.c.hkv, pair % p.c.hkv, blockIdx.x & 1);
    return;
  }
  const int b = block / p.per_seq, first = (block % p.per_seq) * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const int fills = __ldg(&p.seqs[b].fills);
  const int32_t* const kept = p.kept + static_cast<int64_t>(b) * p.keep;
  const int32_t* const list = p.holes + static_cast<int64_t>(b) * p.keep;
  uint8_t* const base = lane < 18 ? static_cast<uint8_t*>(lane < 9 ? p.c.k : p.c.v) +
                                        (lane < 9 ? lane : lane - 9) * static_cast<int>(sizeof(Piece<D>))
                                  : reinterpret_cast<uint8_t*>(p.weight);
  const int64_t stride = lane < 18 ? kv4::kRow<D> : 4;
  for (int i = first; i < fills; i += p.per_seq * (kMoveThreads / 32)) {
    const int t = __ldg(list + i), source = __ldg(kept + t);
    if (source < p.keep) continue;
    const int to = row_of(p, b, t), from = row_of(p, b, source);
    if (lane > 18) continue;
    for (int h = 0; h < p.c.hkv; h += kHeads) {
      Piece<D> x[kHeads];
#pragma unroll
      for (int j = 0; j < kHeads; ++j)
        if (h + j < p.c.hkv) {
          const uint8_t* const at = base + (from + ((h + j) << p.page_log2)) * stride;
          if (lane < 18) x[j] = *reinterpret_cast<const Piece<D>*>(at);
          else *reinterpret_cast<uint32_t*>(&x[j]) = *reinterpret_cast<const uint32_t*>(at);
        }
#pragma unroll
      for (int j = 0; j < kHeads; ++j)
        if (h + j < p.c.hkv) {
          uint8_t* const at = base + (to + ((h + j) << p.page_log2)) * stride;
          if (lane < 18) *reinterpret_cast<Piece<D>*>(at) = x[j];
          else *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(&x[j]);
        }
    }
  }
}

struct Layout {
  int cluster, room, per_seq;
  int64_t holes_off, store_off, bytes;
  int smem;
};
// Blocks of a sequence: enough that one has two rounds of weights to read, as the page table's width tells, while the SMs
// hold them all: a cluster's barriers cost as much as a round.
Layout layout_of(const cp_kv4_evict_desc& d, int sms) {
  Layout r;
  const int64_t most = static_cast<int64_t>(d.max_pages) * d.cache.page_size, seqs = d.n_seqs > 0 ? d.n_seqs : 1;
  r.cluster = 1;
  while (r.cluster < kMostCluster && most > 8192 * static_cast<int64_t>(r.cluster) &&
         (seqs * r.cluster * 2 <= sms || most > kMostInSmem * static_cast<int64_t>(r.cluster)))
    r.cluster *= 2;
  r.room = static_cast<int>(((most + r.cluster - 1) / r.cluster + 31) / 32 * 32);
  const bool fits = r.room <= kMostInSmem;
  const int64_t words = r.room + static_cast<int64_t>(r.room) / 32 * 3;
  r.smem = fits ? static_cast<int>(words * 4) : 0;
  // a warp for each fill, of which there are as many as tokens that stay from slot z on, up to 8 blocks an SM
  int64_t fills = most - d.keep < d.keep - d.recent ? most - d.keep : d.keep - d.recent;
  if (fills < 1) fills = 1;
  const int64_t per = kMoveThreads / 32, share = (8 * static_cast<int64_t>(sms) + seqs - 1) / seqs;
  r.per_seq = static_cast<int>((fills + per - 1) / per < share ? (fills + per - 1) / per : share);
  r.holes_off = (seqs * static_cast<int64_t>(sizeof(Sequence)) + 255) / 256 * 256;
  const int64_t holes = most > d.keep ? d.keep : 0;
  r.store_off = r.holes_off + (seqs * holes * 4 + 255) / 256 * 256;
  r.bytes = r.store_off + (fits ? 0 : seqs * r.cluster * words * 4);
  return r;
}

}  // namespace

int64_t kv4_evict_workspace(const cp_kv4_evict_desc& d, int num_sms) { return layout_of(d, num_sms).bytes; }

cp_status launch_kv4_evict(const cp_kv4_evict_desc& d, int num_sms, cudaStream_t s) {
  const Layout l = layout_of(d, num_sms);
  uint8_t* const ws = static_cast<uint8_t*>(d.workspace);
  EvictParams p{};
  p.c = d.cache;
  p.weight = d.weight;
  p.tokens = d.tokens;
  p.table = d.page_table;
  p.n_seqs = d.n_seqs;
  p.max_pages = d.max_pages;
  p.keep = d.keep;
  p.recent = d.recent;
  p.page_log2 = d.cache.page_size == 16 ? 4 : d.cache.page_size == 32 ? 5 : d.cache.page_size == 64 ? 6 : 7;
  p.kept = d.kept;
  p.new_tokens = d.new_tokens;
  p.status = d.status;
  p.seqs = reinterpret_cast<Sequence*>(ws);
  p.holes = reinterpret_cast<int32_t*>(ws + l.holes_off);
  p.store = l.smem == 0 ? reinterpret_cast<uint32_t*>(ws + l.store_off) : nullptr;
  p.cluster = l.cluster;
  p.room = l.room;
  p.ordered = d.recent > 0 ? d.n_seqs * d.cache.hkv * 2 : 0;
  p.per_seq = l.per_seq;
  constexpr int most_smem = (kMostInSmem + kMostInSmem / 32 * 3) * 4;
  // The limit is the function's, not the call's: always the same, for other host threads launch the kernel too.
  cudaError_t e = cudaFuncSetAttribute(kv4_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
  if (e != cudaSuccess) return cuda_fail(e, "kv4_select_kernel attribute");
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(l.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = l.cluster > 1 ? 2 : 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(d.n_seqs * l.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(l.smem);
  if ((e = cudaLaunchKernelEx(&cfg, kv4_select_kernel, p)) != cudaSuccess) return cuda_fail(e, "kv4_select_kernel launch");
  if (static_cast<int64_t>(d.max_pages) * d.cache.page_size <= d.keep) return CP_OK;  // nothing can be too long
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(static_cast<unsigned>(p.ordered + (d.keep > d.recent ? d.n_seqs * l.per_seq : 0)));
  cfg.blockDim = dim3(kMoveThreads);
  e = cudaLaunchKernelEx(&cfg, d.cache.d == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, p);
  if (e != cudaSuccess) return cuda_fail(e, "kv4_move_kernel launch");
  return CP_OK;
}

}  // namespace cpattn

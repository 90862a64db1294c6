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
// The weights are read once; the rest is latency, of some ten barriers of a cluster.
// Second kernel, blocks for each (sequence, head): the fills, whose sources and holes do not overlap, then the recent rows,
// which move towards the front by n - keep: a batch is read before it is written, and the batches in order.  They may
// overwrite slots that fills come from, so they are the task of the block of a (sequence, head) that ends last.
#include <type_traits>

#include "internal.h"
#include "kv4_common.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostInSmem = 40960;  // tokens of a block
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
  int32_t* done;       // [n_seqs, hkv]: blocks of the second kernel that have made their fills
  int32_t* holes;      // [n_seqs, keep]
  uint32_t* store;     // [n_seqs, cluster] of room + 3 room / 32 words, where shared memory is too small; else null
  int32_t cluster, room;  // room: tokens of a block, a multiple of 32
  int32_t splits;      // blocks of a (sequence, head) in the second kernel
};

__device__ __forceinline__ int page_of(const EvictParams& p, int b, int token) {
  return __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + (token >> p.page_log2));
}
// Row of a token among the cache's rows for head 0.
__device__ __forceinline__ int64_t row_of(const EvictParams& p, int b, int token) {
  return (static_cast<int64_t>(page_of(p, b, token)) * p.c.hkv << p.page_log2) + (token & ((1 << p.page_log2) - 1));
}

// The sum of a token's weights over the heads, rounded once: the rounding errors of the additions are summed apart
// (Knuth's two-sum), so that the order of the heads does not decide between tokens.
__device__ __forceinline__ float weight_of(const EvictParams& p, int64_t row) {
  const float* w = p.weight + row;
  float s = 0.0f, err = 0.0f;
#pragma unroll 8
  for (int h = 0; h < p.c.hkv; ++h) {
    const float x = w[static_cast<int64_t>(h) << p.page_log2];
    const float t = __fadd_rn(s, x), y = __fsub_rn(t, s);
    err = __fadd_rn(err, __fadd_rn(__fsub_rn(s, __fsub_rn(t, y)), __fsub_rn(x, y)));
    s = t;
  }
  return fabsf(s) < INFINITY && fabsf(err) < INFINITY ? __fadd_rn(s, err) : s;
}
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
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scratch[w];
    all += scratch[w];
  }
  return before + in - x;
}

__device__ __forceinline__ int ld_cluster_int(uint32_t addr) { return __float_as_int(ptx::ld_cluster(addr)); }

// Bit k of a word of tokens: the first `count` of them.
__device__ __forceinline__ uint32_t first_bits(int count) {
  return count <= 0 ? 0u : count >= 32 ? kFull : (1u << count) - 1u;
}

__global__ void __launch_bounds__(kThreads) kv4_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ int hist[3][kBins];
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
  const int held = __ldg(p.tokens + b);
  const int n = held < 0 ? 0 : held;
  const bool over = n > static_cast<int64_t>(p.max_pages) << p.page_log2;
  int32_t* const kept = p.kept + static_cast<int64_t>(b) * p.keep;
  // A sequence that stays as it is.
  const auto leave = [&]() {
    for (int i = rank * kThreads + tid; i < p.keep; i += cluster * kThreads) kept[i] = i < n ? i : -1;
    if (rank == 0 && tid == 0) {
      p.new_tokens[b] = n;
      p.seqs[b] = Sequence{n, 0, 0, 0};
    }
  };
  for (int i = rank * kThreads + tid; i < p.c.hkv; i += cluster * kThreads)
    p.done[static_cast<int64_t>(b) * p.c.hkv + i] = 0;
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

  // Pages of all tokens, the recent ones too, have to be there before anything is read or changed.
  for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  int bad = 0;
  const int pages = (n + (1 << p.page_log2) - 1) >> p.page_log2;
  for (int i = rank * kThreads + tid; i < pages; i += cluster * kThreads) {
    const int page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + i);
    bad |= page < 0 || page >= p.c.n_pages;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) counts[0] = bad;
  meet();
  if (cluster > 1) {
    bad = 0;
    for (int r = 0; r < cluster; ++r) bad |= ld_cluster_int(ptx::cluster_addr(ptx::smem_u32(&counts[0]), r));
    ptx::cluster_sync();  // a block that ends now may be asked no more
  }
  if (bad) {
    if (rank == 0 && tid == 0) kv::report(p.status, kv::kSitePage);
    leave();
    return;
  }

  for (int i = tid; i < mine; i += kThreads) {
    const uint32_t k = order_of(weight_of(p, row_of(p, b, from + i)));
    key[i] = k;
    atomicAdd(&hist[0][k >> 21], 1);
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
      meet();
      constexpr int kPer = kBins / kThreads;
      int count[kPer], sum = 0;
      const int per = bins / kThreads;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {  // from the last bin on
        count[j] = 0;
        if (j < per) {
          int* const at = &hist[pass][bins - 1 - (tid * per + j)];
          if (cluster > 1) {
            for (int r = 0; r < cluster; ++r) count[j] += ld_cluster_int(ptx::cluster_addr(ptx::smem_u32(at), r));
          } else {
            count[j] = *at;
          }
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
    for (int r = 0; r < rank; ++r)
      ties_before += ld_cluster_int(ptx::cluster_addr(ptx::smem_u32(&hist[2][bits & 1023u]), r));
  }

  // What stays, 32 tokens a word; the first `want` of the tokens that equal the z-th largest.
  int holes = 0, movers = 0, ties = ties_before;
  for (int base = 0; base < words; base += kThreads) {
    const int w = base + tid;
    uint32_t more = 0, same = 0;
    if (w < words && z > 0)
      for (int j = 0; j < 32; ++j) {
        const int k = (j + lane) & 31;  // another bank for each lane
        if (32 * w + k >= mine) continue;
        const uint32_t x = key[32 * w + k];
        more |= (x > bits ? 1u : 0u) << k;
        same |= (x == bits ? 1u : 0u) << k;
      }
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
    for (int r = 0; r < cluster; ++r) {
      const int h = ld_cluster_int(ptx::cluster_addr(ptx::smem_u32(&counts[1]), r));
      if (r < rank) {
        holes_before += h;
        movers_before += ld_cluster_int(ptx::cluster_addr(ptx::smem_u32(&counts[2]), r));
      }
      fills += h;
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
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(const __grid_constant__ EvictParams p) {
  using Piece = typename std::conditional<D == 128, uint2, uint32_t>::type;
  constexpr int kUnits = 19;   // of a token: K, V, weight
  constexpr int kAhead = 8;    // of a thread
  __shared__ int last;
  ptx::wait_dependencies();
  const int split = blockIdx.x % p.splits;
  const int64_t item = blockIdx.x / p.splits;
  const int b = static_cast<int>(item / p.c.hkv), head = static_cast<int>(item - static_cast<int64_t>(b) * p.c.hkv);
  const Sequence s = p.seqs[b];
  const int tid = threadIdx.x;
  if (s.recent == 0 && s.fills == 0) return;
  const int64_t head_rows = static_cast<int64_t>(head) << p.page_log2;
  const int32_t* const kept = p.kept + static_cast<int64_t>(b) * p.keep;
  const int32_t* const list = p.holes + static_cast<int64_t>(b) * p.keep;
  // Moves `rows` tokens, the i-th from source(i) to target(i), in batches; `ordered`: a batch is read before it is written.
  const auto move = [&](int first, int step, int rows, bool ordered, auto target, auto source) {
    const int64_t units = static_cast<int64_t>(rows) * kUnits;
    for (int64_t base = static_cast<int64_t>(first) * kMoveThreads * kAhead; base < units;
         base += static_cast<int64_t>(step) * kMoveThreads * kAhead) {
      Piece x[kAhead];
      void* to[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t unit = base + j * kMoveThreads + tid;
        to[j] = nullptr;
        if (unit < units) {
          const int i = static_cast<int>(unit / kUnits), e = static_cast<int>(unit - static_cast<int64_t>(i) * kUnits);
          const int t = target(i);
          const int64_t at = row_of(p, b, t) + head_rows, src = row_of(p, b, source(i, t)) + head_rows;
          if (e < 18) {
            uint8_t* const rows8 = static_cast<uint8_t*>(e < 9 ? p.c.k : p.c.v);
            const int piece = (e < 9 ? e : e - 9) * static_cast<int>(sizeof(Piece));
            x[j] = *reinterpret_cast<const Piece*>(rows8 + src * kv4::kRow<D> + piece);
            to[j] = rows8 + at * kv4::kRow<D> + piece;
          } else {
            *reinterpret_cast<float*>(&x[j]) = p.weight[src];
            to[j] = p.weight + at;
          }
        }
      }
      if (ordered) __syncthreads();
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t unit = base + j * kMoveThreads + tid;
        if (to[j] != nullptr) {
          if (unit % kUnits < 18) *static_cast<Piece*>(to[j]) = x[j];
          else *static_cast<float*>(to[j]) = *reinterpret_cast<const float*>(&x[j]);
        }
      }
    }
  };
  move(split, p.splits, s.fills, false, [&](int i) { return __ldg(list + i); },
       [&](int, int t) { return __ldg(kept + t); });
  if (s.recent == 0) return;
  if (p.splits > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(p.done + item, 1) == p.splits - 1 ? 1 : 0;
    __syncthreads();
    if (!last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  const int by = s.n - p.keep;
  move(0, 1, s.recent, true, [&](int i) { return s.z + i; }, [&](int, int t) { return t + by; });
}

struct Layout {
  int cluster, room, splits;
  int64_t done_off, holes_off, store_off, bytes;
  int smem;
};
// Blocks of a sequence: enough that one has 4096 tokens or fewer, as the page table's width tells, while the SMs hold
// them all.
Layout layout_of(const cp_kv4_evict_desc& d, int sms) {
  Layout r;
  const int64_t most = static_cast<int64_t>(d.max_pages) * d.cache.page_size, seqs = d.n_seqs > 0 ? d.n_seqs : 1;
  r.cluster = 1;
  while (r.cluster < 8 && most > 4096 * static_cast<int64_t>(r.cluster) &&
         (seqs * r.cluster * 2 <= sms || most > kMostInSmem * static_cast<int64_t>(r.cluster)))
    r.cluster *= 2;
  r.room = static_cast<int>(((most + r.cluster - 1) / r.cluster + 31) / 32 * 32);
  const bool fits = r.room <= kMostInSmem;
  const int64_t words = r.room + static_cast<int64_t>(r.room) / 32 * 3;
  r.smem = fits ? static_cast<int>(words * 4) : 0;
  const int64_t items = seqs * d.cache.hkv;
  r.splits = static_cast<int>(items >= 4 * sms ? 1 : (4 * sms + items - 1) / items);
  const int64_t turns = (static_cast<int64_t>(d.keep) * 19 + kMoveThreads * 8 - 1) / (kMoveThreads * 8);
  if (r.splits > turns) r.splits = turns > 0 ? static_cast<int>(turns) : 1;
  r.done_off = (seqs * static_cast<int64_t>(sizeof(Sequence)) + 255) / 256 * 256;
  r.holes_off = r.done_off + (items * 4 + 255) / 256 * 256;
  r.store_off = r.holes_off + (seqs * d.keep * 4 + 255) / 256 * 256;
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
  p.done = reinterpret_cast<int32_t*>(ws + l.done_off);
  p.holes = reinterpret_cast<int32_t*>(ws + l.holes_off);
  p.store = l.smem == 0 ? reinterpret_cast<uint32_t*>(ws + l.store_off) : nullptr;
  p.cluster = l.cluster;
  p.room = l.room;
  p.splits = l.splits;
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
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(d.n_seqs) * d.cache.hkv * l.splits));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, d.cache.d == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>, p);
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "kv4_move_kernel launch");
}

}  // namespace cpattn

// The attention weight that the tokens of the paged 4-bit cache gather (cp_kv4_cache_weigh).
//
//   weight_j := decay weight_j + sum over the rows i that see j and the query heads of the KV head of
//               2^(log2 e (scale (q_i . k_j) - LSE_i)),
// with the rows' final LSE, so that the weights of all ranks' tokens are parts of one softmax.  Given the LSE there is
// no running maximum and nothing to join: every key is on its own.  Bound: keys and weights are read once and weights
// written once; values are not touched.
//
// The unit of work is a granule (4096 / D tokens of one sequence and head) with all of the sequence's rows, so each
// weight has one writer and its sum one order; two share a stage of the ring, its wait and its copies.  Granules are
// numbered sequence after sequence, each head beginning with kSetup numbers more, and every warp has an equal share of
// consecutive ones.  A share's part of a head is gone over once for each block of RT query rows; the keys come by a ring
// of copies as for attention, the old weights with them.
//
// Bound by instructions: the conversions, products and exponentials of two granules are some 370 instructions for 64 keys
// at D = 128, issued at 60 % of the SMs' rate.  Measured (GB300, in a graph): 64 x 256-8192 tokens, 32/8 heads, D = 128,
// bf16: 41.5 us for 173 MB, 4.2 TB/s (12 warps 49); 4 x 1-4 rows over 30000-65536, 64/8, D = 64, fp32: 49.5 us, of which the
// tensor cores are busy for 42 % (32 query rows of two f16 parts).  With shares of whole stages it took 54, some warps
// having 9 and some 10 of them (14 calls of many kinds 9 % more in the mean; 16 rows of 4 at D = 128, bf16, 59 against
// 62).  Shares by the cost of a sequence's rows were slower (84: a granule's time depends little on its tiles), as were
// predicates around tiles without rows (60); queries in shared memory and 12 warps gained 3 to 8 % for fp32 and lost 25 %
// for bf16 at D = 128.
#include "kv4_tile.cuh"

namespace cpattn {
namespace kvattn {

namespace {

// What a head costs besides its granules, in granules (1 / 2 / 4: the batch above 41.9 / 41.5 / 41.4 us).
constexpr int kSetup = 2;

struct WeighParams {
  Params p;  // q, lse (read), rows, tile[0], ...
  float* weight;
  const int32_t* known;
  float decay;
};

template <int D, int NT, int QP>
struct WeighShape {
  static constexpr int kKeys = Granule<D>::kKeys;
  static constexpr int kQ = NT * QP * D / 8;  // registers of query operands
  static constexpr int kWarps = kQ <= 16 ? 16 : kQ <= 32 ? 12 : 8;
  static constexpr int kRows = NT * 8;  // RT
  static constexpr int kStages = kWarps == 16 ? 2 : kWarps == 12 ? 3 : 4;
  static constexpr int kOldOff = Granule<D>::kPair;         // old weights of the stage's keys
  static constexpr int kPageOff = kOldOff + 2 * kKeys * 4;  // pages of their parts, 8 at most
  static constexpr int kStage = kPageOff + 32;
  // The plan is looked at before the first copies and lies where they go.
  static constexpr int kBarOff = kWarps * kStages * kStage;
  static constexpr int kCtlOff = kBarOff + (kWarps * kStages + 1) * 8;
  static constexpr int kScanOff = (kCtlOff + 8 + 15) / 16 * 16;
  static constexpr int kBytes = kScanOff + 16 * 8;
  static_assert(kBarOff >= (CP_KV_MAX_SEQS + 1) * 8, "the plan fits the rings");
};

struct WeighSeq {
  int64_t r0, pos0;
  int32_t rows, tokens, known, gpi, blocks;
  bool over;
};
template <int KEYS, int RT>
__device__ __forceinline__ WeighSeq weigh_seq(const WeighParams& w, int b) {
  const Params& p = w.p;
  WeighSeq s;
  s.r0 = kv::row_at(p.rows, b);
  const int64_t r1 = kv::row_at(p.rows, b + 1);
  s.rows = r1 > s.r0 ? static_cast<int32_t>(r1 - s.r0) : 0;
  const int64_t t = __ldg(p.rows.tokens + b), room = static_cast<int64_t>(p.rows.max_pages) << p.page_log2;
  s.over = t > room;
  s.tokens = t < 0 ? 0 : static_cast<int32_t>(t < room ? t : room);
  s.known = w.known != nullptr ? __ldg(w.known + b) : s.tokens;
  s.pos0 = p.q_first != nullptr ? __ldg(p.q_first + b) : 0;
  s.gpi = s.rows > 0 ? (s.tokens + KEYS - 1) / KEYS : 0;
  s.blocks = s.rows > 0 ? (s.rows * p.group + RT - 1) / RT : 0;
  return s;
}

// A walk over a share: for each sequence and head the granules g0 .. g1 - 1, once for each block of rows.
template <int KEYS, int RT>
struct Walk {
  int b, head, block, g, g0, g1;
  int left;  // numbers of the share behind this part
  WeighSeq s;

  // Takes the part that begins with granule g0 out of `left` numbers that begin there.
  __device__ __forceinline__ void enter(int from) {
    block = 0;
    g = g0 = from;
    g1 = s.gpi - from < left ? s.gpi : from + left;
    left -= g1 - g0;
  }
  // How many granules go through the ring together.
  __device__ __forceinline__ int step() const { return together(g, g1); }
  // To the granules behind these; false at the end of the share.
  __device__ __forceinline__ bool next(const WeighParams& w) {
    g += step();
    if (g < g1) return true;
    if (++block < s.blocks) {
      g = g0;
      return true;
    }
    left -= kSetup;
    if (left <= 0) return false;
    if (++head == w.p.hkv) {
      head = 0;
      do {
        if (++b >= w.p.rows.n_seqs) return false;
        s = weigh_seq<KEYS, RT>(w, b);
      } while (s.gpi == 0);
    }
    enter(0);
    return true;
  }
};

template <int D, int NT, int QP>
__global__ void __launch_bounds__(WeighShape<D, NT, QP>::kWarps * 32, 1)
    kv4_weigh_kernel(const __grid_constant__ WeighParams w) {
  using S = WeighShape<D, NT, QP>;
  constexpr int RT = S::kRows, kMt = D / 16, kSt = S::kStages, kKeys = S::kKeys, kSteps = kKeys / 16;
  const Params& p = w.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((128u - (ptx::smem_u32(smem_raw) & 127u)) & 127u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  int64_t* const plan = reinterpret_cast<int64_t*>(smem);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + S::kCtlOff);
  const uint32_t base = ptx::smem_u32(smem);
  const uint32_t ring = base + warp * kSt * S::kStage;
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
  ptx::wait_dependencies();
  const int n_seqs = p.rows.n_seqs;
  const sync::Ctl ctl{abort_flag, p.status, p.timeout_ns};
  make_plan_of<S::kWarps * 32>(n_seqs, plan, reinterpret_cast<int64_t*>(smem + S::kScanOff), [&](int b) {
    const WeighSeq s = weigh_seq<S::kKeys, RT>(w, b);
    if (s.over && s.rows > 0 && blockIdx.x == 0) kv::report(p.status, kv::kSiteTokens);
    return s.gpi > 0 ? static_cast<int64_t>(p.hkv) * (s.gpi + kSetup) : 0;
  });
  const bool stalled = p.stall && blockIdx.x == 0 && warp == 0;  // test only
  const int64_t W = plan[n_seqs];
  const int64_t most = static_cast<int64_t>(gridDim.x) * S::kWarps, n_workers = W < most ? W : most;
  const int64_t worker = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;  // neighbours on different SMs
  Walk<S::kKeys, RT> c;
  c.left = 0;
  bool idle = worker >= n_workers || stalled;
  if (!idle) {
    const int64_t lo = share(W, n_workers, worker);
    int a = 0, z = n_seqs - 1;  // the last sequence whose numbers begin at or before lo
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (plan[mid] <= lo) a = mid;
      else z = mid - 1;
    }
    c.b = a;
    c.s = weigh_seq<S::kKeys, RT>(w, a);
    const int64_t off = lo - plan[a];
    c.head = static_cast<int>(off / (c.s.gpi + kSetup));
    const int at = static_cast<int>(off - static_cast<int64_t>(c.head) * (c.s.gpi + kSetup));
    c.left = static_cast<int>(share(W, n_workers, worker + 1) - lo);
    if (at < kSetup) c.left -= kSetup - at;
    idle = c.left <= 0;
    if (!idle) c.enter(at < kSetup ? 0 : at - kSetup);
  }
  ptx::fence_proxy_async_smem();
  __syncthreads();  // the plan has been read: the copies may begin
  if (stalled) sync::wait_warp(stall_bar, 0, ctl, kv::kSiteWait);
  if (idle) return;
  Walk<S::kKeys, RT> f = c;  // where the copies are
  bool more = true;   // to copy
  Feed<D, 1> feed{f.b, f.head, f.s.tokens, -32, -1};

  auto issue = [&](int st) {
    const uint32_t dst = ring + st * S::kStage, bar = bars + st * 8;
    if (feed.b != f.b) {
      feed.b = f.b;
      feed.keys = f.s.tokens;
      feed.window = -32;
    }
    feed.head = f.head;
    // Pages too, for the way back, and old weights for the first block of rows.
    feed.stage(p, lane, f.g, f.step(), dst, bar, [&](int i, int page, int slot, int rows) {
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + S::kPageOff + 4 * i), "r"(page) : "memory");
      if (page < 0 || f.block > 0) return 0u;
      const uint32_t bytes = ((rows + 3) & ~3) * 4;
      const int64_t at = (page * p.hkv + f.head) * p.page + slot;
      ptx::bulk_load(dst + S::kOldOff + 4 * (i << p.page_log2), w.weight + at, bytes, bar);
      return bytes;
    });
    more = f.next(w);
  };

  uint32_t qf[NT * QP][kMt][2];
  float fac[NT][2], lse2[NT][2];  // of the lane's two query rows 2 tig, 2 tig + 1 in each tile
  int lim[NT][2];
  int lim_min = 0;
  auto begin_block = [&]() {
    const int row_q = c.block * RT, n_rows = c.s.rows * p.group;
    int lmin = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int rho = row_q + n * 8 + gid;  // the lane's part of query row gid of the tile
      const bool live = rho < n_rows;
      const int t = live ? rho / p.group : 0;
      const int64_t out = (c.s.r0 + t) * p.hq + c.head * p.group + (rho - t * p.group);
      const int lm = live ? visible(p, c.s.tokens, c.s.pos0 + t) : 0;
      // A row whose LSE is not finite has no weights to give: 2^(0 - inf) with zeros for its operands, since its query, which
      // the LSE mostly comes from, need not be finite.
      const float lse = live ? __ldg(p.lse + out) : INFINITY;
      const bool gives = fabsf(lse) < INFINITY;
      const float l2 = gives ? lse * kLog2e : INFINITY;
      if (live) lmin = min(lmin, lm);
      const float f = query_operands<D, QP>(p, out * D, live, tig, &qf[n * QP]);  // loads that do not wait for the LSE
      if (!gives) {
#pragma unroll
        for (int part = 0; part < QP; ++part)
#pragma unroll
          for (int j = 0; j < kMt; ++j) qf[n * QP + part][j][0] = qf[n * QP + part][j][1] = 0u;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        fac[n][r] = __shfl_sync(kFull, f, (2 * tig + r) * 4);
        lim[n][r] = __shfl_sync(kFull, lm, (2 * tig + r) * 4);
        lse2[n][r] = __shfl_sync(kFull, l2, (2 * tig + r) * 4);
      }
    }
    lim_min = __reduce_min_sync(kFull, lmin);
  };

  auto granule = [&](uint32_t stage, int i, int part_log2) {
    const uint32_t tile = stage + i * Granule<D>::kHalf;
    const int key0 = (c.g + i) * kKeys;
    const bool masked = key0 + kKeys > lim_min;
    float sum[2 * kSteps];  // key key_at(i, u, gid)
#pragma unroll
    for (int step0 = 0; step0 < kSteps; step0 += 2) {
      float s[NT][2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.0f;
      key_operands<D>(tile, step0, gid, tig, [&](int j, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
#pragma unroll
        for (int part = 0; part < QP; ++part)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            ptx::mma_f16(s[n][0], a, qf[n * QP + part][j][0], qf[n * QP + part][j][1]);
            ptx::mma_f16(s[n][1], b, qf[n * QP + part][j][0], qf[n * QP + part][j][1]);
          }
      });
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = 0.0f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float e = ex2(fmaf(s[n][half][2 * u + r], fac[n][r], -lse2[n][r]));
              x += masked && key0 + key_at<D>(step0 + half, u, gid) >= lim[n][r] ? 0.0f : e;
            }
          x += __shfl_xor_sync(kFull, x, 1);
          x += __shfl_xor_sync(kFull, x, 2);
          sum[2 * (step0 + half) + u] = x;
        }
    }
    // lane (gid, tig) writes the keys of sums tig, tig + 4, ...
#pragma unroll
    for (int q = 0; q < kSteps / 2; ++q) {
      const float x = tig == 0 ? sum[4 * q] : tig == 1 ? sum[4 * q + 1] : tig == 2 ? sum[4 * q + 2] : sum[4 * q + 3];
      const int k = key_at<D>(2 * q + (tig >> 1), tig & 1, gid), key = key0 + k;
      if (key >= c.s.tokens) continue;
      const int page = static_cast<int>(lds32(stage + S::kPageOff + 4 * (i * kKeys + k >> part_log2)));
      if (page < 0) continue;
      float* const at = w.weight + ((page * p.hkv + c.head) * p.page + (key & (p.page - 1)));
      float old = 0.0f;
      if (c.block > 0) old = *at;  // what this lane wrote
      else if (key < c.s.known && w.decay != 0.0f)
        old = w.decay * __uint_as_float(lds32(stage + S::kOldOff + 4 * (i * kKeys + k)));
      *at = old + x;
    }
  };

  auto wait = [&](uint32_t bar, uint32_t par) {
    const bool ok = __all_sync(kFull, ptx::mbar_try_wait(bar, par)) || sync::wait_warp(bar, par, ctl, kv::kSiteWait);
    __syncwarp();  // the stage's pages, which a lane wrote
    return ok;
  };
  int st = 0, in_flight = 0;
  uint32_t parity = 0;
  for (int i = 0; i < kSt; ++i)
    if (more) {
      issue(i);
      ++in_flight;
    }
  begin_block();
  while (in_flight > 0) {
    if (!wait(bars + st * 8, parity)) break;
    const int n = c.step(), part_log2 = p.page >= n * kKeys ? 31 : p.page_log2;  // the stage's tokens of one page
#pragma unroll 1
    for (int i = 0; i < n; ++i) granule(ring + st * S::kStage, i, part_log2);
    __syncwarp();
    if (more) issue(st);
    else --in_flight;
    if (++st == kSt) {
      st = 0;
      parity ^= 1u;
    }
    const int block = c.block, head = c.head, b = c.b;
    if (c.next(w) && (c.block != block || c.head != head || c.b != b)) begin_block();
  }
  for (int i = 0; i < in_flight; ++i) {  // after a wait that ran out: copies in flight must not outlive the block
    sync::wait_drain(bars + st * 8, parity, p.timeout_ns);
    if (++st == kSt) {
      st = 0;
      parity ^= 1u;
    }
  }
}

template <int D, int NT, int QP>
cp_status run_weigh(const WeighParams& w, int num_sms, cudaStream_t s) {
  using S = WeighShape<D, NT, QP>;
  constexpr int smem = 128 + S::kBytes;
  static_assert(smem <= 232448, "shared memory of a block");
  const auto kernel = kv4_weigh_kernel<D, NT, QP>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "kv4_weigh_kernel attribute");
  const Params& p = w.p;
  const double most = (static_cast<double>(p.rows.max_pages) * p.page / S::kKeys + 1 + kSetup) * p.hkv * p.rows.n_seqs;
  if (most > 1e12) {
    set_error("cp_kv4_cache_weigh: max_pages * page_size * hkv * n_seqs is too large for one call");
    return CP_ERR_INVALID_ARG;
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(most < num_sms ? most : num_sms));
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, kernel, w);
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "kv4_weigh_kernel launch");
}

template <int D>
cp_status run_weigh_d(const WeighParams& w, int nt, int num_sms, cudaStream_t s) {
  if (w.p.q_bf16)
    return nt == 1   ? run_weigh<D, 1, 1>(w, num_sms, s)
           : nt == 2 ? run_weigh<D, 2, 1>(w, num_sms, s)
                     : run_weigh<D, 4, 1>(w, num_sms, s);
  if constexpr (D == 64)
    if (nt == 4) return run_weigh<D, 4, 2>(w, num_sms, s);
  return nt == 1 ? run_weigh<D, 1, 2>(w, num_sms, s) : run_weigh<D, 2, 2>(w, num_sms, s);
}

}  // namespace
}  // namespace kvattn

cp_status launch_kv4_weigh(const cp_kv4_weigh_desc& d, float scale, int64_t timeout_ns, int num_sms, cudaStream_t s) {
  using namespace kvattn;
  const cp_kv4_cache& c = d.cache;
  WeighParams w{};
  Params& p = w.p;
  p.tile[0] = static_cast<const uint8_t*>(c.k);
  p.rows = d.rows;
  p.n_pages = c.n_pages;
  p.q = d.q;
  p.lse = const_cast<float*>(d.lse);
  p.q_first = d.q_first;
  p.hq = d.hq;
  p.hkv = c.hkv;
  p.group = d.hq / c.hkv;
  p.page = c.page_size;
  p.page_log2 = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.q_bf16 = d.in_dtype == CP_BF16;
  p.stall = (d.flags & CP_FLAG_TEST_STALL) != 0;
  p.scale_log2 = scale * kLog2e;
  p.kv_pos = d.kv_pos;
  p.status = d.status;
  p.timeout_ns = timeout_ns;
  w.weight = d.weight;
  w.known = d.known;
  w.decay = d.decay;
  // The fewest tiles of 8 rows that hold a sequence's rows on average, 4 at most (2 of fp32 queries at D = 128), since every
  // pass converts the keys again.  4 x 30000-65536 tokens, 64/8 heads, one / two / four tiles, us: D = 64, fp32, 8 rows
  // 23 / 30 / 47, 16: 41 / 30 / 47, 24: 58 / 56 / 48, 32: 75 / 57 / 48; D = 128, bf16, 8: 30 / 39 / 58, 16: 56 / 40 / 59,
  // 24: 79 / 78 / 60, 32: 104 / 80 / 61.
  const int64_t per = (d.rows.n_rows + d.rows.n_seqs - 1) / d.rows.n_seqs * p.group;
  const int nt = per <= 8 ? 1 : per <= 16 || (!p.q_bf16 && c.d == 128) ? 2 : 4;
  return c.d == 128 ? run_weigh_d<128>(w, nt, num_sms, s) : run_weigh_d<64>(w, nt, num_sms, s);
}

}  // namespace cpattn

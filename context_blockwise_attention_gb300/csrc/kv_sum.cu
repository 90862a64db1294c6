// The second kernel of attention over a paged cache: the sum of the workers' partials.
#include "kv_split.cuh"

namespace cpattn {
namespace kvattn {

namespace {

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
  const int64_t from = plan[b] + (static_cast<int64_t>(head) * seq.blocks + block) * (seq.gpi + p.setup) + p.setup;
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

}  // namespace

template <int D, int RT>
cp_status launch_sum(const Params& p, int64_t workers, int64_t items, int num_sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  // Eight warps an output row while there are few rows (320 rows of 8 partials: 8 us against 14), or many
  // partials to a row; else one (2176 rows of 5 partials: 104 us the whole call, against 116 with eight; 45 x 0-103
  // tokens, 1-4 rows of 128/32 heads 22 and 75).
  const int64_t parts = workers / (items < 1 ? 1 : items), outs = p.rows.n_rows * p.hq;
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
  const auto sum = columns ? kv_attn_combine_columns_kernel<D, RT>
                   : wide  ? kv_attn_combine_kernel<D, RT, 8>
                           : kv_attn_combine_kernel<D, RT, 1>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sum, p, workers);
  return e == cudaSuccess ? CP_OK : cuda_fail(e, "kv_attn_combine_kernel launch");
}
#define CP_SUM(D, RT) template cp_status launch_sum<D, RT>(const Params&, int64_t, int64_t, int, cudaStream_t)
CP_SUM(64, 8);
CP_SUM(64, 16);
CP_SUM(128, 8);
CP_SUM(128, 16);
CP_SUM(128, 24);
#undef CP_SUM

}  // namespace kvattn
}  // namespace cpattn

// Writing tokens into the paged 4-bit cache and reading them back (cp_kv4_cache_write / _read).
//
// Every group of 16 numbers is on its own: its scale, its codes, 9 bytes.  So the unit of work is a group of a
// (row of the call, head), a thread's: 16 numbers in or out with 16-byte accesses, 8 bytes of codes and a scale byte.
// Memory bound: a number costs its own size and 9/16 of a byte.
// A block takes kRows rows of the call: it looks their pages up once, side by side, and goes over the rows of one
// head after the other, so that neighbouring lanes write (or read) consecutive rows of a page.
// Measured (GB300, 29 k tokens of 8 heads, D = 128, bf16, 152 MB each way): writing 31 us, reading 30 (floor 22.5 each).
// One group of a thread at a time is best: two took 33 and 33 us, four and eight 32 and 37, since more registers leave
// fewer warps; so were half a group a thread for reading (whole lines of stores, 34) and smaller or larger blocks (59 us for
// both kernels in turn, 60 to 63 with 16 or 64 rows or more blocks to an SM).
#include "internal.h"
#include "kv4_common.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;  // of a block

struct CopyParams {
  cp_kv4_cache c;
  cp_kv_rows rows;
  void* x[2];  // k, v
  int32_t* status;
  int32_t parts, per;  // blocks of a block of rows, and items of each
};

// Where the rows of a block of rows live: row (page * hkv * page_size + slot) of the cache's rows for head 0, or -1.
struct Places {
  int32_t start[CP_KV_MAX_SEQS + 1];
  int32_t at[kRows];
};
__device__ __forceinline__ void look_up(const CopyParams& p, int64_t row0, bool speaks, Places& s) {
  const cp_kv_rows& r = p.rows;
  for (int i = threadIdx.x; i <= r.n_seqs; i += kThreads) s.start[i] = static_cast<int32_t>(kv::row_at(r, i));
  __syncthreads();
  if (threadIdx.x < kRows) {
    const int64_t row = row0 + threadIdx.x;
    int32_t at = -1;
    if (row < r.n_rows) {
      int b = 0, z = r.n_seqs - 1;  // the last sequence that begins at or before the row
      while (b < z) {
        const int mid = (b + z + 1) >> 1;
        if (s.start[mid] <= row) b = mid;
        else z = mid - 1;
      }
      const int64_t first = __ldg(r.tokens + b);
      if (s.start[b] <= row && row < s.start[b + 1] && first >= 0) {
        const int shift = 31 - __clz(p.c.page_size);
        const int64_t token = first + (row - s.start[b]);
        const int64_t page = kv::page_at(r, p.c.n_pages, b, token >> shift);
        if (page >= 0) at = static_cast<int32_t>(page * p.c.hkv * p.c.page_size + (token & (p.c.page_size - 1)));
        else if (speaks) kv::report(p.status, kv::kSitePage);
      }
    }
    s.at[threadIdx.x] = at;
  }
  __syncthreads();
}

// Item i of a block of rows: group fastest, then row, then head, then K or V.
template <int D>
struct Item {
  int group, row, head, which;
  __device__ __forceinline__ Item(int i, int hkv) {
    constexpr int kGroups = D / 16;
    group = i % kGroups;
    row = i / kGroups % kRows;
    head = i / (kGroups * kRows);
    which = head >= hkv ? 1 : 0;
    head -= which ? hkv : 0;
  }
};

__device__ __forceinline__ void load16(const float* p, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + j);
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, uint32_t (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + j);
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
}

// Largest magnitude as the bits of an fp32 number; as whole numbers, so that NaN counts for the largest.
__device__ __forceinline__ uint32_t magnitude_bits(const uint32_t (&w)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = max(m, w[j] & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t magnitude_bits(const uint32_t (&w)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
  return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ float number(const uint32_t (&w)[16], int i) { return __uint_as_float(w[i]); }
__device__ __forceinline__ float number(const uint32_t (&w)[8], int i) {
  return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ CopyParams p) {
  constexpr int kGroups = D / 16, kWords = sizeof(T) == 4 ? 16 : 8;
  __shared__ Places s;
  ptx::wait_dependencies();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.parts) * kRows;
  const int part = static_cast<int>(blockIdx.x % p.parts);
  look_up(p, row0, part == 0, s);
  const int hkv = p.c.hkv;
  const int end = min(2 * hkv * kRows * kGroups, (part + 1) * p.per);
  for (int i = part * p.per + threadIdx.x; i < end; i += kThreads) {
    const Item<D> it(i, hkv);
    const int32_t at = s.at[it.row];
    if (at < 0) continue;
    uint32_t w[kWords];
    load16(static_cast<const T*>(p.x[it.which]) + ((row0 + it.row) * hkv + it.head) * D + it.group * 16, w);
    const uint32_t top = magnitude_bits(w);
    uint32_t code = kv4::kNaN;
    uint32_t packed[2] = {0u, 0u};
    if (top < 0x7f800000u) {
      code = kv4::scale_code(__uint_as_float(top));
      float hi, lo;
      kv4::reciprocal(kv4::scale_of(code), hi, lo);
      const uint64_t hi2 = ptx::f2_pack(hi, hi), lo2 = ptx::f2_pack(lo, lo);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t two = ptx::f2_pack(number(w, 8 * q + 2 * j), number(w, 8 * q + 2 * j + 1));
          ptx::f2_unpack(ptx::f2_fma(two, hi2, ptx::f2_mul(two, lo2)), x[2 * j], x[2 * j + 1]);  // as kv4::times
        }
        packed[q] = code != 0u ? kv4::to_e2m1x8(x) : 0u;
      }
    }
    uint8_t* const out = static_cast<uint8_t*>(it.which ? p.c.v : p.c.k) +
                         (at + static_cast<int64_t>(it.head) * p.c.page_size) * kv4::kRow<D>;
    if constexpr (D == 128) {  // rows begin at multiples of 8 bytes
      *reinterpret_cast<uint2*>(out + it.group * 8) = make_uint2(packed[0], packed[1]);
    } else {
      reinterpret_cast<uint32_t*>(out)[it.group * 2] = packed[0];
      reinterpret_cast<uint32_t*>(out)[it.group * 2 + 1] = packed[1];
    }
    out[D / 2 + it.group] = static_cast<uint8_t>(code);
  }
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ void store4(float* p, float2 a, float2 b) {
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}

template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ CopyParams p) {
  constexpr int kGroups = D / 16;
  __shared__ Places s;
  ptx::wait_dependencies();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.parts) * kRows;
  const int part = static_cast<int>(blockIdx.x % p.parts);
  look_up(p, row0, part == 0, s);
  const int hkv = p.c.hkv;
  const int end = min(2 * hkv * kRows * kGroups, (part + 1) * p.per);
  for (int i = part * p.per + threadIdx.x; i < end; i += kThreads) {
    const Item<D> it(i, hkv);
    const int32_t at = s.at[it.row];
    if (at < 0) continue;
    const uint8_t* const in = static_cast<const uint8_t*>(it.which ? p.c.v : p.c.k) +
                              (at + static_cast<int64_t>(it.head) * p.c.page_size) * kv4::kRow<D>;
    uint32_t word[2];
    if constexpr (D == 128) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(in + it.group * 8));
      word[0] = v.x, word[1] = v.y;
    } else {
      word[0] = __ldg(reinterpret_cast<const uint32_t*>(in) + it.group * 2);
      word[1] = __ldg(reinterpret_cast<const uint32_t*>(in) + it.group * 2 + 1);
    }
    const uint32_t scale = kv4::scale_twice(__ldg(in + D / 2 + it.group), 0);
    T* const out = static_cast<T*>(p.x[it.which]) + ((row0 + it.row) * hkv + it.head) * D + it.group * 16;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t h[4];
      kv4::to_f16x2(word[q], h);
      float2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = f16x2_to_float2(kv4::mul_f16x2(h[j], scale));
      if constexpr (sizeof(T) == 4) {
        store4(out + 8 * q, f[0], f[1]);
        store4(out + 8 * q + 4, f[2], f[3]);
      } else {
        *reinterpret_cast<uint4*>(out + 8 * q) =
            make_uint4(ptx::pack_bf16x2(f[0].x, f[0].y), ptx::pack_bf16x2(f[1].x, f[1].y),
                       ptx::pack_bf16x2(f[2].x, f[2].y), ptx::pack_bf16x2(f[3].x, f[3].y));
      }
    }
  }
}

// Blocks of rows are cut by heads until the SMs have some four blocks each.
void cut(CopyParams& p, int num_sms, int64_t& blocks) {
  const int64_t groups = (p.rows.n_rows + kRows - 1) / kRows;
  const int all = 2 * p.c.hkv * kRows * (p.c.d / 16);  // at most 2^25
  const int most = (all + kThreads - 1) / kThreads;
  int64_t parts = (4 * static_cast<int64_t>(num_sms) + groups - 1) / groups;
  if (parts > most) parts = most;
  const int turns = static_cast<int>((most + parts - 1) / parts);
  p.per = turns * kThreads;
  p.parts = (all + p.per - 1) / p.per;
  blocks = groups * p.parts;
}

template <class K>
cp_status launch(K kernel, const CopyParams& p, int64_t blocks, cudaStream_t s, const char* what) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? CP_OK : cuda_fail(e, what);
}

}  // namespace

cp_status launch_kv4_write(const cp_kv4_cache& c, const cp_kv_rows& rows, const void* k, const void* v, bool bf16,
                           int32_t* status, int num_sms, cudaStream_t s) {
  CopyParams p{c, rows, {const_cast<void*>(k), const_cast<void*>(v)}, status, 0, 0};
  int64_t blocks;
  cut(p, num_sms, blocks);
  const auto kernel = c.d == 128 ? (bf16 ? kv4_write_kernel<128, __nv_bfloat16> : kv4_write_kernel<128, float>)
                                 : (bf16 ? kv4_write_kernel<64, __nv_bfloat16> : kv4_write_kernel<64, float>);
  return launch(kernel, p, blocks, s, "kv4_write_kernel launch");
}

cp_status launch_kv4_read(const cp_kv4_cache& c, const cp_kv_rows& rows, void* k, void* v, bool bf16, int32_t* status,
                          int num_sms, cudaStream_t s) {
  CopyParams p{c, rows, {k, v}, status, 0, 0};
  int64_t blocks;
  cut(p, num_sms, blocks);
  const auto kernel = c.d == 128 ? (bf16 ? kv4_read_kernel<128, __nv_bfloat16> : kv4_read_kernel<128, float>)
                                 : (bf16 ? kv4_read_kernel<64, __nv_bfloat16> : kv4_read_kernel<64, float>);
  return launch(kernel, p, blocks, s, "kv4_read_kernel launch");
}

}  // namespace cpattn

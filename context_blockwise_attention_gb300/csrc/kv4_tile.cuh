// What the kernels over the 4-bit cache share: a warp's ring of granules (4096 / D consecutive tokens of one
// sequence and head), the copies that fill it, and the operands of mma.sync made of its rows.
//
// A granule's rows lie in shared memory as in the cache, 72 or 36 bytes apart.  The operands' rows are free to be any
// of its keys as long as both products agree; key_at is chosen so that the lanes of a load meet no bank twice:
//   D = 128: a row is 18 banks.  A lane reads 16 bytes of key c = gid (two 8-byte loads; half a warp holds c = 0..3 or
//            4..7, keys x, x + 1, x + 8, x + 9, which begin at banks 0, 18, 16, 2) and 8 bytes of the values of
//            c = 2 tig (+ 1) (half a warp: keys x, x + 4, x + 8, x + 12, banks 0, 8, 16, 24).
//   D = 64:  a row is 9 banks; 4-byte loads of keys 8 a + e (e = 0, 1): banks 8 a + 9 e.
#pragma once

#include "kv4_common.cuh"
#include "kv_split.cuh"
#include "sync.cuh"

namespace cpattn {
namespace kvattn {

template <int D>
struct Granule {
  static constexpr int kKeys = kKeysOf<D>;
  static constexpr int kSteps = kKeys / 16;  // steps of 16 keys
  static constexpr int kRow = kv4::kRow<D>;
  static constexpr int kHalf = kKeys * kRow;  // bytes of K (or V): 2304
  static constexpr int kPair = 2 * kHalf;     // K (or V) of a stage, which holds one granule or two
};
// How many granules from g on go through the ring together, of those up to `end`: two from an even one on, which lie in one
// page or in whole pages.  One wait and one set of copies for two: the rings' upkeep was a quarter of the instructions.
__device__ __forceinline__ int together(int g, int end) { return (g & 1) == 0 && g + 1 < end ? 2 : 1; }

// Key of row c of group u (the operand's rows 8 u .. 8 u + 7) in step i.
template <int D>
__device__ __forceinline__ constexpr int key_at(int i, int u, int c) {
  return D == 128 ? 16 * i + 2 * u + (c & 1) + 8 * (c >> 1 & 1) + 4 * (c >> 2)
                  : 32 * (i >> 1) + 4 * (i & 1) + 2 * u + 8 * (c >> 1) + (c & 1);
}

__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// The operands of K in steps i0 and i0 + 1 of the granule at `tile`: use(j, a, b) for each 16 dimensions, a of the one
// step and b of the other, so that neighbouring products need not wait for one another.  Lane (gid, tig) holds dimensions
// D / 4 * tig .. + D / 4 - 1 of rows gid of both groups, four of them in each operand.
template <int D, class F>
__device__ __forceinline__ void key_operands(uint32_t tile, int i0, int gid, int tig, F&& use) {
  using G = Granule<D>;
  uint32_t word[2][2][D / 32], scale[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t row = tile + key_at<D>(i0 + i, u, gid) * G::kRow;
      if constexpr (D == 128) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint2 v = ptx::lds64(row + 16 * tig + 8 * q);
          word[i][u][2 * q] = v.x, word[i][u][2 * q + 1] = v.y;
        }
        scale[i][u] = lds16(row + 64 + 2 * tig);
      } else {
        word[i][u][0] = lds32(row + 8 * tig), word[i][u][1] = lds32(row + 8 * tig + 4);
        scale[i][u] = lds8(row + 32 + tig);
      }
    }
#pragma unroll
  for (int q = 0; q < D / 32; ++q) {
    uint32_t x[2][2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t s = kv4::scale_twice(scale[i][u], q >> 1);
        kv4::to_f16x2(word[i][u][q], x[i][u]);
#pragma unroll
        for (int h = 0; h < 4; ++h) x[i][u][h] = kv4::mul_f16x2(x[i][u][h], s);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a[4] = {x[0][0][2 * h], x[0][1][2 * h], x[0][0][2 * h + 1], x[0][1][2 * h + 1]};
      const uint32_t b[4] = {x[1][0][2 * h], x[1][1][2 * h], x[1][0][2 * h + 1], x[1][1][2 * h + 1]};
      use(2 * q + h, a, b);
    }
  }
}

// The operands of V^T in step i of the values at `tile`: use(w, a) for four tiles w .. w + 3 of 16 columns of O; rows gid
// and gid + 8 of tile w are columns D / 8 * gid + 2 w and + 1.  Nibbles of two keys are put side by side before they
// become halves.
template <int D, class F>
__device__ __forceinline__ void value_operands(uint32_t tile, int i, int gid, int tig, F&& use) {
  using G = Granule<D>;
  uint32_t word[4][D / 64], scale[2];
  {
    uint32_t byte[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t row = tile + key_at<D>(i, x >> 1, 2 * tig + (x & 1)) * G::kRow;
      if constexpr (D == 128) {
        const uint2 v = ptx::lds64(row + 8 * gid);
        word[x][0] = v.x, word[x][D / 64 - 1] = v.y;
        byte[x] = lds8(row + 64 + gid);
      } else {
        word[x][0] = lds32(row + 4 * gid);
        byte[x] = lds8(row + 32 + (gid >> 1));
      }
    }
    scale[0] = kv4::scale_pair(byte[0], byte[1]);
    scale[1] = kv4::scale_pair(byte[2], byte[3]);
  }
  constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    uint32_t h[2][2][4];  // [keys 2 x, 2 x + 1][even or odd column][column pair]
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t a = word[2 * x][q], b = word[2 * x + 1][q];
      kv4::to_f16x2((a & kLow) | ((b << 4) & ~kLow), h[x][0]);
      kv4::to_f16x2(((a >> 4) & kLow) | (b & ~kLow), h[x][1]);
    }
    uint32_t a[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j][0] = kv4::mul_f16x2(h[0][0][j], scale[0]), a[j][1] = kv4::mul_f16x2(h[0][1][j], scale[0]);
      a[j][2] = kv4::mul_f16x2(h[1][0][j], scale[1]), a[j][3] = kv4::mul_f16x2(h[1][1][j], scale[1]);
    }
    use(4 * q, a);
  }
}

// The operands of the lane's part of query row gid of a tile, whose elements begin at `at` (zeros where not `live`):
// dimensions D / 4 * tig and on, four to an operand, as QP f16 parts, qf[part][step].  The row is scaled by a power of two
// to at most 2^15, so a bf16 row is exact (over 2^28 of range) and an fp32 one split into a high and a low part has
// 22 bits.  Returns the factor that turns the products into scores in base 2.
template <int D, int QP>
__device__ __forceinline__ float query_operands(const Params& p, int64_t at, bool live, int tig,
                                                uint32_t (*qf)[D / 16][2]) {
  constexpr int kMt = D / 16;
  float x[kMt][4];
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < kMt; ++j) {
    if (live) load4(p, at + tig * (D / 4) + j * 4, x[j]);
    else x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[j][e]));
  }
  top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
  top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
  // 2^e <= top < 2^(e + 1) goes to [2^14, 2^15); rows of (almost) zeros keep a finite factor
  const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
  const float up = kv::pow2(14 - e);
#pragma unroll
  for (int j = 0; j < kMt; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float a = x[j][2 * h] * up, b = x[j][2 * h + 1] * up;
      qf[0][j][h] = to_f16x2(a, b);
      if (QP == 2) {
        const float2 back = from_f16x2(qf[0][j][h]);
        qf[QP - 1][j][h] = to_f16x2(a - back.x, b - back.y);
      }
    }
  // Kept above 0 and finite: else a masked product, -inf, or one of zeros would become NaN.  Where it is less than 2^-126 all
  // scores, of products below 2^39, are as good as 0.
  return fminf(fmaxf(p.scale_log2 * kv::pow2(e - 14), 0x1p-126f), 3.402823466e38f);
}

// Where a warp's copies are: the granules of its share, in order, into the stages of its ring.  TENSORS: K, or K and V.
template <int D, int TENSORS>
struct Feed {
  using G = Granule<D>;
  int b, head;  // sequence and KV head
  int keys;     // tokens of the sequence that are wanted
  int window, pages;  // lane i holds page window + i of the sequence, -1 behind its keys

  // Makes the window hold the pages ord .. ord + n - 1; n is at most 8.
  __device__ __forceinline__ void look(const Params& p, int lane, int ord, int n) {
    if (ord < window || ord + n > window + 32) {
      window = ord;
      // entries that hold no token are the caller's to change at any time: they are not read
      pages = -1;
      if ((static_cast<int64_t>(ord) + lane) << p.page_log2 < keys)
        pages = static_cast<int>(kv::page_at(p.rows, p.n_pages, b, ord + lane));
    }
  }
  // Stands in for tokens that have no page: keys that are NaN, which reach the rows that see them, and values of 0.
  __device__ __forceinline__ void stand_in(const Params& p, int lane, uint32_t dst, int rows) {
    for (int i = lane; i < rows * G::kRow / 4; i += 32) {
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 4 * i), "r"(0xffffffffu) : "memory");
      if (TENSORS == 2) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + G::kPair + 4 * i), "r"(0u) : "memory");
    }
    ptx::fence_proxy_async_smem();  // before the next copies into the stage
    __syncwarp();
    if (lane == 0) kv::report(p.status, kv::kSitePage);
  }
  // One lane's: copies `rows` rows, up to a whole group of 4, which is a multiple of 16 bytes and does not leave the page.
  __device__ __forceinline__ uint32_t copy(const Params& p, int page, int slot, int rows, uint32_t dst, uint32_t bar) {
    const uint32_t bytes = ((rows + 3) & ~3) * G::kRow;
    const int64_t at = static_cast<int64_t>((page * p.hkv + head) * p.page + slot) * G::kRow;  // rows: below 2^31
    ptx::bulk_load(dst, p.tile[0] + at, bytes, bar);
    if (TENSORS == 2) ptx::bulk_load(dst + G::kPair, p.tile[1] + at, bytes, bar);
    return TENSORS * bytes;
  }

  // Starts the copies of n granules from g on to `dst`, as far as there are tokens; they arrive at `bar`, whose phase ends
  // with this call's arrival and the bytes of the copies.  more(i, page, slot, rows) is called by one lane for each page's
  // part i, and answers with the bytes of its own copies to `bar`; page is -1 where there is none.
  template <class F>
  __device__ __forceinline__ void stage(const Params& p, int lane, int g, int n, uint32_t dst, uint32_t bar, F&& more) {
    const int key0 = g * G::kKeys;
    const int wanted = min(keys - key0, n * G::kKeys);
    const int ord = key0 >> p.page_log2;
    if (p.page >= n * G::kKeys) {
      look(p, lane, ord, 1);
      const int page = __shfl_sync(kFull, pages, ord - window);
      if (page < 0) stand_in(p, lane, dst, n * G::kKeys);
      if (lane == 0) {
        const int slot = key0 & (p.page - 1);
        uint32_t tx = more(0, page, slot, wanted);
        if (page >= 0) tx += copy(p, page, slot, wanted, dst, bar);
        ptx::mbar_arrive_expect_tx(bar, tx);
      }
      return;
    }
    // several pages: the lane that holds a page copies its part
    const int parts = (wanted + p.page - 1) >> p.page_log2;
    look(p, lane, ord, parts);
    const int i = lane - (ord - window);
    const bool mine = static_cast<unsigned>(i) < static_cast<unsigned>(parts);
    uint32_t tx = 0;
    if (mine) {
      const int rows = min(wanted - (i << p.page_log2), p.page);
      tx = more(i, pages, 0, rows);
      if (pages >= 0) tx += copy(p, pages, 0, rows, dst + (i << p.page_log2) * G::kRow, bar);
    }
    tx = __reduce_add_sync(kFull, tx);
    unsigned bad = __ballot_sync(kFull, mine && pages < 0) >> (ord - window);
    for (; bad != 0u; bad &= bad - 1u)
      stand_in(p, lane, dst + ((__ffs(bad) - 1) << p.page_log2) * G::kRow, p.page);
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, tx);
  }
  __device__ __forceinline__ void stage(const Params& p, int lane, int g, int n, uint32_t dst, uint32_t bar) {
    stage(p, lane, g, n, dst, bar, [](int, int, int, int) { return 0u; });
  }
};

}  // namespace kvattn
}  // namespace cpattn

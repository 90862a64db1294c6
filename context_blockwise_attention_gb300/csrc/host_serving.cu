// C entry points of the 8-bit cache and of the rotary positions: argument validation (host only,
// before any launch) and dispatch to the launchers.
#include <math.h>

#include "internal.h"

using namespace cpattn;

#define CP_INVALID(...)             \
  do {                              \
    cpattn::set_error(__VA_ARGS__); \
    return CP_ERR_INVALID_ARG;      \
  } while (0)

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

cp_status validate_cache(const char* who, const cp_kv_cache& c) {
  if (c.d != 64 && c.d != 128) CP_INVALID("%s: head_dim %d not in {64, 128}", who, c.d);
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
    CP_INVALID("%s: page_size %d not in {16, 32, 64, 128}", who, c.page_size);
  if (c.hkv <= 0) CP_INVALID("%s: head counts must be positive", who);
  if (c.n_pages < 0) CP_INVALID("%s: negative page count", who);
  // rows of the cache seen as [n_pages * hkv * page_size, d], and page ids, stay int32
  if (c.n_pages > INT32_MAX / (static_cast<int64_t>(c.hkv) * c.page_size))
    CP_INVALID("%s: n_pages * hkv * page_size must stay below 2^31", who);
  if (c.reserved != 0) CP_INVALID("%s: cache.reserved must be 0", who);
  if (c.n_pages > 0) {
    if (c.k == nullptr || c.v == nullptr || c.k_scale == nullptr || c.v_scale == nullptr)
      CP_INVALID("%s: the cache's k, v, k_scale and v_scale must not be NULL", who);
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))
      CP_INVALID("%s: the cache's k and v must be 16-byte aligned, its scales 4-byte aligned", who);
  }
  return CP_OK;
}

cp_status validate_rows(const char* who, const cp_kv_rows& r) {
  if (r.n_seqs < 0 || r.n_seqs > CP_KV_MAX_SEQS)
    CP_INVALID("%s: n_seqs %d not in [0, %d]", who, r.n_seqs, CP_KV_MAX_SEQS);
  if (r.n_rows < 0 || r.n_rows > (int64_t(1) << 31) - 256) CP_INVALID("%s: n_rows out of range", who);
  if (r.n_seqs > 0) {
    if (r.max_pages < 1) CP_INVALID("%s: max_pages must be positive", who);
    if (r.row_start == nullptr || r.tokens == nullptr || r.page_table == nullptr)
      CP_INVALID("%s: row_start, tokens and page_table must not be NULL", who);
    if (!aligned(r.row_start, 4) || !aligned(r.tokens, 4) || !aligned(r.page_table, 4))
      CP_INVALID("%s: row_start, tokens and page_table must be 4-byte aligned", who);
  }
  return CP_OK;
}

cp_status validate_copy(const char* who, const cp_kv_cache* cache, const cp_kv_rows* rows, const void* k,
                        const void* v, int32_t dtype, const int32_t* status) {
  if (cache == nullptr || rows == nullptr) CP_INVALID("%s: cache and rows must not be NULL", who);
  cp_status st = validate_cache(who, *cache);
  if (st != CP_OK) return st;
  if ((st = validate_rows(who, *rows)) != CP_OK) return st;
  if (dtype != CP_F32 && dtype != CP_BF16) CP_INVALID("%s: dtype %d is not CP_F32 or CP_BF16", who, dtype);
  if (!aligned(status, 4)) CP_INVALID("%s: status must be 4-byte aligned", who);
  if (rows->n_rows > 0) {
    if (k == nullptr || v == nullptr) CP_INVALID("%s: k and v must not be NULL", who);
    if (!aligned(k, 16) || !aligned(v, 16)) CP_INVALID("%s: k and v must be 16-byte aligned", who);
  }
  return CP_OK;
}

cp_status validate_attn(const char* who, const cp_kv_attn_desc& d) {
  cp_status st = validate_cache(who, d.cache);
  if (st != CP_OK) return st;
  if ((st = validate_rows(who, d.rows)) != CP_OK) return st;
  if (d.in_dtype != CP_F32 && d.in_dtype != CP_BF16)
    CP_INVALID("%s: in_dtype %d is not CP_F32 or CP_BF16", who, d.in_dtype);
  if (d.o_dtype != CP_F32 && d.o_dtype != CP_BF16)
    CP_INVALID("%s: o_dtype %d is not CP_F32 or CP_BF16", who, d.o_dtype);
  if (d.hq <= 0) CP_INVALID("%s: head counts must be positive", who);
  if (d.hq % d.cache.hkv != 0) CP_INVALID("%s: hq %d is not a multiple of hkv %d", who, d.hq, d.cache.hkv);
  if (static_cast<int64_t>(d.rows.max_pages) * d.cache.page_size > 2000000000)
    CP_INVALID("%s: max_pages * page_size exceeds 2e9 tokens", who);
  if (d.rows.n_rows * d.hq > 0x7fffff00)  // query rows, rounded up to their blocks, stay int32
    CP_INVALID("%s: n_rows * hq must stay below 2^31", who);
  return CP_OK;
}

// The fraction of a turn per position, inv_freq / 2 pi, in units of 2^-64 and modulo one turn.
// 1 / 2 pi is taken to twice fp64's precision: times a position of up to 2^31 one fp64 rounding
// would show in the result.
uint64_t turn_of(double inv_freq) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  const double f = fabs(inv_freq), w = f * hi;  // below 2^8
  const double rest = fma(f, hi, -w) + f * lo;
  const double part = w - static_cast<double>(static_cast<int64_t>(w));
  uint64_t u = static_cast<uint64_t>(part * 0x1p64);  // exact: part is below 1
  u += static_cast<uint64_t>(static_cast<int64_t>(rest * 0x1p64));
  return inv_freq < 0.0 ? uint64_t(0) - u : u;
}

}  // namespace

CP_API cp_status cp_kv_cache_write(const cp_kv_cache* cache, const cp_kv_rows* rows, const void* k, const void* v,
                                   int32_t in_dtype, int32_t* status, cudaStream_t stream) {
  clear_error();
  cp_status st = validate_copy("cp_kv_cache_write", cache, rows, k, v, in_dtype, status);
  if (st != CP_OK) return st;
  if (rows->n_rows == 0 || rows->n_seqs == 0) return CP_OK;
  // units of work (page, head, K or V) are numbered in 32 bits
  if ((rows->n_rows / cache->page_size + 2 * static_cast<int64_t>(rows->n_seqs)) * cache->hkv > INT32_MAX)
    CP_INVALID("cp_kv_cache_write: (n_rows / page_size + 2 n_seqs) * hkv must stay below 2^31");
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  if (status != nullptr && (st = launch_kv_check(*rows, status, stream)) != CP_OK) return st;
  return launch_kv_write(*cache, *rows, k, v, in_dtype == CP_BF16, status, sms, stream);
}

CP_API cp_status cp_kv_cache_read(const cp_kv_cache* cache, const cp_kv_rows* rows, void* k, void* v,
                                  int32_t out_dtype, int32_t* status, cudaStream_t stream) {
  clear_error();
  cp_status st = validate_copy("cp_kv_cache_read", cache, rows, k, v, out_dtype, status);
  if (st != CP_OK) return st;
  if (rows->n_rows == 0 || rows->n_seqs == 0) return CP_OK;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  if (status != nullptr && (st = launch_kv_check(*rows, status, stream)) != CP_OK) return st;
  return launch_kv_read(*cache, *rows, k, v, out_dtype == CP_BF16, status, sms, stream);
}

CP_API cp_status cp_kv_cache_attn_workspace(const cp_kv_attn_desc* desc, int64_t* bytes_out) {
  clear_error();
  const char* who = "cp_kv_cache_attn_workspace";
  if (desc == nullptr || bytes_out == nullptr) CP_INVALID("%s: desc and bytes_out must not be NULL", who);
  cp_status st = validate_attn(who, *desc);
  if (st != CP_OK) return st;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  *bytes_out = kv_attn_workspace(*desc, sms);
  return CP_OK;
}

CP_API cp_status cp_kv_cache_attn(const cp_kv_attn_desc* desc, cudaStream_t stream) {
  clear_error();
  const char* who = "cp_kv_cache_attn";
  if (desc == nullptr) CP_INVALID("%s: desc is NULL", who);
  const cp_kv_attn_desc& d = *desc;
  cp_status st = validate_attn(who, d);
  if (st != CP_OK) return st;
  if (d.kv_pos.stride < 1) CP_INVALID("%s: position strides must be >= 1", who);
  if (d.kv_pos.base < 0) CP_INVALID("%s: positions must be >= 0", who);
  if (d.kv_pos.stride > 2000000000 || d.kv_pos.base > 2000000000) CP_INVALID("%s: global positions exceed 2e9", who);
  if (!(d.scale >= 0.0f) || isinf(d.scale)) CP_INVALID("%s: scale must be finite and >= 0", who);
  if (d.flags & ~CP_FLAG_TEST_STALL) CP_INVALID("%s: unknown flag bits 0x%x", who, d.flags);
  if (d.wait_timeout_ms < 0) CP_INVALID("%s: wait_timeout_ms must be >= 0", who);
  if (!aligned(d.status, 4) || !aligned(d.q_first, 4)) CP_INVALID("%s: status and q_first must be 4-byte aligned", who);
  if (d.rows.n_rows == 0 || d.rows.n_seqs == 0) return CP_OK;
  if (d.cache.n_pages == 0) CP_INVALID("%s: the cache has no pages", who);
  if (d.q == nullptr || d.o == nullptr || d.lse == nullptr) CP_INVALID("%s: q, o and lse must not be NULL", who);
  if (!aligned(d.q, 16) || !aligned(d.o, 16) || !aligned(d.lse, 4))
    CP_INVALID("%s: q and o must be 16-byte aligned, lse 4-byte aligned", who);
  if (d.workspace_bytes < 0 || !aligned(d.workspace, 16) || (d.workspace == nullptr && d.workspace_bytes > 0))
    CP_INVALID("%s: workspace must be 16-byte aligned device memory of workspace_bytes", who);
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  const int64_t need = kv_attn_workspace(d, sms);
  if (d.workspace_bytes < need)
    CP_INVALID("%s: the workspace has %lld bytes, %lld are needed (cp_kv_cache_attn_workspace)", who,
               static_cast<long long>(d.workspace_bytes), static_cast<long long>(need));
  const float scale = d.scale > 0.0f ? d.scale : 1.0f / sqrtf(static_cast<float>(d.cache.d));
  const int64_t timeout_ns = static_cast<int64_t>(d.wait_timeout_ms > 0 ? d.wait_timeout_ms : 2000) * 1000000LL;
  if (d.status != nullptr && (st = launch_kv_check(d.rows, d.status, stream)) != CP_OK) return st;
  return launch_kv_attn(d, scale, timeout_ns, sms, stream);
}

CP_API cp_status cp_rope_axes(int32_t n_tensors, const void* const* in, void* const* out, const int32_t* heads,
                              int64_t tokens, int32_t d, int32_t rot, int32_t dtype, const int32_t* positions,
                              int32_t n_axes, const int32_t* sections, const double* inv_freq, int32_t interleaved,
                              int32_t inverse, cudaStream_t stream) {
  clear_error();
  const char* who = "cp_rope_axes";
  if (n_tensors < 1 || n_tensors > 4) CP_INVALID("%s: n_tensors=%d not in [1, 4]", who, n_tensors);
  if (in == nullptr || out == nullptr || heads == nullptr || sections == nullptr || inv_freq == nullptr)
    CP_INVALID("%s: in, out, heads, sections and inv_freq must not be NULL", who);
  if (tokens < 0 || tokens > (int64_t(1) << 31) - 256) CP_INVALID("%s: tokens out of range", who);
  if (d < 8 || d > 256 || d % 8 != 0) CP_INVALID("%s: head_dim %d is not a multiple of 8 up to 256", who, d);
  if (rot < 16 || rot > d || rot % 16 != 0)
    CP_INVALID("%s: rot %d is not a multiple of 16 from 16 to head_dim %d", who, rot, d);
  if (dtype != CP_F32 && dtype != CP_BF16) CP_INVALID("%s: dtype %d is not CP_F32 or CP_BF16", who, dtype);
  if (n_axes < 1 || n_axes > 4) CP_INVALID("%s: n_axes=%d not in [1, 4]", who, n_axes);
  if (interleaved != 0 && interleaved != 1) CP_INVALID("%s: interleaved must be 0 or 1", who);
  if (inverse != 0 && inverse != 1) CP_INVALID("%s: inverse must be 0 or 1", who);
  int64_t sum = 0;
  for (int i = 0; i < n_axes; ++i) {
    if (sections[i] < 0) CP_INVALID("%s: section %d is negative", who, i);
    sum += sections[i];
  }
  if (sum != rot / 2) CP_INVALID("%s: the sections cover %lld pairs, not rot/2 = %d", who, (long long)sum, rot / 2);
  int64_t all = 0;
  for (int t = 0; t < n_tensors; ++t) {
    if (heads[t] <= 0) CP_INVALID("%s: head counts must be positive", who);
    all += heads[t];
  }
  if (all > 65536) CP_INVALID("%s: more than 65536 heads in all", who);
  RopeArgs a{n_tensors, in, out, heads, tokens, d, rot, dtype == CP_BF16, positions, n_axes, sections,
             interleaved, inverse, {}};
  for (int i = 0; i < rot / 2; ++i) {
    if (!(fabs(inv_freq[i]) <= 1e3)) CP_INVALID("%s: inv_freq[%d] is not finite or above 1e3", who, i);
    a.turn[i] = turn_of(inv_freq[i]);
  }
  if (tokens == 0) return CP_OK;
  if (positions == nullptr || !aligned(positions, 4)) CP_INVALID("%s: positions must not be NULL", who);
  for (int t = 0; t < n_tensors; ++t) {
    if (in[t] == nullptr || out[t] == nullptr) CP_INVALID("%s: in[%d] and out[%d] must not be NULL", who, t, t);
    if (!aligned(in[t], 16) || !aligned(out[t], 16)) CP_INVALID("%s: every tensor must be 16-byte aligned", who);
  }
  int sms = 0;
  cp_status st = require_sm103(nullptr, &sms);
  if (st != CP_OK) return st;
  return launch_rope(a, sms, stream);
}

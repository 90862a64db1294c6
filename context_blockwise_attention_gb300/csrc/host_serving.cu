// C entry points of the 8-bit and 4-bit caches and of the rotary positions: argument validation (host only,
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

cp_status validate_pool(const char* who, int64_t n_pages, int32_t page_size, int32_t hkv, int32_t d, int32_t reserved) {
  if (d != 64 && d != 128) CP_INVALID("%s: head_dim %d not in {64, 128}", who, d);
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    CP_INVALID("%s: page_size %d not in {16, 32, 64, 128}", who, page_size);
  if (hkv <= 0) CP_INVALID("%s: head counts must be positive", who);
  if (n_pages < 0) CP_INVALID("%s: negative page count", who);
  // rows of the cache seen as [n_pages * hkv * page_size, d], and page ids, stay int32
  if (n_pages > INT32_MAX / (static_cast<int64_t>(hkv) * page_size))
    CP_INVALID("%s: n_pages * hkv * page_size must stay below 2^31", who);
  if (reserved != 0) CP_INVALID("%s: cache.reserved must be 0", who);
  return CP_OK;
}

cp_status validate_cache(const char* who, const cp_kv_cache& c) {
  const cp_status st = validate_pool(who, c.n_pages, c.page_size, c.hkv, c.d, c.reserved);
  if (st != CP_OK) return st;
  if (c.n_pages > 0) {
    if (c.k == nullptr || c.v == nullptr || c.k_scale == nullptr || c.v_scale == nullptr)
      CP_INVALID("%s: the cache's k, v, k_scale and v_scale must not be NULL", who);
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))
      CP_INVALID("%s: the cache's k and v must be 16-byte aligned, its scales 4-byte aligned", who);
  }
  return CP_OK;
}

// values: whether the call looks at V.
cp_status validate_cache(const char* who, const cp_kv4_cache& c, bool values = true) {
  const cp_status st = validate_pool(who, c.n_pages, c.page_size, c.hkv, c.d, c.reserved);
  if (st != CP_OK) return st;
  if (c.hkv > 65536) CP_INVALID("%s: more than 65536 KV heads", who);
  if (c.n_pages > 0) {
    if (c.k == nullptr || (values && c.v == nullptr)) CP_INVALID("%s: the cache's k and v must not be NULL", who);
    if (!aligned(c.k, 16) || (values && !aligned(c.v, 16)))
      CP_INVALID("%s: the cache's k and v must be 16-byte aligned", who);
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

template <class Cache>
cp_status validate_copy(const char* who, const Cache* cache, const cp_kv_rows* rows, const void* k,
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

// What attention and the weights that it gives have in common.
cp_status validate_queries(const char* who, const cp_kv_rows& rows, int32_t page_size, int32_t hkv, int32_t hq,
                           int32_t in_dtype) {
  const cp_status st = validate_rows(who, rows);
  if (st != CP_OK) return st;
  if (in_dtype != CP_F32 && in_dtype != CP_BF16) CP_INVALID("%s: in_dtype %d is not CP_F32 or CP_BF16", who, in_dtype);
  if (hq <= 0) CP_INVALID("%s: head counts must be positive", who);
  if (hq % hkv != 0) CP_INVALID("%s: hq %d is not a multiple of hkv %d", who, hq, hkv);
  if (static_cast<int64_t>(rows.max_pages) * page_size > 2000000000)
    CP_INVALID("%s: max_pages * page_size exceeds 2e9 tokens", who);
  if (rows.n_rows * hq > 0x7fffff00)  // query rows, rounded up to their blocks, stay int32
    CP_INVALID("%s: n_rows * hq must stay below 2^31", who);
  return CP_OK;
}

cp_status validate_call(const char* who, const cp_posmap& kv_pos, float scale, int32_t flags, int32_t wait_timeout_ms,
                        const int32_t* status, const int32_t* q_first) {
  if (kv_pos.stride < 1) CP_INVALID("%s: position strides must be >= 1", who);
  if (kv_pos.base < 0) CP_INVALID("%s: positions must be >= 0", who);
  if (kv_pos.stride > 2000000000 || kv_pos.base > 2000000000) CP_INVALID("%s: global positions exceed 2e9", who);
  // the kernels take scores in base 2
  if (!(scale >= 0.0f) || isinf(scale * 1.4426950408889634f)) CP_INVALID("%s: scale must be >= 0 and at most 2e38", who);
  if (flags & ~CP_FLAG_TEST_STALL) CP_INVALID("%s: unknown flag bits 0x%x", who, flags);
  if (wait_timeout_ms < 0) CP_INVALID("%s: wait_timeout_ms must be >= 0", who);
  if (!aligned(status, 4) || !aligned(q_first, 4)) CP_INVALID("%s: status and q_first must be 4-byte aligned", who);
  return CP_OK;
}

cp_status validate_workspace(const char* who, const void* workspace, int64_t bytes) {
  if (bytes < 0 || !aligned(workspace, 16) || (workspace == nullptr && bytes > 0))
    CP_INVALID("%s: workspace must be 16-byte aligned device memory of workspace_bytes", who);
  return CP_OK;
}

template <class Desc>
cp_status validate_attn(const char* who, const Desc& d) {
  cp_status st = validate_cache(who, d.cache);
  if (st != CP_OK) return st;
  if ((st = validate_queries(who, d.rows, d.cache.page_size, d.cache.hkv, d.hq, d.in_dtype)) != CP_OK) return st;
  if (d.o_dtype != CP_F32 && d.o_dtype != CP_BF16)
    CP_INVALID("%s: o_dtype %d is not CP_F32 or CP_BF16", who, d.o_dtype);
  return CP_OK;
}

cp_status validate_evict(const char* who, const cp_kv4_evict_desc& d) {
  const cp_status st = validate_cache(who, d.cache);
  if (st != CP_OK) return st;
  if (d.n_seqs < 0 || d.n_seqs > CP_KV_MAX_SEQS)
    CP_INVALID("%s: n_seqs %d not in [0, %d]", who, d.n_seqs, CP_KV_MAX_SEQS);
  if (d.keep < 1) CP_INVALID("%s: keep must be positive", who);
  if (d.recent < 0 || d.recent > d.keep) CP_INVALID("%s: recent %d not in [0, keep = %d]", who, d.recent, d.keep);
  if (static_cast<int64_t>(d.n_seqs) * d.keep > INT32_MAX) CP_INVALID("%s: n_seqs * keep must stay below 2^31", who);
  if (d.n_seqs > 0 && d.max_pages < 1) CP_INVALID("%s: max_pages must be positive", who);
  if (static_cast<int64_t>(d.max_pages) * d.cache.page_size > 2000000000)
    CP_INVALID("%s: max_pages * page_size exceeds 2e9 tokens", who);
  return CP_OK;
}

template <class Desc>
cp_status attn_workspace(const char* who, const Desc* desc, int64_t* bytes_out, int64_t (*need)(const Desc&, int)) {
  clear_error();
  if (desc == nullptr || bytes_out == nullptr) CP_INVALID("%s: desc and bytes_out must not be NULL", who);
  cp_status st = validate_attn(who, *desc);
  if (st != CP_OK) return st;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  *bytes_out = need(*desc, sms);
  return CP_OK;
}

template <class Desc>
cp_status attn(const char* who, const Desc* desc, cudaStream_t stream, int64_t (*workspace)(const Desc&, int),
               cp_status (*launch)(const Desc&, float, int64_t, int, cudaStream_t)) {
  clear_error();
  if (desc == nullptr) CP_INVALID("%s: desc is NULL", who);
  const Desc& d = *desc;
  cp_status st = validate_attn(who, d);
  if (st != CP_OK) return st;
  if ((st = validate_call(who, d.kv_pos, d.scale, d.flags, d.wait_timeout_ms, d.status, d.q_first)) != CP_OK) return st;
  if (d.rows.n_rows == 0 || d.rows.n_seqs == 0) return CP_OK;
  if (d.cache.n_pages == 0) CP_INVALID("%s: the cache has no pages", who);
  if (d.q == nullptr || d.o == nullptr || d.lse == nullptr) CP_INVALID("%s: q, o and lse must not be NULL", who);
  if (!aligned(d.q, 16) || !aligned(d.o, 16) || !aligned(d.lse, 4))
    CP_INVALID("%s: q and o must be 16-byte aligned, lse 4-byte aligned", who);
  if ((st = validate_workspace(who, d.workspace, d.workspace_bytes)) != CP_OK) return st;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  const int64_t need = workspace(d, sms);
  if (d.workspace_bytes < need)
    CP_INVALID("%s: the workspace has %lld bytes, %lld are needed (%s_workspace)", who,
               static_cast<long long>(d.workspace_bytes), static_cast<long long>(need), who);
  const float scale = d.scale > 0.0f ? d.scale : 1.0f / sqrtf(static_cast<float>(d.cache.d));
  const int64_t timeout_ns = static_cast<int64_t>(d.wait_timeout_ms > 0 ? d.wait_timeout_ms : 2000) * 1000000LL;
  if (d.status != nullptr && (st = launch_kv_check(d.rows, d.status, stream)) != CP_OK) return st;
  return launch(d, scale, timeout_ns, sms, stream);
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
  return attn_workspace("cp_kv_cache_attn_workspace", desc, bytes_out, kv_attn_workspace);
}

CP_API cp_status cp_kv_cache_attn(const cp_kv_attn_desc* desc, cudaStream_t stream) {
  return attn("cp_kv_cache_attn", desc, stream, kv_attn_workspace, launch_kv_attn);
}

CP_API cp_status cp_kv4_cache_write(const cp_kv4_cache* cache, const cp_kv_rows* rows, const void* k, const void* v,
                                    int32_t in_dtype, int32_t* status, cudaStream_t stream) {
  clear_error();
  cp_status st = validate_copy("cp_kv4_cache_write", cache, rows, k, v, in_dtype, status);
  if (st != CP_OK) return st;
  if (rows->n_rows == 0 || rows->n_seqs == 0) return CP_OK;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  if (status != nullptr && (st = launch_kv_check(*rows, status, stream)) != CP_OK) return st;
  return launch_kv4_write(*cache, *rows, k, v, in_dtype == CP_BF16, status, sms, stream);
}

CP_API cp_status cp_kv4_cache_read(const cp_kv4_cache* cache, const cp_kv_rows* rows, void* k, void* v,
                                   int32_t out_dtype, int32_t* status, cudaStream_t stream) {
  clear_error();
  cp_status st = validate_copy("cp_kv4_cache_read", cache, rows, k, v, out_dtype, status);
  if (st != CP_OK) return st;
  if (rows->n_rows == 0 || rows->n_seqs == 0) return CP_OK;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  if (status != nullptr && (st = launch_kv_check(*rows, status, stream)) != CP_OK) return st;
  return launch_kv4_read(*cache, *rows, k, v, out_dtype == CP_BF16, status, sms, stream);
}

CP_API cp_status cp_kv4_cache_attn_workspace(const cp_kv4_attn_desc* desc, int64_t* bytes_out) {
  return attn_workspace("cp_kv4_cache_attn_workspace", desc, bytes_out, kv4_attn_workspace);
}

CP_API cp_status cp_kv4_cache_attn(const cp_kv4_attn_desc* desc, cudaStream_t stream) {
  return attn("cp_kv4_cache_attn", desc, stream, kv4_attn_workspace, launch_kv4_attn);
}

CP_API cp_status cp_kv4_cache_weigh(const cp_kv4_weigh_desc* desc, cudaStream_t stream) {
  clear_error();
  const char* who = "cp_kv4_cache_weigh";
  if (desc == nullptr) CP_INVALID("%s: desc is NULL", who);
  const cp_kv4_weigh_desc& d = *desc;
  cp_status st = validate_cache(who, d.cache, false);
  if (st != CP_OK) return st;
  if ((st = validate_queries(who, d.rows, d.cache.page_size, d.cache.hkv, d.hq, d.in_dtype)) != CP_OK) return st;
  if ((st = validate_call(who, d.kv_pos, d.scale, d.flags, d.wait_timeout_ms, d.status, d.q_first)) != CP_OK) return st;
  if (!(d.decay >= 0.0f && d.decay <= 1.0f)) CP_INVALID("%s: decay must be in [0, 1]", who);
  if (!aligned(d.known, 4)) CP_INVALID("%s: known must be 4-byte aligned", who);
  if (d.rows.n_rows == 0 || d.rows.n_seqs == 0) return CP_OK;
  if (d.cache.n_pages == 0) CP_INVALID("%s: the cache has no pages", who);
  if (d.weight == nullptr || d.q == nullptr || d.lse == nullptr) CP_INVALID("%s: weight, q and lse must not be NULL", who);
  if (!aligned(d.weight, 16) || !aligned(d.q, 16) || !aligned(d.lse, 4))
    CP_INVALID("%s: weight and q must be 16-byte aligned, lse 4-byte aligned", who);
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  const float scale = d.scale > 0.0f ? d.scale : 1.0f / sqrtf(static_cast<float>(d.cache.d));
  const int64_t timeout_ns = static_cast<int64_t>(d.wait_timeout_ms > 0 ? d.wait_timeout_ms : 2000) * 1000000LL;
  if (d.status != nullptr && (st = launch_kv_check(d.rows, d.status, stream)) != CP_OK) return st;
  return launch_kv4_weigh(d, scale, timeout_ns, sms, stream);
}

CP_API cp_status cp_kv4_cache_evict_workspace(const cp_kv4_evict_desc* desc, int64_t* bytes_out) {
  clear_error();
  const char* who = "cp_kv4_cache_evict_workspace";
  if (desc == nullptr || bytes_out == nullptr) CP_INVALID("%s: desc and bytes_out must not be NULL", who);
  cp_status st = validate_evict(who, *desc);
  if (st != CP_OK) return st;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  *bytes_out = kv4_evict_workspace(*desc, sms);
  return CP_OK;
}

CP_API cp_status cp_kv4_cache_evict(const cp_kv4_evict_desc* desc, cudaStream_t stream) {
  clear_error();
  const char* who = "cp_kv4_cache_evict";
  if (desc == nullptr) CP_INVALID("%s: desc is NULL", who);
  const cp_kv4_evict_desc& d = *desc;
  cp_status st = validate_evict(who, d);
  if (st != CP_OK) return st;
  if (!aligned(d.status, 4)) CP_INVALID("%s: status must be 4-byte aligned", who);
  if (d.n_seqs == 0) return CP_OK;
  if (d.cache.n_pages == 0) CP_INVALID("%s: the cache has no pages", who);
  if (d.weight == nullptr || d.tokens == nullptr || d.page_table == nullptr || d.kept == nullptr || d.new_tokens == nullptr)
    CP_INVALID("%s: weight, tokens, page_table, kept and new_tokens must not be NULL", who);
  if (!aligned(d.weight, 16) || !aligned(d.tokens, 4) || !aligned(d.page_table, 4) || !aligned(d.kept, 4) ||
      !aligned(d.new_tokens, 4))
    CP_INVALID("%s: weight must be 16-byte aligned; tokens, page_table, kept and new_tokens 4-byte aligned", who);
  if ((st = validate_workspace(who, d.workspace, d.workspace_bytes)) != CP_OK) return st;
  int sms = 0;
  if ((st = require_sm103(nullptr, &sms)) != CP_OK) return st;
  const int64_t need = kv4_evict_workspace(d, sms);
  if (d.workspace_bytes < need)
    CP_INVALID("%s: the workspace has %lld bytes, %lld are needed (%s_workspace)", who,
               static_cast<long long>(d.workspace_bytes), static_cast<long long>(need), who);
  return launch_kv4_evict(d, sms, stream);
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

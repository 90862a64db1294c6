// Attention over the paged 8-bit cache: the choice of the kernel variant, workspace and launch.
#include "kv_attn.cuh"

namespace cpattn {

using namespace kvattn;

namespace kvattn {
extern template cp_status run_d<64>(const Params&, const Plan&, const CUtensorMap&, const CUtensorMap&, int64_t, int,
                                    cudaStream_t);
extern template cp_status run_d<128>(const Params&, const Plan&, const CUtensorMap&, const CUtensorMap&, int64_t, int,
                                     cudaStream_t);
}  // namespace kvattn

namespace {

Plan plan_of(const cp_kv_attn_desc& d, int sms) {
  Plan r;
  const int64_t group = d.hq / d.cache.hkv, seqs = d.rows.n_seqs > 0 ? d.rows.n_seqs : 1;
  const int64_t per = (d.rows.n_rows + seqs - 1) / seqs * group;
  r.qp = d.in_dtype == CP_BF16 ? 1 : 2;
  r.pp = d.in_dtype == CP_BF16 && d.o_dtype == CP_BF16 ? 1 : 2;
  // Two tiles of rows at once halve the copies and conversions, at 8 warps an SM (12 x 8192-16384 tokens, one
  // against two tiles: D = 128, 16 rows 95 / 81 us, 32 rows 154 / 123; D = 64, 16 rows 49 / 61, 32 rows 78 / 79,
  // 64 rows 140 / 124).
  r.nt = per <= (d.cache.d == 128 ? 8 : 32) ? 1 : 2;
  r.rows = r.nt * 8;
  r.warps = r.nt * d.cache.d >= 256 || r.nt * r.qp >= 4 ? 8 : 12;
  // numbers at most, in fp64: the page table's width times the heads may pass 64 bits
  r.most = (static_cast<double>(d.rows.max_pages) * d.cache.page_size * d.cache.d / 4096 + 1 + kSetup) * d.cache.hkv *
           static_cast<double>(seqs + d.rows.n_rows * group / r.rows);
  r.grid = r.most < sms ? static_cast<int64_t>(r.most) : sms;
  // Solo: no more items than SMs, and few granules to a warp by the page table's width: 4, or 16 where the
  // items occupy most SMs (1 x 8 items of 1024 / 2048 tokens at D = 128: 9.6 / 14.0 us against 11.6 / 12.1
  // split; 18 x 8 items of 2048 / 6144: 14.7 / 35.7 against 19.9 / 39.6).  One row a sequence, as far as can
  // be told from their numbers, or few rows in all, since a block takes blocks of rows one after the other.
  const int64_t width = (static_cast<int64_t>(d.rows.max_pages) * d.cache.page_size * d.cache.d + 4095) / 4096;
  const int64_t solo_items = seqs * d.cache.hkv;
  r.solo = solo_items <= sms && width <= r.warps * (2 * solo_items > sms ? 16 : 4) &&
           (d.rows.n_rows <= seqs || d.rows.n_rows * group <= 4 * r.rows);
  if (r.solo) {
    r.grid = solo_items;
    r.ml_off = r.o_off = r.aside_off = r.bytes = 0;
    return r;
  }
  const int64_t slots = r.grid * r.warps * 2 * r.rows;
  r.ml_off = 0;
  r.o_off = (r.ml_off + slots * 8 + 255) / 256 * 256;
  r.aside_off = r.o_off + slots * d.cache.d * 4;
  r.bytes = r.aside_off + slots / 2 * d.cache.d * 4;
  return r;
}

}  // namespace

int64_t kv_attn_workspace(const cp_kv_attn_desc& d, int num_sms) { return plan_of(d, num_sms).bytes; }

cp_status launch_kv_attn(const cp_kv_attn_desc& d, float scale, int64_t timeout_ns, int num_sms, cudaStream_t s) {
  const Plan pl = plan_of(d, num_sms);
  if (pl.most > 1e12) {  // their products with a worker's number stay int64
    set_error("cp_kv_cache_attn: max_pages * page_size * hkv * n_seqs is too large for one call");
    return CP_ERR_INVALID_ARG;
  }
  const cp_kv_cache& c = d.cache;
  const int64_t lines = c.n_pages * c.hkv * c.page_size * c.d / 128;
  const int keys = 4096 / c.d;
  const int box = (c.page_size < keys ? c.page_size : keys) * c.d / 128;
  CUtensorMap mk, mv;
  if (!encode_map_bytes(&mk, c.k, lines, box) || !encode_map_bytes(&mv, c.v, lines, box)) {
    set_error("cp_kv_cache_attn: tensor map encoding failed");
    return CP_ERR_CUDA;
  }
  uint8_t* const ws = static_cast<uint8_t*>(d.workspace);
  Params p{};
  p.scale[0] = c.k_scale;
  p.scale[1] = c.v_scale;
  p.rows = d.rows;
  p.n_pages = c.n_pages;
  p.q = d.q;
  p.o = d.o;
  p.lse = d.lse;
  p.q_first = d.q_first;
  p.hq = d.hq;
  p.hkv = c.hkv;
  p.group = d.hq / c.hkv;
  p.page = c.page_size;
  p.page_log2 = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.q_bf16 = d.in_dtype == CP_BF16;
  p.o_bf16 = d.o_dtype == CP_BF16;
  p.stall = (d.flags & CP_FLAG_TEST_STALL) != 0;
  p.scale_log2 = scale * kLog2e;
  p.kv_pos = d.kv_pos;
  p.status = d.status;
  p.timeout_ns = timeout_ns;
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + pl.o_off);
  p.aside = reinterpret_cast<float*>(ws + pl.aside_off);
  const int64_t seqs = d.rows.n_seqs;
  const int64_t items = (seqs + d.rows.n_rows * p.group / pl.rows) * c.hkv;
  p.few = 128 * items;
  return c.d == 128 ? run_d<128>(p, pl, mk, mv, items, num_sms, s) : run_d<64>(p, pl, mk, mv, items, num_sms, s);
}

}  // namespace cpattn

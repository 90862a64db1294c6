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
  const auto tiles = [&](int nt) {
    r.nt = nt;
    r.rows = nt * 8;
    r.warps = nt * d.cache.d >= 256 || nt * r.qp >= 4 ? 8 : 12;
  };
  // Solo, by the page table's width in granules: as many blocks an item as the SMs hold clusters of (12 to 15 of
  // 8 blocks, 36 of 4), where a block's warps have some granules each (32/8 heads, D = 128: 1 x 1000 / 4000
  // tokens 9.4 / 20.6 us with one block, 8.5 / 10.0 with 8; 4 x 4000 21.1, 11.9 with 4; 8 x 4000 21.1, 15.8 with 2;
  // 1 x 500 7.4, 8.4 with 8), as long as splitting is slower, which uses all SMs but has a second kernel: 1 x 4000
  // tokens 10.0 us against 12.8, 4 x 4000 11.9 / 16.6, 4 x 8000 16.0 / 20.0, 8 x 4000 15.8 / 18.6, one KV head of
  // 4000 9.5 / 9.6, of 8000 11.8 / 10.7; 18 x 8 items of 2048 / 6144 tokens, one block each, 14.7 / 35.7 against
  // 19.9 / 39.6.  One row a sequence, as far as can be told from their numbers, or few rows in all, since the
  // blocks take an item's blocks of rows one after the other.
  tiles(per <= 8 ? 1 : 2);
  const int64_t width = (static_cast<int64_t>(d.rows.max_pages) * d.cache.page_size * d.cache.d + 4095) / 4096;
  const int64_t solo_items = seqs * d.cache.hkv;
  r.cluster = 1;
  if (width > 2 * r.warps) {
    if (solo_items * 8 <= sms * 5 / 8) r.cluster = 8;
    else if (solo_items * 4 <= sms * 6 / 7) r.cluster = 4;
    else if (solo_items * 2 <= sms * 6 / 7 && width > 3 * r.warps) r.cluster = 2;
  }
  const int64_t blocks = solo_items * r.cluster;
  // Of clusters the more granules a warp the more of the SMs they take, and fewer for several blocks of rows,
  // as the longest sequence can have and all have on average; a third less than equal lengths would bear, since
  // splitting alone evens out different ones (28 x 0-7758 tokens, 4/2 heads, D = 64, 2 blocks an item: 18.8 us, split
  // 15.4; 4 x 5027, 32/2 heads, D = 64, two blocks of rows: 15.0, split 12.9).
  const int64_t most_rows = d.rows.n_rows > seqs ? d.rows.n_rows - seqs + 1 : 1;
  const int64_t turns = ((most_rows * group + r.rows - 1) / r.rows) * ((per + r.rows - 1) / r.rows);
  const bool narrow = r.cluster > 1 ? (d.cache.d == 128 ? 20 : 28) * width * turns <= r.warps * r.cluster * blocks
                                    : width <= r.warps * (2 * blocks > sms ? 16 : 4);
  r.solo = blocks <= sms && narrow &&
           (d.rows.n_rows <= seqs || d.rows.n_rows * group <= 4 * r.rows);
  if (r.solo) {
    r.grid = blocks;
    r.ml_off = r.o_off = r.aside_off = r.bytes = 0;
    r.most = 0;
    return r;
  }
  // Two tiles of rows at once halve the copies and conversions, at 8 warps an SM and with half of the work in vain
  // for items that end in the first.  One against two tiles, 12 x 8192-16384 tokens, us: D = 128, 8 KV heads (302 MB,
  // more than the L2 cache keeps for the second block of rows), 16 rows 90 / 72, 24 rows 142 / 118, 32 rows 150 / 121;
  // 4 KV heads, 16 rows 50 / 50, 24 rows 68 / 68, to fp32 74 / 84, 32 rows 79 / 72; different numbers of rows, 8 to
  // 24 of 36 x 7334 tokens 33 / 35, 4 to 20 of 344 x 853 32 / 35; D = 64, 8 KV heads, 16 rows 47 / 52, 24 rows 64 / 73,
  // 32 rows 79 / 76, to fp32 88 / 97, 64 rows 146 / 132.
  const int64_t table = seqs * d.rows.max_pages, pages = table < d.cache.n_pages ? table : d.cache.n_pages;
  const bool cached = pages * d.cache.hkv * d.cache.page_size * d.cache.d * 2 <= 160000000;
  tiles(per <= (d.cache.d == 64 ? 32 : cached ? 24 : 8) ? 1 : 2);
  // numbers at most, in fp64: the page table's width times the heads may pass 64 bits
  r.most = (static_cast<double>(d.rows.max_pages) * d.cache.page_size * d.cache.d / 4096 + 1 + kSetup) * d.cache.hkv *
           static_cast<double>(seqs + d.rows.n_rows * group / r.rows);
  r.grid = r.most < sms ? static_cast<int64_t>(r.most) : sms;
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
  p.cluster = pl.cluster;
  return c.d == 128 ? run_d<128>(p, pl, mk, mv, items, num_sms, s) : run_d<64>(p, pl, mk, mv, items, num_sms, s);
}

}  // namespace cpattn

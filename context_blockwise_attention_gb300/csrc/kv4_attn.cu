// Attention over the paged 4-bit cache: the choice of the kernel variant, workspace and launch.
#include "kv4_attn.cuh"

namespace cpattn {

using namespace kvattn;

namespace kvattn {
extern template cp_status run4_d<64>(const Params&, const Plan&, int64_t, int, cudaStream_t);
extern template cp_status run4_d<128>(const Params&, const Plan&, int64_t, int, cudaStream_t);
}  // namespace kvattn

namespace {

Plan plan_of(const cp_kv4_attn_desc& d, int sms) {
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
  // Solo, by the page table's width in granules, which bounds the tokens, the one thing about them that is known here: as
  // many blocks an item as the SMs hold clusters of, where a block's warps have some granules each, as long as splitting,
  // which uses all SMs but has a second kernel, is slower.  Equal sequences, 1, 2, 4, 8 blocks an item / split, us:
  //   D = 128  4 x 8 items (sequences x KV heads) of 1000 tokens 8.7, 9.1, 8.3, - / 12.9; 4000: 20, 15, 11.5, - / 16; 8000:
  //            34, 22, 15.5, - / 19; 8 x 8 of 8000: 35, 25, -, - / 27; 16 x 8 of 4000: 23 / 28
  //            1 item of 1000 9.3, 9.4, 8.4, 8.8 / 9.0; 4000: 20, 15, 11.4, 10.6 / 9.7; 4 items of 8000: 33, 22, 16, 12.2 / 14.5
  //   D = 64   4 x 8 of 1000 6.8, 7.3, 7.3, - / 11.7; 8000: 20, 15, 10.9, - / 15; 8 x 8 of 8000: 20, 15, -, - / 17
  //            1 item of 2000 8.4, 8.3, 7.2, 7.4 / 8.3; 8000: 20, 15, 10.4, 9.1 / 8.8; 4 items of 8000: 20, 15, 10.5, 9.1 / 12.1
  // One row a sequence, as far as can be told from their numbers, or few rows in all, since the blocks take an item's
  // blocks of rows one after the other.  What it costs is short sequences under a wide table, which are split.
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
  const int64_t most_rows = d.rows.n_rows > seqs ? d.rows.n_rows - seqs + 1 : 1;
  const int64_t turns = ((most_rows * group + r.rows - 1) / r.rows) * ((per + r.rows - 1) / r.rows);
  const bool narrow = r.cluster > 1 ? 12 * width * turns <= r.warps * r.cluster * blocks
                                    : width <= r.warps * (2 * blocks > sms ? 16 : 4);
  r.solo = blocks <= sms && narrow &&
           (d.rows.n_rows <= seqs || d.rows.n_rows * group <= 4 * r.rows);
  if (r.solo) {
    r.grid = blocks;
    r.ml_off = r.o_off = r.aside_off = r.bytes = 0;
    r.most = 0;
    return r;
  }
  // Tiles of rows at once: two share the conversion of the keys, which costs more than a tile's products, but leave 8 warps
  // an SM instead of 12 at D = 128, and half of the work is in vain for items that end in the first.  Measured over
  // 16 x 2000-16000 tokens, 8 KV heads, bf16, one / two tiles (three), us:
  //   D = 128, equal rows  8: 45 / 55 (64); 12: 66 / 62 (70); 16: 67 / 63 (71); 24: 91 / 95 (80); 32: 116 / 99 (121);
  //            48: 168 / 143 (131); 64: 215 / 181 (182); 96: 315 / 260 (237)
  //            of 8-16 rows 54 / 61, of 8-24 64 / 69 (77), of 16-32 82 / 76, of 16-48 102 / 93 (98)
  //   D = 64,  equal rows  8: 32 / 36; 12: 43 / 39; 16: 44 / 39; 24: 58 / 56; 32: 72 / 59; of 8-16 36 / 37, of 8-24 42 / 41
  // So one tile up to 8 rows; three where that saves a third of the passes; and one again for mixed numbers of rows up
  // to 16 (12 at D = 64), as a total that the sequences do not divide shows, while the L2 cache hands the keys to the
  // second block of rows.
  const int64_t mean = (d.rows.n_rows * group + seqs - 1) / seqs;
  const bool mixed = d.rows.n_rows % seqs != 0;
  const int64_t table = seqs * d.rows.max_pages, pages = table < d.cache.n_pages ? table : d.cache.n_pages;
  const bool cached = pages * d.cache.hkv * d.cache.page_size * d.cache.d * 9 / 8 <= 160000000;
  if (mixed && cached && r.pp == 1) tiles(mean <= (d.cache.d == 64 ? 12 : 16) ? 1 : 2);
  else if (r.pp == 1 && d.cache.d == 128 && !mixed && 4 * ((mean + 23) / 24) < 3 * ((mean + 15) / 16)) tiles(3);
  else tiles(mean <= 8 ? 1 : 2);
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

int64_t kv4_attn_workspace(const cp_kv4_attn_desc& d, int num_sms) { return plan_of(d, num_sms).bytes; }

cp_status launch_kv4_attn(const cp_kv4_attn_desc& d, float scale, int64_t timeout_ns, int num_sms, cudaStream_t s) {
  const Plan pl = plan_of(d, num_sms);
  if (pl.most > 1e12) {  // their products with a worker's number stay int64
    set_error("cp_kv4_cache_attn: max_pages * page_size * hkv * n_seqs is too large for one call");
    return CP_ERR_INVALID_ARG;
  }
  const cp_kv4_cache& c = d.cache;
  uint8_t* const ws = static_cast<uint8_t*>(d.workspace);
  Params p{};
  p.tile[0] = static_cast<const uint8_t*>(c.k);
  p.tile[1] = static_cast<const uint8_t*>(c.v);
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
  p.setup = kSetup;
  p.few = 128 * items;
  p.cluster = pl.cluster;
  return c.d == 128 ? run4_d<128>(p, pl, items, num_sms, s) : run4_d<64>(p, pl, items, num_sms, s);
}

}  // namespace cpattn

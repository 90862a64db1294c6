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
  // Solo, by the page table's width in granules, which bounds the tokens, the one thing about them that is known here:
  // as many blocks an item as the SMs hold clusters of (12 to 15 of 8 blocks, 36 of 4), where a block's warps have some
  // granules each (32/8 heads, D = 128, tables as wide as the sequences: 1 x 1000 / 4000 tokens 9.3 / 21.3 us with one
  // block, 8.2 / 9.8 with 8; 4 x 4000 21.5, 11.7 with 4; 8 x 4000 21.6, 15.9 with 2; 1 x 500 7.2, 8.0 with 8), as long as
  // splitting is slower, which uses all SMs but has a second kernel: 1 x 4000 tokens 9.8 us against 12.4, 4 x 4000
  // 11.7 / 16.2, 4 x 8000 16.2 / 19.4, 8 x 4000 15.9 / 18.1, one KV head of 4000 9.4 / 9.0, of 8000 11.6 / 10.1; 18 x 8
  // items of 2048 / 6144 tokens, one block each, 13.8 / 40.1 against 21.1 / 47.5.  One row a sequence, as far as can be
  // told from their numbers, or few rows in all, since the blocks take an item's blocks of rows one after the other.
  // What it costs is short sequences under a wide table: 1 x 1000 tokens with a table for 8192 8.0 us, for 16384 and more
  // 11.3; 4 x 2000 9.3 and 14.1; 16 x 2000 with a table for 2000 14.3, for 8192 and more 19.4.
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
  // splitting alone evens out different ones (28 x 0-7758 tokens, 4/2 heads, D = 64, 2 blocks an item: 15.3 us, split
  // 14.1; 4 x 5027, 32/2 heads, D = 64, two blocks of rows: 18.3, split 13.8).
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
  // more than the L2 cache keeps for the second block of rows), 16 rows 90 / 73, 24 rows 143 / 120, 32 rows 151 / 123;
  // 4 KV heads, 16 rows 49 / 50, 24 rows 68 / 69, to fp32 74 / 84, 32 rows 80 / 72; D = 64, 8 KV heads, 16 rows
  // 48.5 / 48.6, 24 rows 65 / 70, 32 rows 82 / 73, to fp32 91 / 88, 64 rows 153 / 127; 30 x 239-719 tokens, 1-3 rows of
  // 128/32 heads, 36 / 51; 52 x 0-1534, 64/8, 24 / 31.
  // Where the rule is wrong: 16 rows whose keys are 150 MB and fit the L2 by this border (9 x 8567 tokens, 128/8, D = 128:
  // 54.7 / 48.8), 50 requests of some tokens with 1-4 rows of 128/16 heads (D = 64, to fp32 18.3 / 16.0), and calls of many
  // rows over very few tokens, which two tiles answer slowly (1 x 8 tokens, 11 rows of 128/16 heads, D = 64: 8.0 / 15.5;
  // 55 x 64-192, 1-15 rows of 64/8, D = 128: 36 / 49).
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
  p.setup = kSetup;
  p.few = 128 * items;
  p.cluster = pl.cluster;
  return c.d == 128 ? run_d<128>(p, pl, mk, mv, items, num_sms, s) : run_d<64>(p, pl, mk, mv, items, num_sms, s);
}

}  // namespace cpattn

"""The 8-bit cache, attention over it and rotary positions on the GPU against the float64 oracle.

Tolerances are per element and follow from the arithmetic:

* cache bytes, scales and read-back values are equal to the oracle's.
* rotation, fp32: the angle is off by at most 2e-7 (fraction of a turn to 24 bits), cos and sin by
  2^-23, two products and a sum by 2^-24 each: 5e-7 (|a| + |b|) in all; bf16 outputs add half a step.
* attention: a score is an fp32 sum of D products, off by at most 2^-20 of the sum of their
  magnitudes A (D / 16 accumulations of 2^-23 at D = 128, and 2^-21 for the softmax scale and the
  exponent's argument) plus 2^-22 |s|; weights have 22 bits for an fp32 output and 11 for a bf16
  one, ex2 2^-22; sums over n keys add n / 16 accumulations of 2^-23.  So with delta the largest
  score error of a row, |dO| <= (sum_j p_j |v_j|) (2 delta + w + n 2^-27 + 2^-20), w = 2^-21 or
  2^-11, plus half a step of the output type, and |dLSE| <= delta + n 2^-24 + 2^-22 |LSE| + 2^-20.
  Where the heavy tokens hold zeros in a column the light ones are all there is: a weight times its
  page's scale is held as f16, the largest at 2^15, and f16 has no step below 2^-24, so a weight is
  off by up to 2^-25 2^-15 = 2^-40 of the largest scale S of the sequence's pages besides: with
  values v_j = s_j w_j that adds 2^-40 S sum_j |w_j| to the sum of p_j v_j, where the largest p is 1.
"""

import numpy as np
import pytest
import torch

import helpers
import oracle
from oracle import cache as oc

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
from context_blockwise_attention_gb300 import PosMap, api  # noqa: E402

DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)


class Pool:
    """A cache and its host copy, with a page table that deals out pages in a random order."""

    def __init__(self, seqs, tokens, page, hkv, d, seed, spare=2, fill=0x7F):
        rng = np.random.default_rng(seed)
        used = [max(0, -(-int(t) // page)) for t in tokens]
        self.page, self.hkv, self.d = page, hkv, d
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        self.width = max(1, max(used) if used else 1)
        self.table = np.full((seqs, self.width), -1, dtype=np.int64)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        # every byte starts as NaN, every scale too: what nobody wrote must not show
        self.bytes = [np.full((self.n_pages, hkv, page, d), fill, np.uint8) for _ in range(2)]
        self.scale = [np.full((self.n_pages, hkv), np.nan, np.float32) for _ in range(2)]

    def fill(self, tokens, seed, spread=3.0):
        """Random tokens for each sequence, quantised by the oracle."""
        rng = np.random.default_rng(seed)
        for b, n in enumerate(tokens):
            for which in range(2):
                x = rng.standard_normal((int(n), self.hkv, self.d)) * 2.0 ** rng.uniform(-spread, spread, (int(n), self.hkv, 1))
                oc.cache_write(self.bytes[which], self.scale[which], x.astype(np.float32).astype(np.float64), [0, int(n)],
                               [0], self.table[b:b + 1])

    def device(self):
        f8 = [torch.from_numpy(b).to(DEV).view(torch.float8_e4m3fn) for b in self.bytes]
        return cpa.KvCache(f8[0], f8[1], *(torch.from_numpy(s).to(DEV) for s in self.scale))

    def tokens_of(self, b, n):
        pages = self.table[b][:-(-int(n) // self.page)]
        return [oc.cache_tokens(self.bytes[w], self.scale[w], pages, int(n)) for w in range(2)]


def _same_cache(cache, pool):
    for got, want in ((cache.k, pool.bytes[0]), (cache.v, pool.bytes[1])):
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    for got, want in ((cache.k_scale, pool.scale[0]), (cache.v_scale, pool.scale[1])):
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)


# ------------------------------------------------------------------ writing and reading
WRITES = [  # rows of each sequence, tokens before them, page, hkv, d, dtype
    ([1], [0], 16, 1, 64, BF16),
    ([1, 1, 1, 1], [15, 16, 17, 200], 16, 2, 128, BF16),
    ([0, 3, 0, 1], [5, 30, 0, 63], 32, 3, 64, F32),
    ([200, 0, 77, 64], [0, 9, 60, 64], 64, 2, 128, BF16),
    ([129, 500], [127, 1], 128, 2, 64, F32),
    ([33, 31, 16], [0, 1, 47], 16, 5, 128, F32),
    ([257], [255], 128, 1, 128, BF16),
    ([2] * 70, list(range(70)), 16, 2, 64, BF16),
    ([40], [8], 64, 1, 64, BF16),
    ([3] * 700, [i % 37 for i in range(700)], 16, 1, 64, BF16),
    ([20, 0, 0, 0, 9] * 30, [i % 50 for i in range(150)], 16, 3, 128, BF16),
]


@pytest.mark.parametrize("rows,held,page,hkv,d,dtype", WRITES)
def test_write_and_read_are_exact(rows, held, page, hkv, d, dtype):
    total = [a + b for a, b in zip(rows, held)]
    pool = Pool(len(rows), total, page, hkv, d, 1)
    pool.fill(held, 2)
    cache = pool.device()
    start = _starts(rows)
    extra = 5  # rows of no sequence
    gen = torch.Generator().manual_seed(3)
    # magnitudes from far below to far above what the continued pages hold
    x = [(torch.randn((int(start[-1]) + extra, hkv, d), generator=gen) *
          torch.exp2(torch.randint(-9, 9, (int(start[-1]) + extra, hkv, 1), generator=gen).float())).to(dtype)
         for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (_i32(start), _i32(held), _i32(pool.table))
    for again in range(2):  # writing the same tokens again changes nothing
        cpa.kv_cache_write(cache, x[0].to(DEV), x[1].to(DEV), *args, status=status)
        if again == 0:
            for w in range(2):
                oc.cache_write(pool.bytes[w], pool.scale[w], x[w].double().numpy(), start, held, pool.table)
        _same_cache(cache, pool)
    # read the new rows, and everything from the first token on, in both types
    for first, n in ((held, rows), ([0] * len(rows), total)):
        s = _starts(n)
        for out in (BF16, F32):
            k = torch.full((int(s[-1]) + 3, hkv, d), 7.0, dtype=out, device=DEV)
            v = torch.full_like(k, 7.0)
            cpa.kv_cache_read(cache, _i32(s), _i32(first), args[2], k.shape[0], k=k, v=v, status=status)
            for w, got in ((0, k), (1, v)):
                assert bool((got[int(s[-1]):] == 7.0).all())
                for b in range(len(rows)):
                    want = pool.tokens_of(b, first[b] + n[b])[w][first[b]:]
                    assert np.array_equal(got[int(s[b]):int(s[b + 1])].double().cpu().numpy(), want)
    assert status.item() == 0


@pytest.mark.parametrize("rows", [[3], [100]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_special_values(rows, dtype):
    pool = Pool(1, [120], 64, 2, 64, 5)
    pool.fill([10], 6)
    cache = pool.device()
    x = torch.randn((rows[0], 2, 64), generator=torch.Generator().manual_seed(7)).to(dtype)
    x[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0])
    x[1] = 0
    x[2, 1, 5] = torch.finfo(dtype).max / 4
    x[2, 1, 6] = 1e-39
    cpa.kv_cache_write(cache, x.to(DEV), x.to(DEV), _i32([0, rows[0]]), _i32([10]), _i32(pool.table))
    for w in range(2):
        oc.cache_write(pool.bytes[w], pool.scale[w], x.double().numpy(), [0, rows[0]], [10], pool.table)
    for got, want in ((cache.k, pool.bytes[0]), (cache.v, pool.bytes[1])):
        got = got.view(torch.uint8).cpu().numpy()
        nan = (want & 127) == 127  # a NaN's sign is free
        assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(cache.k_scale.cpu().numpy(), pool.scale[0], equal_nan=True)
    # a page of zeros takes the smallest scale
    z = torch.zeros((5, 2, 64), dtype=dtype, device=DEV)
    cpa.kv_cache_write(cache, z, z, _i32([0, 5]), _i32([64]), _i32(pool.table))
    assert cache.k_scale[int(pool.table[0, 1])].tolist() == [2.0 ** -64] * 2


def test_bad_pages_and_rows_are_skipped_and_reported():
    pool = Pool(3, [64, 64, 64], 16, 2, 64, 8)
    pool.fill([64, 64, 64], 9)
    cache = pool.device()
    bad = pool.table.copy()
    bad[0, 1], bad[1, 2] = -7, pool.n_pages
    start = [0, 64, 128, 192]
    x = torch.randn((192, 2, 64), generator=torch.Generator().manual_seed(1)).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k = torch.full((192, 2, 64), 12345.0, device=DEV)  # no cached value
    v = torch.full_like(k, 7.0)
    cpa.kv_cache_read(cache, _i32(start), _i32([0, 0, 0]), _i32(bad), 192, k=k, v=v, status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    skipped = [16 <= r < 32 or 64 + 32 <= r < 64 + 48 for r in range(192)]
    assert bool((k[torch.tensor(skipped)] == 12345.0).all()) and not bool((k[~torch.tensor(skipped)] == 12345.0).any())
    status.zero_()
    cpa.kv_cache_write(cache, x, x, _i32(start), _i32([0, 0, 0]), _i32(bad), status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    kept = pool.table[0, 1], pool.table[1, 2]
    for page in kept:
        assert np.array_equal(cache.k[int(page)].view(torch.uint8).cpu().numpy(), pool.bytes[0][page])
    for n in range(len(pool.table[2])):
        page = pool.table[2, n]
        assert not np.array_equal(cache.k[int(page)].view(torch.uint8).cpu().numpy(), pool.bytes[0][page])
    # behind the table, before the first token, rows out of order or out of range: nothing is written
    _clean = pool.device()
    for s, held in (([0, 64], [64]), ([0, 5], [-3]), ([64, 0], [0]), ([-100, -1], [0])):
        cpa.kv_cache_write(_clean, x, x, _i32(s), _i32(held), _i32(pool.table[:1]), status=status)
    _same_cache(_clean, pool)


# ------------------------------------------------------------------ attention
def _check_attn(pool, cache, q, rows, held, q_first, kv_pos, o_dtype, scale=0.0, wide=0):
    start = _starts(rows)
    n, hq, d = q.shape
    o = torch.full((n, hq, d), float("nan"), dtype=o_dtype, device=DEV)
    lse = torch.full((n, hq), float("nan"), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = pool.table if wide == 0 else np.concatenate([pool.table, np.full((len(rows), wide), -1)], 1)
    cpa.kv_cache_attn(q.to(DEV), cache, _i32(start), _i32(held), _i32(table),
                      q_first=None if q_first is None else _i32(q_first), kv_pos=kv_pos, scale=scale, o=o, lse=lse,
                      status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    got_o, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(got_o[int(start[-1]):]).all() and np.isnan(got_l[int(start[-1]):]).all()
    sc = scale or d ** -0.5
    qd = q.double().numpy()
    worst = 0.0
    for b in range(len(rows)):
        r0, r1, m = int(start[b]), int(start[b + 1]), int(held[b])
        if r1 == r0:
            continue
        k, v = pool.tokens_of(b, m)
        kpos = kv_pos.base + kv_pos.stride * np.arange(m)
        qpos = np.arange(r1 - r0) + (q_first[b] if q_first is not None else 0)
        seen = kpos[None, :] <= qpos[:, None] if q_first is not None else np.ones((r1 - r0, m), bool)
        group = hq // pool.hkv
        scales = pool.scale[1][pool.table[b][:-(-m // pool.page)]].astype(np.float64)  # [pages, hkv]
        of_token = np.repeat(scales, pool.page, 0)[:m]
        for h in range(hq):
            kh, vh = k[:, h // group], v[:, h // group]
            light = 2.0 ** -40 * scales[:, h // group].max() * np.abs(vh) / of_token[:, h // group, None] if m else 0.0
            for i in range(r1 - r0):
                idx = np.nonzero(seen[i])[0]
                go, gl = got_o[r0 + i, h], got_l[r0 + i, h]
                if idx.size == 0:
                    assert np.all(go == 0.0) and gl == -np.inf
                    continue
                s = sc * (kh[idx] @ qd[r0 + i, h])
                a = sc * (np.abs(kh[idx]) @ np.abs(qd[r0 + i, h]))
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                ref, ref_l = (p @ vh[idx]) / z, top + np.log(z)
                delta = float((2.0 ** -20 * a + 2.0 ** -22 * np.abs(s)).max())
                w = 2.0 ** -11 if o_dtype == BF16 else 2.0 ** -21
                tol = (p @ np.abs(vh[idx])) / z * (2 * delta + w + idx.size * 2.0 ** -27 + 2.0 ** -20)
                tol = tol + light[idx].sum(0) / z + np.abs(ref) * (2.0 ** -8 if o_dtype == BF16 else 2.0 ** -24) * 1.01 + 1e-30
                err = np.abs(go - ref)
                assert np.all(err <= tol), (b, i, h, float((err / tol).max()), float(err.max()))
                tol_l = delta + idx.size * 2.0 ** -24 + 2.0 ** -22 * abs(ref_l) + 2.0 ** -20
                assert abs(gl - ref_l) <= tol_l, (b, i, h, gl, ref_l)
                worst = max(worst, float((err / tol).max()), abs(gl - ref_l) / tol_l)
    return o, lse, worst


ATTN = [  # rows, held, page, hq, hkv, d, in, out, stride of the shard or None (not causal)
    ([1], [1], 16, 1, 1, 64, BF16, F32, 1),
    ([1], [1], 128, 8, 8, 128, F32, BF16, None),
    ([1, 1, 1], [0, 33, 31], 16, 8, 1, 128, BF16, BF16, None),
    ([1], [1000], 64, 32, 8, 128, BF16, BF16, 1),
    ([1] * 9, [1, 15, 16, 17, 32, 64, 65, 500, 129], 16, 8, 2, 64, BF16, F32, 1),
    ([1] * 9, [1, 15, 16, 17, 32, 64, 65, 500, 129], 32, 8, 2, 128, F32, F32, 1),
    ([2, 0, 5, 1], [300, 40, 5, 7], 64, 8, 2, 128, BF16, F32, 1),
    ([4, 8, 3], [4, 513, 260], 128, 16, 2, 64, BF16, BF16, 1),
    ([17, 1], [300, 3], 32, 10, 2, 128, BF16, BF16, 1),
    ([7, 33], [100, 90], 16, 12, 1, 64, F32, F32, 1),
    ([3, 40], [1200, 64], 64, 16, 1, 128, BF16, F32, 1),
    ([3, 40], [1200, 64], 64, 16, 1, 128, BF16, BF16, 1),
    ([5, 9], [700, 1100], 128, 32, 2, 64, F32, BF16, 1),
    ([2, 3], [90, 1000], 64, 4, 4, 128, BF16, F32, 8),
    ([6, 2], [31, 640], 32, 8, 1, 64, BF16, BF16, 3),
    ([1, 1], [5000, 4097], 128, 4, 2, 64, BF16, F32, 1),
    ([2, 1], [2500, 3333], 16, 5, 1, 128, F32, F32, None),
]


# a table as wide as the longest sequence needs, and much wider ones: short rows take one block a sequence and
# head by the first, a cluster of blocks by some, and are split by the widest
@pytest.mark.parametrize("wide", [0, 600, 2500])
@pytest.mark.parametrize("rows,held,page,hq,hkv,d,din,dout,stride", ATTN)
def test_attention(rows, held, page, hq, hkv, d, din, dout, stride, wide):
    pool = Pool(len(rows), held, page, hkv, d, 11)
    pool.fill(held, 12)
    q = (torch.randn((sum(rows) + 2, hq, d), generator=torch.Generator().manual_seed(13)) *
         torch.exp2(torch.randint(-3, 2, (sum(rows) + 2, hq, 1), generator=torch.Generator().manual_seed(14)).float())).to(din)
    base = 0 if stride is None else stride - 1
    first = None
    if stride is not None:  # the last row sees everything
        first = [base + stride * (m - 1) - (n - 1) for n, m in zip(rows, held)]
    _check_attn(pool, pool.device(), q, rows, held, first, PosMap(base, stride or 1), dout, wide=wide)


@pytest.mark.parametrize("wide", [0, 600, 2500])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_attention_rows_that_see_little_or_nothing(dout, wide):
    rows, held = [6, 3, 2, 4], [50, 200, 0, 31]
    pool = Pool(4, held, 16, 2, 64, 21)
    pool.fill(held, 22)
    q = torch.randn((15, 8, 64), generator=torch.Generator().manual_seed(23)).to(BF16)
    # a shard at positions 5, 9, 13, ...: the first rows stand before it, a later one in its middle
    _check_attn(pool, pool.device(), q, rows, held, [2, 300, 7, -100], PosMap(5, 4), dout, wide=wide)
    _check_attn(pool, pool.device(), q, rows, held, [2, 300, 7, -100], PosMap(0, 1), dout, scale=0.7, wide=wide)


@pytest.mark.parametrize("g,d,page", [(1, 64, 32), (8, 64, 16), (16, 64, 128), (3, 128, 32), (16, 128, 16)])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_attention_ignores_nan_and_infinity_behind_a_row(g, d, page, dout):
    """Tokens that some rows see and others do not hold NaN values (and keys): the rows before them
    are as if they were not there, the others are NaN in those columns."""
    held, rows = [70], [4]
    pool = Pool(1, held, page, 1, d, 31)
    pool.fill(held, 32)
    q = torch.randn((4, g, d), generator=torch.Generator().manual_seed(33)).to(BF16)
    last, slot = pool.table[0, 69 // page], 69 % page  # the last token: row 3 alone sees it
    pool.bytes[1][last, 0, slot, :7] = 0x7F
    pool.bytes[1][last, 0, slot, 9] = 0xFF
    cache = pool.device()
    start, first = _i32([0, 4]), _i32([66])
    o, lse = cpa.kv_cache_attn(q.to(DEV), cache, start, _i32(held), _i32(pool.table), q_first=first, o_dtype=dout)
    clean = Pool(1, held, page, 1, d, 31)
    clean.fill(held, 32)
    o2, l2 = cpa.kv_cache_attn(q.to(DEV), clean.device(), start, _i32(held), _i32(pool.table), q_first=first, o_dtype=dout)
    assert torch.equal(o[:3], o2[:3]) and torch.equal(lse, l2)
    nan = torch.zeros(d, dtype=torch.bool, device=DEV)
    nan[:7] = True
    nan[9] = True
    assert bool(o[3][:, nan].isnan().all()) and torch.equal(o[3][:, ~nan], o2[3][:, ~nan])
    # a NaN key: the scores of the rows that see it are NaN
    pool.bytes[0][last, 0, slot, 3] = 0x7F
    o, lse = cpa.kv_cache_attn(q.to(DEV), pool.device(), start, _i32(held), _i32(pool.table), q_first=first, o_dtype=dout)
    assert torch.equal(o[:3], o2[:3]) and torch.equal(lse[:3], l2[:3])
    assert bool(o[3].isnan().all()) and bool(lse[3].isnan().all())
    # an infinite query spoils its own row alone
    q[1, 0, 5] = float("inf")
    o, lse = cpa.kv_cache_attn(q.to(DEV), clean.device(), start, _i32(held), _i32(pool.table), q_first=first, o_dtype=dout)
    keep = torch.ones((4, g), dtype=torch.bool, device=DEV)
    keep[1, 0] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], l2[keep])
    assert bool(o[1, 0].isnan().all())


@pytest.mark.parametrize("wide", [0, 600, 2500])
@pytest.mark.parametrize("d,page", [(64, 32), (128, 16)])
@pytest.mark.parametrize("which,value", [(0, float("nan")), (0, float("inf")), (1, float("nan")), (1, float("inf"))])
def test_attention_scale_that_is_not_finite_reaches_the_rows_that_see_its_page(which, value, d, page, wide):
    held, rows, g = [page * 5], [3], 6
    pool = Pool(1, held, page, 1, d, 34)
    pool.fill(held, 35)
    last = pool.table[0, 4]
    pool.scale[1][last] = 2.0 ** -20  # not the largest: weights are held relative to the largest of a tile
    q = torch.randn((3, g, d), generator=torch.Generator().manual_seed(36)).to(BF16).to(DEV)
    table = _i32(np.concatenate([pool.table, np.full((1, wide), -1)], 1))
    args = (_i32([0, 3]), _i32(held), table)
    first = _i32([4 * page - 2])  # the last row alone sees the last page, one token of it
    clean = cpa.kv_cache_attn(q, pool.device(), *args, q_first=first, o_dtype=F32)
    pool.scale[which][last] = value
    o, lse = cpa.kv_cache_attn(q, pool.device(), *args, q_first=first, o_dtype=F32)
    assert torch.equal(o[:2], clean[0][:2]) and torch.equal(lse[:2], clean[1][:2])
    assert bool(clean[0].isfinite().all())
    spoilt = torch.ones(g, dtype=torch.bool, device=DEV)
    if which == 0 and value == float("inf"):  # a score of -inf is a weight of zero: the sign of q . k decides
        k8 = torch.from_numpy(pool.bytes[0][last, 0, 0]).view(torch.float8_e4m3fn).double().to(DEV)
        spoilt = q[2].double() @ k8 > 0
        assert 0 < int(spoilt.sum()) < g
    assert not bool(o[2][spoilt].isfinite().any()) and bool(o[2][~spoilt].isfinite().all())


@pytest.mark.parametrize("dout", [BF16, F32])
def test_attention_scales_far_apart(dout):
    """Value pages whose scales differ by 2^40, and keys that make one token far heavier than the rest."""
    held = [160]
    pool = Pool(1, held, 16, 1, 128, 41)
    rng = np.random.default_rng(42)
    for which in range(2):
        x = rng.standard_normal((160, 1, 128))
        if which:
            x *= 2.0 ** np.repeat([0, -40, 20, -20, 0, 5, -5, 30, -30, 1], 16)[:, None, None]
        else:
            x[3] *= 30
            x[77] *= 40
        oc.cache_write(pool.bytes[which], pool.scale[which], x, [0, 160], [0], pool.table)
    q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(43)).to(BF16)
    _check_attn(pool, pool.device(), q, [2], held, [158], PosMap(0, 1), dout)


@pytest.mark.parametrize("d,page,dout", [(128, 128, F32), (128, 64, BF16), (64, 128, F32)])
def test_attention_very_long_rows(d, page, dout):
    """Millions of cached tokens, the same pages over and over: the softmax of the repeated keys is that
    of the keys, and LSE grows by ln(repeats).  The sums are put aside on the way: at most A truncated
    accumulations of 2^-23 to a sum (64 granules of 4 for bf16 outputs, 64 or 32 in all for fp32 ones), whatever
    the length; 2^-19 for the fp32 sums of the parts."""
    once, repeats = 1024, 4096
    pool = Pool(1, [once], page, 2, d, 45)
    pool.fill([once], 46, spread=1.0)
    q = torch.randn((2, 6, d), generator=torch.Generator().manual_seed(47)).to(BF16)
    table = np.tile(pool.table, (1, repeats))
    o, lse = cpa.kv_cache_attn(q.to(DEV), pool.device(), _i32([0, 2]), _i32([once * repeats]), _i32(table), o_dtype=dout)
    k, v = pool.tokens_of(0, once)
    acc = 256 if dout == BF16 else 64
    for i in range(2):
        for h in range(6):
            kh, vh, x = k[:, h // 3], v[:, h // 3], q[i, h].double().numpy()
            s = kh @ x * d ** -0.5
            p = np.exp(s - s.max())
            z = p.sum()
            delta = float((2.0 ** -20 * (np.abs(kh) @ np.abs(x)) * d ** -0.5 + 2.0 ** -22 * np.abs(s)).max())
            ref = p @ vh / z
            w = 2.0 ** -11 if dout == BF16 else 2.0 ** -21
            tol = p @ np.abs(vh) / z * (2 * delta + w + acc * 2.0 ** -23 + 2.0 ** -19)
            tol = tol + np.abs(ref) * (2.0 ** -8 if dout == BF16 else 2.0 ** -24) * 1.01
            assert np.all(np.abs(o[i, h].double().cpu().numpy() - ref) <= tol)
            ref_l = s.max() + np.log(z) + np.log(repeats)
            assert abs(float(lse[i, h]) - ref_l) <= delta + 2.0 ** -19 + 2.0 ** -22 * abs(ref_l)


def test_attention_many_sequences():
    n = cpa.KV_MAX_SEQS
    held = [(7 * i) % 41 for i in range(n)]
    rows = [1 if i % 5 else 0 for i in range(n)]
    pool = Pool(n, held, 16, 1, 64, 48)
    pool.fill(held, 49)
    q = torch.randn((sum(rows) + 1, 2, 64), generator=torch.Generator().manual_seed(50)).to(BF16)
    first = [m - 1 - (i % 3) for i, m in enumerate(held)]
    _check_attn(pool, pool.device(), q, rows, held, first, PosMap(0, 1), F32)


@pytest.mark.parametrize("held,page,hq,hkv,d,n,dout", [
    (50000, 128, 5, 1, 128, 1, BF16), (50000, 128, 8, 2, 64, 2, F32), (4100, 16, 4, 1, 128, 3, F32),
    (9000, 32, 24, 3, 64, 1, BF16)])
def test_attention_one_long_sequence(held, page, hq, hkv, d, n, dout):
    """Hundreds of partials to a row."""
    pool = Pool(1, [held], page, hkv, d, 81)
    pool.fill([held], 82)
    q = torch.randn((n, hq, d), generator=torch.Generator().manual_seed(83)).to(BF16)
    _check_attn(pool, pool.device(), q, [n], [held], [held - n], PosMap(0, 1), dout)


@pytest.mark.parametrize("rows,held,page,hq,hkv,d,din,dout", [
    ([1], [1200], 32, 4, 1, 128, BF16, BF16),
    ([1, 1], [4000, 3], 64, 8, 2, 64, BF16, F32),
    ([5, 1], [1500, 900], 16, 20, 5, 128, BF16, F32),       # an item of several blocks of rows
    ([1, 0, 1], [2100, 50, 0], 128, 32, 8, 128, F32, F32),  # 24 items: four blocks each
    ([1] * 7, [1100, 0, 900, 2000, 1, 33, 1500], 16, 16, 8, 128, BF16, BF16),  # 56 items: two
    ([2, 1], [1700, 2300], 32, 8, 4, 64, F32, BF16),
    ([1], [1700], 16, 80, 5, 64, F32, F32)])
def test_attention_clusters(rows, held, page, hq, hkv, d, din, dout):
    """Few rows over caches that are too long for one block an item and too short for a second kernel."""
    pool = Pool(len(rows), held, page, hkv, d, 87)
    pool.fill(held, 88)
    q = torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(89)).to(din)
    first = [m - n for n, m in zip(rows, held)]
    assert cpa.kv_cache_attn_workspace(pool.device(), sum(rows), hq, len(rows), pool.table.shape[1], din, dout) == 0
    _check_attn(pool, pool.device(), q, rows, held, first, PosMap(0, 1), dout)
    _check_attn(pool, pool.device(), q, rows, held, [f // 2 for f in first], PosMap(1, 2), dout)


@pytest.mark.parametrize("d,page,dout", [(64, 16, BF16), (128, 32, F32)])
def test_attention_many_short_items(d, page, dout):
    """More rows and heads than the second kernel has warps, most of them finished by one worker."""
    held = [(13 * i) % 90 for i in range(60)]
    rows = [1 + i % 5 for i in range(60)]
    pool = Pool(60, held, page, 8, d, 84)
    pool.fill(held, 85)
    q = torch.randn((sum(rows), 32, d), generator=torch.Generator().manual_seed(86)).to(BF16)
    first = [m - 1 - (i % 3) for i, m in enumerate(held)]
    _check_attn(pool, pool.device(), q, rows, held, first, PosMap(0, 1), dout)


def test_attention_bad_pages_answer_nan_and_report():
    held, rows = [100, 100, 100], [2, 2, 2]
    pool = Pool(3, held, 16, 2, 64, 51)
    pool.fill(held, 52)
    bad = pool.table.copy()
    bad[0, 4], bad[1, 0] = pool.n_pages + 3, -1
    q = torch.randn((6, 4, 64), generator=torch.Generator().manual_seed(53)).to(BF16).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (pool.device(), _i32([0, 2, 4, 6]))
    good, lgood = cpa.kv_cache_attn(q, *args, _i32(held), _i32(pool.table))
    o, lse = cpa.kv_cache_attn(q, *args, _i32(held), _i32(bad), status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    assert bool(o[:4].isnan().all()) and bool(lse[:4].isnan().all())
    assert torch.equal(o[4:], good[4:]) and torch.equal(lse[4:], lgood[4:])
    # causal rows that do not reach the bad page are right
    status.zero_()
    o, lse = cpa.kv_cache_attn(q, *args, _i32(held), _i32(bad), q_first=_i32([62, 98, 98]), status=status)
    ref, lref = cpa.kv_cache_attn(q, *args, _i32(held), _i32(pool.table), q_first=_i32([62, 98, 98]))
    assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1]) and bool(o[2:4].isnan().all())
    # nor those that only share a tile with it: page 5 is bad, positions 71 and 72 end in page 4
    bad[0, 4], bad[0, 5] = pool.table[0, 4], -1
    o, lse = cpa.kv_cache_attn(q, *args, _i32(held), _i32(bad), q_first=_i32([71, 98, 98]))
    ref, lref = cpa.kv_cache_attn(q, *args, _i32(held), _i32(pool.table), q_first=_i32([71, 98, 98]))
    assert torch.equal(o[:2], ref[:2]) and torch.equal(lse[:2], lref[:2])
    o, lse = cpa.kv_cache_attn(q, *args, _i32(held), _i32(bad), q_first=_i32([79, 98, 98]))
    assert bool(o[0].isfinite().all()) and bool(o[1].isnan().all())
    # more tokens than the table has pages for
    status.zero_()
    o, lse = cpa.kv_cache_attn(q, *args, _i32([100, 2 ** 31 - 1, 100]), _i32(pool.table), status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    assert torch.equal(o[:2], good[:2]) and bool(o[2:4].isnan().all()) and torch.equal(o[4:], good[4:])
    # a negative count is an empty cache
    o, lse = cpa.kv_cache_attn(q, *args, _i32([100, -5, 100]), _i32(pool.table))
    assert bool((o[2:4] == 0).all()) and bool((lse[2:4] == -float("inf")).all()) and torch.equal(o[4:], good[4:])


def test_attention_offsets_beyond_32_bits():
    """Pages whose bytes begin beyond 2^32, in a pool of more than 4 GiB for K and for V."""
    page, hkv, d = 128, 4, 128
    n_pages = (5 << 30) // (page * hkv * d)
    k = torch.zeros((n_pages, hkv, page, d), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    ks = torch.ones((n_pages, hkv), device=DEV)
    vs = torch.ones((n_pages, hkv), device=DEV)
    pool = Pool(1, [500], page, hkv, d, 61, spare=0)
    pool.fill([500], 62)
    far = [n_pages - 1, n_pages - 77, 3, n_pages // 2 + 1]
    for i, p in enumerate(pool.table[0]):
        for dst, src in ((k, pool.bytes[0]), (v, pool.bytes[1])):
            dst[far[i]] = torch.from_numpy(src[p]).to(DEV)
        for dst, src in ((ks, pool.scale[0]), (vs, pool.scale[1])):
            dst[far[i]] = torch.from_numpy(src[p]).to(DEV)
    cache = cpa.KvCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs)
    q = torch.randn((3, 8, d), generator=torch.Generator().manual_seed(63)).to(BF16).to(DEV)
    o, lse = cpa.kv_cache_attn(q, cache, _i32([0, 3]), _i32([500]), _i32([far]))
    want, lwant = cpa.kv_cache_attn(q, pool.device(), _i32([0, 3]), _i32([500]), _i32(pool.table))
    assert torch.equal(o, want) and torch.equal(lse, lwant)
    kk, vv = cpa.kv_cache_read(cache, _i32([0, 500]), _i32([0]), _i32([far]), 500, dtype=F32)
    cpa.kv_cache_write(cache, kk * 3, vv * 3, _i32([0, 500]), _i32([0]), _i32([far]))
    k3, _ = cpa.kv_cache_read(cache, _i32([0, 500]), _i32([0]), _i32([far]), 500, dtype=F32)
    assert bool(((k3 - 3 * kk).abs() <= 3 * kk.abs() * 2.0 ** -4 + 1e-3).all())


def _serving_case(seed, rows, held, page=32, hq=8, hkv=2, d=64):
    pool = Pool(len(rows), held, page, hkv, d, seed)
    pool.fill(held, seed + 1)
    q = torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(seed + 2)).to(BF16).to(DEV)
    return pool, pool.device(), q, _i32(_starts(rows)), _i32(held), _i32(pool.table)


@pytest.mark.parametrize("wide", [0, 60, 3000])  # one block an item, a cluster, split
def test_attention_same_bits_on_streams_at_once_and_in_graphs(wide):
    def widened(*case):
        return (*case[:5], torch.cat([case[5], case[5].new_full((case[5].shape[0], wide), -1)], 1))

    cases = [widened(*_serving_case(70, [1, 2, 1], [900, 40, 333])),
             widened(*_serving_case(80, [4], [2000], page=128, hq=16, d=128))]
    alone = [cpa.kv_cache_attn(q, c, s, h, t) for _, c, q, s, h, t in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):  # both at once; one by the stream argument, one by the current stream
        (_, c, q, s, h, t) = cases[0]
        r0 = cpa.kv_cache_attn(q, c, s, h, t, stream=streams[0])
        (_, c, q, s, h, t) = cases[1]
        with torch.cuda.stream(streams[1]):
            r1 = cpa.kv_cache_attn(q, c, s, h, t)
        raw = cpa.kv_cache_attn(q, c, s, h, t, stream=streams[1].cuda_stream)
        torch.cuda.synchronize()
        for got, want in ((r0, alone[0]), (r1, alone[1]), (raw, alone[1])):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a captured step replayed with other lengths, positions and pages
    pool, cache, q, s, h, t = widened(*_serving_case(90, [1, 1, 1], [700, 64, 257], page=16))
    h0, s0 = h.clone(), s.clone()
    first = _i32([699, 63, 256])
    o = torch.empty((3, 8, 64), device=DEV)
    lse = torch.empty((3, 8), device=DEV)
    ws = torch.empty(cpa.kv_cache_attn_workspace(cache, 3, 8, 3, t.shape[1]), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        cpa.kv_cache_attn(q, cache, s, h, t, q_first=first, o=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cpa.kv_cache_attn(q, cache, s, h, t, q_first=first, o=o, lse=lse, workspace=ws)
    for lens, starts in (([700, 64, 257], [0, 1, 2, 3]), ([1, 60, 0], [0, 0, 2, 3]), ([650, 3, 256], [0, 3, 3, 3])):
        h.copy_(_i32(lens))
        s.copy_(_i32(starts))
        first.copy_(_i32([max(0, x - 1) for x in lens]))
        ws.fill_(0xFF)
        g.replay()
        want = cpa.kv_cache_attn(q, cache, s, h, t, q_first=first)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    h.copy_(h0)
    s.copy_(s0)


@pytest.mark.parametrize("wide", [0, 500, 2500])
def test_rows_before_the_first_and_behind_the_last_sequence(wide):
    """row_start may begin behind row 0: the rows before it belong to nobody, in all three calls."""
    rows, held, total = [2, 0, 1], [40, 9, 100], [42, 9, 101]
    pool = Pool(3, total, 16, 2, 64, 105)
    pool.fill(total, 106)
    cache = pool.device()
    table = torch.cat([_i32(pool.table), torch.full((3, wide), -1, dtype=torch.int32, device=DEV)], 1)
    start = _i32([3, 5, 5, 6])
    q = torch.randn((8, 8, 64), generator=torch.Generator().manual_seed(107)).to(BF16).to(DEV)
    o = torch.full((8, 8, 64), 12345.0, device=DEV)
    lse = torch.full((8, 8), 12345.0, device=DEV)
    cpa.kv_cache_attn(q, cache, start, _i32(total), table, q_first=_i32(held), o=o, lse=lse)
    want = cpa.kv_cache_attn(q.roll(-3, 0), cache, start - 3, _i32(total), table, q_first=_i32(held))  # the same shapes
    assert torch.equal(o[3:6], want[0][:3]) and torch.equal(lse[3:6], want[1][:3])
    for x in (o, lse):
        assert bool((x[:3] == 12345.0).all()) and bool((x[6:] == 12345.0).all())
    k = torch.full((8, 2, 64), 12345.0, device=DEV)
    v = torch.full_like(k, 12345.0)
    cpa.kv_cache_read(cache, start, _i32(held), table, 8, k=k, v=v)
    for x in (k, v):
        assert bool((x[:3] == 12345.0).all()) and bool((x[6:] == 12345.0).all())
    cpa.kv_cache_write(cache, k, v, start, _i32(held), table)  # what was read goes back to its place
    for got, was in ((cache.k, pool.bytes[0]), (cache.v, pool.bytes[1])):
        now = oc.e4m3_decode(got.view(torch.uint8).cpu().numpy())
        assert np.array_equal(np.isnan(now), np.isnan(oc.e4m3_decode(was)))
    k2, v2 = cpa.kv_cache_read(cache, start - 3, _i32(held), table, 3, dtype=F32)
    assert torch.equal(k2, k[3:6]) and torch.equal(v2, v[3:6])


def test_a_decoding_step_in_a_graph():
    """Rotation, write and attention captured as one step and replayed for the next tokens."""
    seqs, hq, hkv, d, page = 3, 4, 2, 64, 16
    held = [15, 32, 40]
    pool = Pool(seqs, [64] * seqs, page, hkv, d, 101)
    pool.fill(held, 102)
    eager, graphed = pool.device(), pool.device()
    gen = torch.Generator().manual_seed(103)
    freq = tuple(100.0 ** (-i / 32) for i in range(32))
    table, start = _i32(pool.table), _i32(range(seqs + 1))
    q, k, v = (torch.empty((seqs, h, d), dtype=BF16, device=DEV) for h in (hq, hkv, hkv))
    n, pos = _i32(held), _i32(held)
    after = n + 1

    def step(cache, out=None):
        qr, kr = cpa.rope_axes([q, k], pos, freq)
        cpa.kv_cache_write(cache, kr, v, start, n, table)
        return cpa.kv_cache_attn(qr, cache, start, after, table, q_first=pos, o_dtype=BF16)

    def load(i):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).to(BF16) * 2.0 ** (i % 4))
        for t in (n, pos):
            t.copy_(_i32([h + i for h in held]))
        after.copy_(n + 1)
    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(graphed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = step(graphed)
    for i in range(20):
        load(i)
        want = step(eager)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        for a, b in zip(eager, graphed):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# a table of few pages: one block a sequence and head; of more: a cluster of blocks; of many: split
@pytest.mark.parametrize("width", [13, 100, 400, 2500])
def test_attention_wait_runs_out(width):
    pool, cache, q, s, h, t = _serving_case(95, [1, 1], [400, 300])
    t = torch.cat([t, t.new_full((2, width - t.shape[1]), -1)], 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cpa.kv_cache_attn(q, cache, s, h, t, status=status, flags=api.CP_FLAG_TEST_STALL, wait_timeout_ms=20)
    torch.cuda.synchronize()
    assert status.item() & 0xFF == api.CP_ERR_TIMEOUT
    want = _check_attn(pool, cache, q.cpu(), [1, 1], [400, 300], None, PosMap(0, 1), F32)
    assert want[0].isfinite().all()


def test_workspace_is_checked():
    pool, cache, q, s, h, t = _serving_case(97, [1, 1], [4000, 300])
    t = torch.cat([t, t.new_full((2, 400), -1)], 1)
    need = cpa.kv_cache_attn_workspace(cache, 2, 8, 2, t.shape[1])
    assert need > 0
    with pytest.raises(cpa.CpError):
        cpa.kv_cache_attn(q, cache, s, h, t, workspace=torch.empty(need - 16, dtype=torch.uint8, device=DEV))
    with pytest.raises(cpa.CpError):
        cpa.kv_cache_attn(q, cache, s, h, t, workspace=torch.empty(need + 16, dtype=torch.uint8, device=DEV)[8:])


def test_calls_refuse_wrong_tensors():
    pool, cache, q, s, h, t = _serving_case(99, [1, 1], [40, 30])
    x = torch.zeros((2, 2, 64), dtype=BF16, device=DEV)
    for call in (
            lambda: cpa.kv_cache_attn(q.double(), cache, s, h, t),
            lambda: cpa.kv_cache_attn(q.transpose(0, 1), cache, s, h, t),
            lambda: cpa.kv_cache_attn(q[:, :, :32].contiguous(), cache, s, h, t),
            lambda: cpa.kv_cache_attn(q[:, :3].contiguous(), cache, s, h, t),
            lambda: cpa.kv_cache_attn(q, cache, s.long(), h, t),
            lambda: cpa.kv_cache_attn(q, cache, s, h[:1], t),
            lambda: cpa.kv_cache_attn(q, cache, s, h, t, q_first=h[:1]),
            lambda: cpa.kv_cache_attn(q, cache, s, h, t, o=torch.empty((2, 8, 32), device=DEV)),
            lambda: cpa.kv_cache_attn(q, cache._replace(k=cache.k.view(torch.uint8)), s, h, t),
            lambda: cpa.kv_cache_attn(q, cache._replace(v_scale=cache.v_scale[1:]), s, h, t),
            lambda: cpa.kv_cache_write(cache, x[:, :1].contiguous(), x, s, h, t),
            lambda: cpa.kv_cache_write(cache, x, x.float(), s, h, t),
            lambda: cpa.kv_cache_read(cache, s, h, t, 2, dtype=torch.float16),
            lambda: cpa.kv_cache_read(cache, s, h, t, 2, k=x[:1], v=x[:1]),
            lambda: cpa.rope_axes([x], h, (1.0,) * 16, (9, 9)),
            lambda: cpa.rope_axes([x], h[:1], (1.0,) * 16),
            lambda: cpa.rope_axes([x, x.float()], h, (1.0,) * 16),
            lambda: cpa.rope_axes([x], h, (1.0,) * 16, out=[x.float()]),
            lambda: cpa.rope_axes([x], h, (1.0,) * 12),
    ):
        with pytest.raises(cpa.CpError):
            call()


# ------------------------------------------------------------------ rotary positions
ROPE = [  # tokens, heads, d, rot, sections, interleaved, dtype, largest position
    (1, (1,), 64, 64, (32,), False, BF16, 10),
    (7, (4, 2), 64, 64, (32,), True, F32, 1 << 30),
    (33, (32, 8), 128, 128, (16, 24, 24), False, BF16, 5000),
    (5, (3, 1, 1, 2), 128, 64, (8, 12, 12), True, BF16, 300),
    (129, (5,), 64, 16, (2, 2, 2, 2), False, F32, 70000),
    (64, (64, 8), 64, 32, (0, 16), False, F32, 1 << 20),
    (3, (2,), 256, 256, (128,), False, F32, 100),
    (9, (1, 1), 24, 16, (8,), True, F32, (1 << 31) - 2),
    (2, (130,), 40, 32, (5, 11), False, BF16, 999),
    (2000, (2, 1), 128, 96, (16, 16, 16), False, BF16, 1 << 18),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("tokens,heads,d,rot,sections,interleaved,dtype,far", ROPE)
def test_rope(tokens, heads, d, rot, sections, interleaved, dtype, far, inverse):
    gen = torch.Generator().manual_seed(5)
    xs = [torch.randn((tokens, h, d), generator=gen).to(dtype) for h in heads]
    pos = torch.randint(-far, far + 1, (len(sections), tokens), generator=gen)
    pos[:, -1] = far
    freq = [1.3 * 10000.0 ** (-2 * i / rot) * (-1 if i % 5 == 4 else 1) for i in range(rot // 2)]
    dev = [x.to(DEV) for x in xs]
    ys = cpa.rope_axes(dev, pos.int().to(DEV), freq, sections, interleaved, inverse)
    for x, y in zip(xs, ys):
        ref = oc.rotate(x.double().numpy(), pos.numpy(), freq, sections, interleaved, inverse)
        a = np.abs(x.double().numpy())
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        tol = np.zeros_like(a)
        tol[..., lo] = tol[..., hi] = 5e-7 * (a[..., lo] + a[..., hi])
        if dtype == BF16:
            tol[..., :rot] += 2.0 ** -8 * 1.01 * np.abs(ref[..., :rot])
        got = y.double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) - tol).max())
        assert np.array_equal(got[..., rot:], x.double().numpy()[..., rot:])
    # in place gives the same bits, and the other direction leads back
    same = [x.clone() for x in dev]
    cpa.rope_axes(same, pos.int().to(DEV), freq, sections, interleaved, inverse, out=same)
    assert all(torch.equal(a, b) for a, b in zip(same, ys))
    back = cpa.rope_axes(ys, pos.int().to(DEV), freq, sections, interleaved, not inverse)
    for x, y in zip(dev, back):
        # twice 5e-7 (|a| + |b|) in fp32; in bf16 the two roundings of a pair's elements, half a step each
        lim = (2.0 ** -6 if dtype == BF16 else 3e-6) * x.float().abs().amax(-1, keepdim=True)
        assert bool(((x.float() - y.float()).abs() <= lim).all())


def test_rope_is_its_gradient():
    """The gradient of sum(w * rope(x)) by the formula (rotate w back) against differences."""
    gen = torch.Generator().manual_seed(6)
    x = torch.randn((4, 2, 32), generator=gen)
    w = torch.randn((4, 2, 32), generator=gen)
    pos = torch.tensor([[3, 1000, -7, 50000], [1, 2, 3, 4]], dtype=torch.int32, device=DEV)
    freq = [100.0 ** (-i / 8) for i in range(8)]
    args = (pos, freq, (3, 5))
    grad = cpa.rope_axes([w.to(DEV)], *args, inverse=True)[0].double().cpu()

    def loss(z):
        return float((w.double() * torch.from_numpy(oc.rotate(z.double().numpy(), pos.cpu().numpy(), freq, (3, 5)))).sum())
    for at in [(0, 0, 0), (1, 1, 11), (2, 0, 12), (3, 1, 23), (3, 0, 24), (1, 0, 31), (2, 1, 5)]:
        e = torch.zeros((4, 2, 32), dtype=torch.float64)
        e[at] = 1.0  # the loss is linear in x: any step gives the exact slope
        diff = loss(x.double() + e) - loss(x.double() - e)
        assert abs(diff / 2 - float(grad[at])) <= 5e-7 * 2 * float(w.abs().max()) + 1e-12
    y = cpa.rope_axes([x.to(DEV)], *args)[0]
    assert abs(float((y.double().cpu() * w).sum()) - float((x * grad).sum())) <= 1e-4


def test_rope_takes_the_shard_layout_s_positions_and_graphs():
    qmap, pos = cpa.shard_layout(4096, 8, 5, "strided", positions=True)
    x = torch.randn((512, 3, 64), generator=torch.Generator().manual_seed(7)).to(BF16).to(DEV)
    freq = tuple(10000.0 ** (-i / 32) for i in range(32))
    y = cpa.rope_axes([x], pos, freq)[0]
    ref = oc.rotate(x.double().cpu().numpy(), [qmap.base + qmap.stride * np.arange(512)], freq, (32,))
    assert np.abs(y.double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-5
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cpa.rope_axes([x], pos, freq, out=[out])
    g.replay()
    assert torch.equal(out, y)
    pos += 1
    g.replay()
    assert torch.equal(out, cpa.rope_axes([x], pos, freq)[0]) and not torch.equal(out, y)
    assert torch.equal(cpa.rope_axes([x], pos, freq, stream=torch.cuda.Stream())[0].cpu(), out.cpu())


# ------------------------------------------------------------------ together
def test_prompt_then_decoding_over_four_ranks():
    """Two sequences served by four ranks with strided shards: the prompt's keys are rotated and
    written into each rank's cache, read back for the prompt's tensor-core attention, then two
    tokens are decoded, each rank over its own cache, and the ranks' partials merged."""
    cp, hq, hkv, d, page = 4, 8, 2, 64, 16
    prompt, steps = [140, 64], 2
    total = [p + steps for p in prompt]
    gen = torch.Generator().manual_seed(8)
    freq = tuple(10000.0 ** (-i / 32) for i in range(32))
    raw = [[torch.randn((n, h, d), generator=gen).to(BF16).to(DEV) for h in (hq, hkv, hkv)] for n in total]
    qk = []
    for b, n in enumerate(total):
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        q, k = cpa.rope_axes(raw[b][:2], pos, freq)
        qk.append((q, k, raw[b][2]))
    width = 12
    caches, tables = [], []
    for r in range(cp):
        caches.append(cpa.kv_cache_empty(2 * width, page, hkv, d))
        tables.append(torch.randperm(2 * width, generator=gen).reshape(2, width).int().to(DEV))

    def local(n, r):  # tokens of the first n that rank r holds
        return max(0, -(-(n - r) // cp))

    def put(lo, hi):
        for r in range(cp):
            have = [local(x, r) for x in lo]
            new = [local(x, r) - y for x, y in zip(hi, have)]
            k, v = (torch.cat([qk[b][w][[r + cp * j for j in range(have[b], have[b] + new[b])]] for b in range(2)])
                    for w in (1, 2))
            cpa.kv_cache_write(caches[r], k, v, _i32(_starts(new)), _i32(have), tables[r])
    put([0, 0], prompt)
    kept = []
    for b in range(2):  # every rank's keys and values as the cache holds them
        parts = []
        for r in range(cp):
            n = local(prompt[b], r)
            parts.append(cpa.kv_cache_read(caches[r], _i32([0, n]), _i32([0]), tables[r][b:b + 1], n))
        kept.append(parts)
        # the prompt's own attention: rank 1's queries against every rank's chunk
        q = qk[b][0][1:prompt[b]:cp].contiguous()
        o, lse = cpa.partial_attn_chunks(q, [(parts[r][0], parts[r][1], PosMap(r, cp)) for r in range(cp)], PosMap(1, cp))
        kpos = np.concatenate([r + cp * np.arange(local(prompt[b], r)) for r in range(cp)])
        o_ref, l_ref = oracle.attention(q.cpu(), torch.cat([p[0] for p in parts]).cpu(), torch.cat([p[1] for p in parts]).cpu(),
                                        1 + cp * np.arange(q.shape[0]), kpos, causal=True)
        helpers.compare_partial(o.cpu().numpy(), lse.cpu().numpy(), o_ref, l_ref, helpers.TOL_BF16_O, helpers.TOL_BF16_LSE)
    for step in range(steps):
        now = [p + step for p in prompt]
        put(now, [n + 1 for n in now])
        q = torch.cat([qk[b][0][now[b]:now[b] + 1] for b in range(2)])
        parts = []
        for r in range(cp):
            lens = _i32([local(n + 1, r) for n in now])
            parts.append(cpa.kv_cache_attn(q, caches[r], _i32([0, 1, 2]), lens, tables[r], q_first=_i32(now),
                                           kv_pos=PosMap(r, cp)))
        o, lse = cpa.merge_partials([p[0] for p in parts], [p[1] for p in parts], out_dtype=F32)
        for b in range(2):
            ks, vs, ps = [], [], []
            for r in range(cp):
                n = local(now[b] + 1, r)
                k, v = cpa.kv_cache_read(caches[r], _i32([0, n]), _i32([0]), tables[r][b:b + 1], n, dtype=F32)
                ks.append(k.cpu())
                vs.append(v.cpu())
                ps.append(r + cp * np.arange(n))
            o_ref, l_ref = oracle.attention(q[b:b + 1].cpu(), torch.cat(ks), torch.cat(vs), [now[b]], np.concatenate(ps))
            assert np.abs(o[b:b + 1].cpu().numpy() - o_ref).max() <= 2e-5
            assert np.abs(lse[b:b + 1].cpu().numpy() - l_ref).max() <= 2e-5

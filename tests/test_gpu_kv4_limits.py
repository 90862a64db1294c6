"""The calls around the 4-bit cache at the ends of what they accept, against the float64 oracle, with the tolerances of the
other tests unless one is derived here.
"""

import os

import numpy as np
import pytest
import torch

import helpers
from oracle import cache4 as o4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
import test_gpu_kv4 as kv4  # noqa: E402
from context_blockwise_attention_gb300 import PosMap  # noqa: E402
from test_gpu_kv4 import BF16, DEV, F32, Pool, _i32  # noqa: E402


@pytest.mark.parametrize("d,page,hq,dtype", [(64, 16, 8, BF16), (64, 64, 24, F32), (128, 32, 8, F32), (128, 128, 40, BF16)])
def test_rows_whose_query_is_not_finite_give_no_weight(d, page, hq, dtype):
    """Their LSE, the attention's own answer, is not finite, so they give nothing; the rows beside them give what they give
    without them."""
    rows, held = [3, 1, 2], [200, 70, 33]
    pool = Pool(3, held, page, 2, d, 201)
    pool.fill(held, 202)
    q = torch.randn((6, hq, d), generator=torch.Generator().manual_seed(203)).to(dtype)
    first = [m - n for n, m in zip(rows, held)]
    clean = cpa.kv4_cache_attn(q.to(DEV), pool.device(), _i32([0, 3, 4, 6]), _i32(held), _i32(pool.table), q_first=_i32(first))[1]
    spoilt = torch.zeros((6, hq), dtype=torch.bool)
    for i, h, e, x in ((0, 0, 3, "nan"), (1, hq - 1, 0, "inf"), (1, 1, d - 1, "-inf"), (2, hq // 2, 17, "nan"), (4, 2, 40, "inf"),
                       (4, hq // 2, 40, "nan")):
        q[i, h, e] = float(x)
        spoilt[i, h] = True
    q[5, 3] = float("inf")  # all of a row
    spoilt[5, 3] = True
    lse = cpa.kv4_cache_attn(q.to(DEV), pool.device(), _i32([0, 3, 4, 6]), _i32(held), _i32(pool.table), q_first=_i32(first))[1]
    assert torch.equal(lse.isfinite().cpu(), ~spoilt) and torch.equal(lse.cpu()[~spoilt], clean.cpu()[~spoilt])
    kv4._check_weigh(pool, q, rows, held, first, PosMap(0, 1), None, 1.0, 204)
    kv4._check_weigh(pool, q, rows, held, first, PosMap(0, 1), [190, 0, 33], 0.5, 205)


@pytest.mark.parametrize("wide,at_once", [(2500, 24), (0, 2), (600, 2)])  # split; one block; a cluster of blocks
@pytest.mark.parametrize("d,page,g,din,dout", [(64, 64, 4, BF16, BF16), (64, 16, 8, F32, F32), (64, 128, 12, BF16, F32),
                                               (128, 32, 4, F32, F32), (128, 64, 16, BF16, BF16), (128, 128, 8, BF16, F32),
                                               (128, 64, 20, BF16, BF16)])
def test_scores_of_any_size(d, page, g, din, dout, wide, at_once):
    """Rows whose largest score, from 2^10 to 2^98, is that of all tokens with one key, beside which the others vanish; and
    rows of the opposite sign, whose largest is that of the tokens with the key's opposite.  Equal keys have equal scores,
    so the answer is the mean of these tokens' values, off by what rounds weights and sums: w + n 2^-27 + 2^-20 of the mean
    magnitude (as for other calls, without the scores' errors), and the output's half step.  LSE is the score, within its own
    error, plus ln n."""
    held, hkv, rows = 700, 2, 24
    pool = Pool(1, [held], page, hkv, d, 211)
    rng = np.random.default_rng(212)
    key = rng.choice([-1.0, 1.0], (1, hkv, d)) * rng.uniform(0.5, 1, (1, hkv, d)) * 2.0 ** 13
    kind = rng.choice([1.0, 1.0, -1.0, 0.0, 0.5], held)
    o4.cache_write(pool.rows[0], kind[:, None, None] * key, [0, held], [0], pool.table)
    o4.cache_write(pool.rows[1], rng.standard_normal((held, hkv, d)), [0, held], [0], pool.table)
    x = torch.from_numpy(np.repeat(np.sign(key), g, 1) * np.abs(rng.standard_normal((rows // 2, hkv * g, d)))).to(F32)
    x = x * torch.exp2(torch.arange(rows // 2) * 8.0 - 4.0)[:, None, None]
    q = torch.stack((x, -3 * x), 1).reshape(rows, hkv * g, d).to(din)
    table = _i32(np.concatenate([pool.table, np.full((1, wide), -1)], 1))
    cache = pool.device()
    got = [cpa.kv4_cache_attn(q[i:i + at_once].to(DEV), cache, _i32([0, at_once]), _i32([held]), table, o_dtype=dout)
           for i in range(0, rows, at_once)]
    o, lse = (torch.cat(t).double().cpu().numpy() for t in zip(*got))
    k, v = pool.tokens_of(0, held)
    for i in range(rows):
        top = kind == (-1.0 if i % 2 else 1.0)
        n = int(top.sum())
        for h in range(hkv * g):
            qd = q[i, h].double().numpy()
            s = (k[:, h // g] @ qd) * d ** -0.5
            assert s[top].min() - np.max(s[~top]) > 200  # the others' weights are below any rounding
            vh = v[top, h // g]
            ref, mean = vh.mean(0), np.abs(vh).mean(0)
            w = 2.0 ** -11 if dout == BF16 else 2.0 ** -21
            tol = mean * (w + n * 2.0 ** -27 + 2.0 ** -20 + 2.0 ** -37)
            tol = tol + np.abs(ref) * (2.0 ** -8 if dout == BF16 else 2.0 ** -24) * 1.01
            err = np.abs(o[i, h] - ref)
            assert np.all(err <= tol), (i, h, s.max(), float((err / tol).max()))
            a = np.abs(k[top, h // g][0]) @ np.abs(qd) * d ** -0.5
            assert abs(lse[i, h] - (s.max() + np.log(n))) <= 2.0 ** -20 * a + 2.0 ** -22 * abs(s.max()) + n * 2.0 ** -24 + 2.0 ** -20


@pytest.mark.parametrize("wide,at_once", [(2500, 20), (0, 2), (600, 2)])
@pytest.mark.parametrize("d,page,din,dout", [(64, 64, BF16, BF16), (64, 16, F32, F32), (128, 32, BF16, F32), (128, 128, F32, F32)])
def test_large_scores_next_to_one_another(d, page, din, dout, wide, at_once):
    """Large scores that differ in their last steps of fp32, in any order.  Each is off by delta, and from 2^20 on those
    within 5 steps (2^-20 of the score) count as equal, so what is known of a row is that it is a mean of the values of tokens
    whose score is the largest but for that, and LSE that score plus the logarithm of at most their number."""
    held, rows = 900, 20
    pool = Pool(1, [held], page, 1, d, 241)
    rng = np.random.default_rng(242)
    key = rng.choice([-1.0, 1.0], (1, 1, d)) * 2.0 ** 13 * np.repeat([6.0, 4.0, 3.0, 2.0], d // 4)
    k = np.repeat(key, held, 0)
    small = rng.integers(0, d, held)  # one element of a token is a step smaller, most steps alike in the sum
    k[np.arange(held), 0, small] *= rng.choice([1.0, 0.75], held)
    o4.cache_write(pool.rows[0], k, [0, held], [0], pool.table)
    o4.cache_write(pool.rows[1], rng.standard_normal((held, 1, d)), [0, held], [0], pool.table)
    x = np.repeat(np.sign(key), 4, 1) * 2.0 ** rng.uniform(-16, 0, (rows, 4, d))
    x[:, :, :d // 2] = np.sign(key)[:, :, :d // 2]
    x = x * 2.0 ** np.arange(-2, rows - 2)[:, None, None] * rng.choice([-1.0, 1.0], (rows, 1, 1))
    q = torch.from_numpy(x).to(din)
    table = _i32(np.concatenate([pool.table, np.full((1, wide), -1)], 1))
    cache = pool.device()
    got = [cpa.kv4_cache_attn(q[i:i + at_once].to(DEV), cache, _i32([0, at_once]), _i32([held]), table, o_dtype=dout)
           for i in range(0, rows, at_once)]
    o, lse = (torch.cat(t).double().cpu().numpy() for t in zip(*got))
    k, v = (t[:, 0] for t in pool.tokens_of(0, held))
    for i in range(rows):
        for h in range(4):
            qd = q[i, h].double().numpy()
            s = (k @ qd) * d ** -0.5
            top = s.max()
            delta = float((2.0 ** -20 * d ** -0.5 * (np.abs(k) @ np.abs(qd)) + 2.0 ** -22 * np.abs(s)).max())
            among = v[s >= top - 2 * delta - 2.0 ** -20 * abs(top) - 40]
            # weights and sums: 2^-11 or 2^-21, 900 2^-27 and 2^-20; the output's half step
            tol = np.abs(among).max(0) * (2.0 ** -7 if dout == BF16 else 2.0 ** -16)
            assert np.all(o[i, h] >= among.min(0) - tol) and np.all(o[i, h] <= among.max(0) + tol), (i, h, top)
            off = delta + 2.0 ** -20 * abs(top) + 2.0 ** -20
            assert top - off <= lse[i, h] <= top + off + np.log(len(s)), (i, h, top, lse[i, h])


@pytest.mark.parametrize("scale,power", [(1e-12, None), (1e-38, -60), (1e-45, 0), (1e30, 20), (2e38, -140), (2e38, 100)])
@pytest.mark.parametrize("wide,d", [(0, 64), (0, 128), (2500, 64), (2500, 128)])
def test_softmax_scales_of_any_size(wide, d, scale, power):
    """Rows whose factor from products to scores leaves fp32's range: of zeros (power None) or small queries with a tiny
    scale, all of whose weights are equal, tokens that a row does not see among the others in a granule; and of a huge scale,
    where keys are zeros, so that scores are zeros all the same."""
    held, rows = 77, 4
    pool = Pool(1, [held], 32, 1, d, 221)
    rng = np.random.default_rng(222)
    if scale < 1:
        o4.cache_write(pool.rows[0], rng.standard_normal((held, 1, d)), [0, held], [0], pool.table)
    else:
        o4.cache_write(pool.rows[0], np.zeros((held, 1, d)), [0, held], [0], pool.table)
    o4.cache_write(pool.rows[1], rng.standard_normal((held, 1, d)), [0, held], [0], pool.table)
    q = torch.randn((rows, 2, d), generator=torch.Generator().manual_seed(223))
    q = q * 2.0 ** power if power is not None else q * 0
    table = _i32(np.concatenate([pool.table, np.full((1, wide), -1)], 1))
    args = (pool.device(), _i32([0, rows]), _i32([held]), table)
    kw = dict(q_first=_i32([held - rows - 9]), scale=scale)
    o, lse = cpa.kv4_cache_attn(q.to(DEV), *args, **kw)
    v = pool.tokens_of(0, held)[1][:, 0]
    w = torch.zeros((pool.n_pages, 1, 32), device=DEV)
    cpa.kv4_cache_weigh(q.to(DEV), lse, args[0], w, *args[1:], **kw)
    gathered = pool.gather(0, held, w.double().cpu().numpy())[:, 0]
    want = np.zeros(held)
    for i in range(rows):
        n = held - rows - 9 + i + 1
        want[:n] += 2 / n
        ref, mean = v[:n].mean(0), np.abs(v[:n]).mean(0)
        for h in range(2):
            assert np.all(np.abs(o[i, h].double().cpu().numpy() - ref) <= mean * (2.0 ** -21 + n * 2.0 ** -27 + 2.0 ** -20)
                          + np.abs(ref) * 2.0 ** -24)
            assert abs(float(lse[i, h]) - np.log(n)) <= 2.0 ** -20 + 2.0 ** -22 * np.log(n)
    # exp(s - LSE) is off by 2^-22 LSE + 2^-20 of itself, eight of them are added
    assert np.all(np.abs(gathered - want) <= want * (2.0 ** -22 * np.log(held) * 2 + 2.0 ** -20 + 10 * 2.0 ** -24))


@pytest.mark.parametrize("n,wide", [(100, 0), (100, 1000), (0, 0), (-4, 600), (9999, 0)])
def test_evict_to_the_largest_keep(n, wide):
    """No limit: nothing is evicted, every slot is answered, nothing is written in front of `kept` or behind it, and the
    workspace is as large as the page table needs.  (9999: more tokens than the table has pages for.)"""
    keep, guard = 2 ** 31 - 1, 4096
    pool = Pool(1, [100], 16, 1, 64, 251)
    pool.fill([100], 252)
    cache = pool.device()
    table = _i32(np.concatenate([pool.table, np.full((1, wide), -1)], 1))
    assert cpa.kv4_cache_evict_workspace(cache, 1, table.shape[1], keep) < 1 << 20
    buf = torch.full((guard + keep + guard,), 77, dtype=torch.int32, device=DEV)
    kept = buf[guard:guard + keep].view(1, keep)
    w = torch.rand((pool.n_pages, 1, 16), device=DEV)
    before = w.clone()
    _, lens = cpa.kv4_cache_evict(cache, w, _i32([n]), table, keep, 10, kept=kept)
    assert lens.item() == max(0, n) and torch.equal(w, before)
    kv4._same_cache(cache, pool)
    assert bool((buf[:guard] == 77).all()) and bool((buf[guard + keep:] == 77).all())
    m = max(0, n)
    assert torch.equal(kept[0, :m], torch.arange(m, dtype=torch.int32, device=DEV))
    for part in kept[0, m:].split(1 << 28):
        assert bool((part == -1).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_zeros_keep_their_sign(d, dtype):
    """Minus zero, and what is rounded to it, in a group of every scale."""
    scales = o4.SCALE[1:o4.MOST + 1]
    x = np.zeros((len(scales), 1, d))
    x[:, 0, 0::16] = 6 * scales[:, None]
    x[:, 0, 1::16] = -0.0
    x[:, 0, 2::16] = -0.2 * scales[:, None]
    x[:, 0, 3::16] = 0.2 * scales[:, None]
    x[:, 0, 15::16] = -0.0
    x = torch.from_numpy(x).to(dtype)
    rows = x.shape[0]
    pool = Pool(1, [rows], 16, 1, d, 231)
    cache = pool.device()
    args = (_i32([0, rows]), _i32([0]), _i32(pool.table))
    cpa.kv4_cache_write(cache, x.to(DEV), (-x).to(DEV), *args)
    o4.cache_write(pool.rows[0], x.double().numpy(), [0, rows], [0], pool.table)
    o4.cache_write(pool.rows[1], -x.double().numpy(), [0, rows], [0], pool.table)
    kv4._same_cache(cache, pool)
    k, v = cpa.kv4_cache_read(cache, *args, rows, dtype=dtype)
    assert torch.equal(torch.signbit(k).cpu(), torch.signbit(x)) and torch.equal(torch.signbit(v).cpu(), torch.signbit(-x))


def test_the_readme_s_serving_example_runs():
    with open(os.path.join(helpers.ROOT, "README.md")) as f:
        text = f.read()
    code = text[text.index("# serving, one rank"):]
    code = code[:code.index("```")]
    n_pages, page_size, hkv, hq, d, cp, rank = 20, 16, 2, 4, 64, 1, 0
    new, pages = [70, 3], 6
    gen = torch.Generator().manual_seed(261)
    names = dict(cpa=cpa, torch=torch, n_pages=n_pages, page_size=page_size, hkv=hkv, d=d, cp=cp, rank=rank,
                 q=torch.randn((73, hq, d), generator=gen).to(BF16).to(DEV), k=torch.randn((73, hkv, d), generator=gen).to(BF16).to(DEV),
                 v=torch.randn((73, hkv, d), generator=gen).to(BF16).to(DEV), row_start=_i32([0, 70, 73]), cached=_i32([0, 0]),
                 kv_lens=_i32(new), q_positions=_i32([0, 0]), positions=_i32(list(range(70)) + list(range(3))),
                 inv_freq=tuple(10000.0 ** (-i / 32) for i in range(32)), page_table=_i32(np.arange(2 * pages).reshape(2, pages)),
                 all_ranks_o=[torch.zeros((73, hq, d), device=DEV)], all_ranks_lse=[torch.zeros((73, hq), device=DEV)],
                 rows=_i32([0, 70, 73]), first=_i32([0, 0]), n_rows=73)
    exec(code, names)
    assert names["kp"].shape == names["vp"].shape == (73, hkv, d) and names["kept_lens"].tolist() == new
    # the prefix is what was written, to e4m3's half step at a page's scale
    assert bool(((names["kp"].float() - names["k"].float()).abs() <= names["k"].float().abs() * 2.0 ** -4 + 2.0 ** -7).all())


@pytest.mark.parametrize("d,page,hq,hkv,dtype", [(64, 16, 8, 2, BF16), (64, 128, 4, 4, F32), (128, 64, 10, 2, BF16), (128, 32, 6, 1, F32)])
def test_weights_of_a_prompt(d, page, hq, hkv, dtype):
    """A prompt's rows over its own tokens, a chunk of one over a longer cache, and single tokens in the same call."""
    rows, held = [300, 1, 130, 1, 2], [300, 420, 500, 1, 33]
    pool = Pool(5, held, page, hkv, d, 271)
    pool.fill(held, 272)
    q = torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(273)).to(dtype)
    first = [m - n for n, m in zip(rows, held)]
    kv4._check_weigh(pool, q, rows, held, first, PosMap(0, 1), [0, 419, 370, 0, 31], 0.75, 274)
    kv4._check_attn(pool, pool.device(), q, rows, held, first, PosMap(0, 1), dtype)


def test_many_heads():
    """1030 KV heads: more items, units of work and moving blocks than the SMs hold at once."""
    rows, held, hkv = [1, 3], [40, 7], 1030
    pool = Pool(2, [40, 7], 16, hkv, 64, 281)
    gen = torch.Generator().manual_seed(282)
    x = [torch.randn((47, hkv, 64), generator=gen).to(BF16) for _ in range(2)]
    cache = pool.device()
    args = (_i32([0, 40, 47]), _i32([0, 0]), _i32(pool.table))
    cpa.kv4_cache_write(cache, x[0].to(DEV), x[1].to(DEV), *args)
    for w in range(2):
        o4.cache_write(pool.rows[w], x[w].double().numpy(), [0, 40, 47], [0, 0], pool.table)
    kv4._same_cache(cache, pool)
    k, v = cpa.kv4_cache_read(cache, *args, 47, dtype=F32)
    for w, got in enumerate((k, v)):
        want = np.concatenate([pool.tokens_of(b, n)[w] for b, n in enumerate(held)])
        assert np.array_equal(got.double().cpu().numpy(), want)
    q = torch.randn((4, 2 * hkv, 64), generator=gen).to(BF16)
    kv4._check_attn(pool, cache, q, rows, held, [39, 4], PosMap(0, 1), F32)
    kv4._check_weigh(pool, q, rows, held, [39, 4], PosMap(0, 1), None, 1.0, 283)
    w = np.random.default_rng(284).uniform(0, 1, (pool.n_pages, hkv, 16)).astype(np.float32)
    kv4._check_evict(pool, held, 20, 5, w)


@pytest.mark.parametrize("wide,rows", [(0, 2), (600, 2), (2500, 2), (2500, 9)])
@pytest.mark.parametrize("d,page,din,dout", [(64, 16, BF16, BF16), (128, 64, F32, F32), (128, 32, BF16, F32)])
def test_infinite_scores_make_a_row_nan(d, page, din, dout, wide, rows):
    """By an infinity in a query that meets no zero and one sign of keys, and by finite products beyond fp32.  A bf16 query of
    minus infinity gives its tokens no weight; an fp32 one is NaN too, as its low part, -inf - -inf, is.  Other rows are as
    they were, to the bit."""
    held = 333
    pool = Pool(1, [held], page, 1, d, 291)
    rng = np.random.default_rng(292)
    k = rng.uniform(1, 2, (held, 1, d))
    o4.cache_write(pool.rows[0], k, [0, held], [0], pool.table)
    o4.cache_write(pool.rows[1], rng.standard_normal((held, 1, d)), [0, held], [0], pool.table)
    q = torch.randn((rows, 4, d), generator=torch.Generator().manual_seed(293)).to(din)
    table = _i32(np.concatenate([pool.table, np.full((1, wide), -1)], 1))
    args = (pool.device(), _i32([0, rows]), _i32([held]), table)
    want, lwant = cpa.kv4_cache_attn(q.to(DEV), *args, o_dtype=dout)
    assert bool(want.isfinite().all())
    q[0, 1, 7] = float("inf")
    q[1, 2] = 3e38  # a sum of d products of 3e38 or more
    q[1, 0, 3] = -float("inf")
    o, lse = cpa.kv4_cache_attn(q.to(DEV), *args, o_dtype=dout)
    left = torch.ones((rows, 4), dtype=torch.bool, device=DEV)
    for i, h in ((0, 1), (1, 2)):
        left[i, h] = False
        assert bool(o[i, h].isnan().all()) and bool(lse[i, h].isnan())
    left[1, 0] = False
    if din == BF16:
        assert bool((o[1, 0] == 0).all()) and lse[1, 0].item() == -float("inf")
    else:
        assert bool(o[1, 0].isnan().all()) and bool(lse[1, 0].isnan())
    assert torch.equal(o[left], want[left]) and torch.equal(lse[left], lwant[left])


@pytest.mark.parametrize("d,din,dout", [(64, BF16, F32), (64, BF16, BF16), (128, BF16, F32), (128, F32, F32)])
def test_light_tokens_count_beside_a_heavy_one(d, din, dout):
    """One token of weight 1 and two million of 2^-24.2, less than half a step of fp32 next to it.  The heavy key is zero, so its
    score is exact.  A warp adds a granule's weights up before they join its sum, which is off by half a step for each of its
    granules then, and not by a weight for each of its keys, of which a lane has 4 or 8 in a granule: (G + 8) 2^-24, and 2^-20
    for the rest."""
    page, hkv, n = 128, 8, 2000000 // 128 * 128
    cache = cpa.kv4_cache_empty(2, page, hkv, d)
    k = torch.zeros((2 * page, hkv, d))
    k[1:, :, 0] = -6.0
    v = torch.ones((2 * page, hkv, d))
    cpa.kv4_cache_write(cache, k.to(DEV), v.to(DEV), _i32([0, 2 * page]), _i32([0]), _i32([[0, 1]]))
    q = torch.zeros((1, hkv, d))
    q[:, :, 0] = 1.0
    scale = float(np.float32(24.2 * np.log(2) / 6))
    table = torch.ones((1, n // page), dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    o, lse = cpa.kv4_cache_attn(q.to(din).to(DEV), cache, _i32([0, 1]), _i32([n]), table, scale=scale, o_dtype=dout)
    light = np.exp(-6 * scale)
    granules = n * d // 4096
    share = hkv * (granules + 3) / (12 * torch.cuda.get_device_properties(DEV).multi_processor_count)
    keys = 512 // d  # of a lane in a granule
    assert light < 2.0 ** -24 and (share - 1) * (keys * light - 2.0 ** -24) / (1 + n * light) > 2.0 ** -20  # what would be lost
    want = np.log1p((n - 1) * light)
    assert bool(((lse.double() - want).abs() <= (share + 8) * 2.0 ** -24 + 2.0 ** -20).all()), (lse - want).abs().max()
    # every value is 6 times the scale nearest to 1 / 6, 11 / 64
    assert bool(((o.double() - 66 / 64).abs() <= 2.0 ** -7).all())

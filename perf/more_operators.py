"""Cases of the operators around a 4-bit cache of a rank that serves: storing keys and values in it
and reading them back, attention of new tokens over it, the attention weight that its tokens gather,
and the eviction of the tokens that gathered least.

``run`` computes each operator in its plain form (elementary torch operations, 32 bits), or, where
``own`` is true, by the calls that a program makes of the library.

The cache holds rows ``[pages, kv_heads, page_size, head_dim * 9 / 16]`` of bytes: the token's
numbers as e2m1 (sign, two exponent bits, one fraction bit; even elements in the low nibbles), then
one scale byte for each 16 of them, the upper bits of a half without its sign (five exponent bits,
three fraction bits).  A scale is the nearest such number to a sixth of the group's largest
magnitude, 10240 at most; a group with a number that is not finite has the byte 255 and codes of 0.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a prompt of several requests enters the cache and is read back as the prompt's attention sees it
        dict(name="store prompts", op="store", seqs=6, new_min=1000, new_max=9000, cached_min=0, cached_max=200,
             hkv=8, d=128, page=64, dtype="bf16", pick=1),
        # one decoding step of a batch, its tokens alone: latency
        dict(name="store one token each", op="store", seqs=128, new_min=1, new_max=1, cached_min=1, cached_max=8000,
             hkv=8, d=128, page=64, dtype="bf16", pick=2),
        # a few short ragged prompts in fp32, small pages, small heads
        dict(name="store short prompts", op="store", seqs=5, new_min=0, new_max=300, cached_min=0, cached_max=100,
             hkv=8, d=64, page=16, dtype="fp32", pick=3),
        # one request, one token: latency
        dict(name="attend one token", op="attn", seqs=1, q_min=1, q_max=1, kv_min=1000, kv_max=1000, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", out="bf16", cp=1, causal=True, pick=4),
        # a batch of requests of uneven length, one token each
        dict(name="attend batch", op="attn", seqs=64, q_min=1, q_max=1, kv_min=256, kv_max=8192, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", out="bf16", cp=1, causal=True, pick=5),
        # one rank's share of very long requests: the (O, LSE) partial is merged with the other ranks'
        dict(name="attend long shard", op="attn", seqs=8, q_min=1, q_max=1, kv_min=90000, kv_max=131072, hq=64, hkv=8,
             d=64, page=128, dtype="bf16", out="fp32", cp=8, causal=True, pick=6),
        # several proposed tokens per request are checked in one pass
        dict(name="attend drafts", op="attn", seqs=16, q_min=2, q_max=6, kv_min=1000, kv_max=20000, hq=32, hkv=8,
             d=128, page=32, dtype="bf16", out="bf16", cp=1, causal=True, pick=7),
        # as many KV heads as query heads, small pages, fp32 queries and partials, no causal limit
        dict(name="attend ungrouped", op="attn", seqs=7, q_min=1, q_max=2, kv_min=0, kv_max=8191, hq=32, hkv=32,
             d=128, page=16, dtype="fp32", out="fp32", cp=2, causal=False, pick=8),
        # the same batch gathers the weight that its tokens received in the step
        dict(name="weigh batch", op="weigh", seqs=64, q_min=1, q_max=1, kv_min=256, kv_max=8192, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", cp=1, causal=True, decay=1.0, pick=9),
        # long shards, checked drafts, older weight forgotten slowly
        dict(name="weigh long drafts", op="weigh", seqs=4, q_min=1, q_max=4, kv_min=30000, kv_max=65536, hq=64, hkv=8,
             d=64, page=128, dtype="fp32", cp=2, causal=True, decay=0.9375, pick=10),
        # a batch at its budget gives up what a hundred steps have added
        dict(name="evict to the budget", op="evict", seqs=64, kv_min=4000, kv_max=4224, keep=4096, recent=64, hkv=8,
             d=128, page=64, pick=11),
        # long prompts shrink to the budget for the first time
        dict(name="evict long prompts", op="evict", seqs=8, kv_min=20000, kv_max=65536, keep=4096, recent=256, hkv=8,
             d=64, page=128, pick=12),
    ]


def _log(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "weigh", "evict"])
    pick = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        seqs = _log(rng, 1, 128)
        most = max(1, min(16384, 29000 * 8 // (seqs * hkv)))
        new = _log(rng, 1, most)
        return dict(op=op, seqs=seqs, new_min=rng.choice([new, new // 2, 0 if seqs > 1 else new]), new_max=new,
                    cached_min=0, cached_max=_log(rng, 1, 2000), hkv=hkv, d=d, page=page, dtype=dtype, pick=pick)
    if op == "evict":
        seqs = _log(rng, 1, 64)
        kv = _log(rng, 2, max(2, min(131072, 400000 * 512 // (seqs * hkv * d))))
        keep = max(1, int(kv * rng.choice([0.03, 0.3, 0.9, 0.97])))
        return dict(op=op, seqs=seqs, kv_min=rng.choice([kv, kv // 2, 0]), kv_max=kv, keep=keep,
                    recent=min(keep, rng.choice([0, 16, 32, 100, 256, 1000])), hkv=hkv, d=d, page=page, pick=pick)
    group = rng.choice([1, 2, 4, 5, 8, 16])
    if hkv * group > 128:
        group = 128 // hkv
    seqs = _log(rng, 1, 64)
    q_max = rng.choice([1, 1, 1, 2, 4, _log(rng, 1, 16)])
    most = max(16, min(131072, 800000 * 512 // (seqs * hkv * d), 16000000 // (seqs * hkv * group * q_max)))
    kv = _log(rng, 1, most)
    case = dict(op=op, seqs=seqs, q_min=1, q_max=q_max, kv_min=rng.choice([kv, kv // 3, 0]), kv_max=kv,
                hq=hkv * group, hkv=hkv, d=d, page=page, dtype=dtype, cp=rng.choice([1, 1, 2, 8]),
                causal=rng.random() < 0.8, pick=pick)
    if op == "attn":
        case["out"] = rng.choice(["bf16", "fp32"])
    else:
        case["decay"] = rng.choice([1.0, 1.0, 0.96875, 0.5])
    return case


def _lengths(case, lo, hi, salt):
    """A length for each sequence, from the case alone: both ends of the range are among them."""
    r = random.Random(case["pick"] * 7 + salt)
    n = [r.randint(lo, hi) for _ in range(case["seqs"])]
    n[-1] = hi
    if len(n) > 1:
        n[r.randrange(len(n) - 1)] = lo
    return n


def _rows_of(case):
    """Rows of the call and cached tokens before them (store) or under them, for each sequence."""
    if case["op"] == "evict":
        return [0] * case["seqs"], _lengths(case, case["kv_min"], case["kv_max"], 2)
    if case["op"] == "store":
        return (_lengths(case, case["new_min"], case["new_max"], 1),
                _lengths(case, case["cached_min"], case["cached_max"], 2))
    return _lengths(case, case["q_min"], case["q_max"], 1), _lengths(case, case["kv_min"], case["kv_max"], 2)


def _first_query(case, rows, held):
    """Position of each sequence's first new token: the last sees every cached token, the first may not."""
    base = case["cp"] - 1
    return [base + case["cp"] * (m - 1) - (n - 1) for n, m in zip(rows, held)]


def _visible(case):
    """Sum over the rows of the cached tokens that each sees, and over the sequences of those that any row sees."""
    rows, held = _rows_of(case)
    if not case["causal"]:
        return sum(n * m for n, m in zip(rows, held)), sum(m for n, m in zip(rows, held) if n)
    pairs = read = 0
    for n, m, f in zip(rows, held, _first_query(case, rows, held)):
        seen = [max(0, min(m, (f + t - (case["cp"] - 1)) // case["cp"] + 1)) for t in range(n)]
        pairs += sum(seen)
        read += seen[-1] if seen else 0
    return pairs, read


def work(case):
    size = 4 if case.get("dtype") == "fp32" else 2
    row = case["d"] * 9 / 16
    rows, held = _rows_of(case)
    if case["op"] == "store":  # numbers in, rows out, rows in, numbers out
        n = 2 * sum(rows) * case["hkv"]
        return {"bytes": 2 * n * (case["d"] * size + row), "flops": 3 * n * case["d"]}
    if case["op"] == "evict":  # all weights; rows that change their place, as many as of equally likely ones
        moved = 0.0
        for n in held:
            if n > case["keep"]:
                old, most = n - case["recent"], case["keep"] - case["recent"]
                moved += (most * (old - most) / old if old else 0) + case["recent"]
        tokens = sum(held)
        return {"bytes": 4 * tokens * case["hkv"] + 2 * moved * case["hkv"] * (2 * row + 4)
                + 4 * sum(min(n, case["keep"]) for n in held), "flops": tokens * case["hkv"]}
    pairs, read = _visible(case)
    if case["op"] == "weigh":  # keys; weights in and out
        return {"bytes": read * case["hkv"] * row + 8 * sum(held) * case["hkv"] + sum(rows) * case["hq"] * (case["d"] * size + 4)
                + 4 * read // case["page"], "flops": 2 * pairs * case["hq"] * case["d"]}
    out = 4 if case["out"] == "fp32" else 2
    return {"bytes": 2 * read * case["hkv"] * row + sum(rows) * case["hq"] * (case["d"] * (size + out) + 4)
            + 4 * read // case["page"], "flops": 4 * pairs * case["hq"] * case["d"]}


# ------------------------------------------------------------------ inputs
def _normal(shape, dtype, gen, outliers=False):
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:  # the spread that keys show: one value in a hundred is eight times larger
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, 8 * x, x)
    return x.to(dtype)


def _filled_cache(pages, case, gen):
    """Rows of random numbers: any codes, scales as those of numbers around 1 (keys with some larger)."""
    out = []
    for outliers in (True, False):
        shape = (pages, case["hkv"], case["page"])
        codes = torch.randint(0, 256, (*shape, case["d"] // 2), generator=gen, device="cuda", dtype=torch.uint8)
        amax = 1.0 + 1.5 * torch.rand((*shape, case["d"] // 16), generator=gen, device="cuda")
        if outliers:
            amax = torch.where(torch.rand(amax.shape, generator=gen, device="cuda") < 0.1, 4 * amax, amax)
        out.append(torch.cat((codes, _scale_code(amax)), -1))
        del codes, amax
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    rows, held = _rows_of(case)
    reach = [n + m if case["op"] == "store" else m for n, m in zip(rows, held)]
    width = max(1, -(-max(reach) // case["page"]))
    used = [-(-r // case["page"]) for r in reach]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([sum(used[:b]) for b in range(len(used))], device="cuda")
    col = torch.arange(width, device="cuda")
    count = torch.tensor(used, device="cuda")
    index = (at[:, None] + col[None, :]).clamp(max=pages - 1)
    s["page_table"] = torch.where(col[None, :] < count[:, None], order[index], -1).to(torch.int32).contiguous()
    s["cache"] = _filled_cache(pages, case, gen)
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    s["row_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["held"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    s["rows"] = starts[-1]
    s["longest"] = max(rows)
    if case["op"] == "evict":  # weights as they gather: most tokens little, some very much
        shape = (pages, case["hkv"], case["page"])
        s["gathered"] = torch.exp(2 * torch.randn(shape, generator=gen, device="cuda") - 8)
        s["weight"] = torch.empty_like(s["gathered"])
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "store":
        s["k"] = _normal((s["rows"], case["hkv"], case["d"]), dt, gen, True)
        s["v"] = _normal((s["rows"], case["hkv"], case["d"]), dt, gen)
        return s
    s["q"] = _normal((s["rows"], case["hq"], case["d"]), dt, gen)
    s["q_first"] = None
    if case["causal"]:
        s["q_first"] = torch.tensor(_first_query(case, rows, held), dtype=torch.int32, device="cuda")
    if case["op"] == "weigh":
        s["weight"] = torch.rand((pages, case["hkv"], case["page"]), generator=gen, device="cuda")
        # the tokens of this step have gathered nothing yet
        s["known"] = torch.tensor([max(0, m - n) for n, m in zip(rows, held)], dtype=torch.int32, device="cuda")
        s["lse"] = _by_row(s, torch.logsumexp(_scores(s), -1)).contiguous()
    return s


# ------------------------------------------------------------------ plain forms
def _scale_code(amax):
    """The byte of the nearest scale to amax / 6, in 32 bits."""
    x = amax / 6
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-14) - 3)
    near = (torch.round(x / step) * step).clamp(max=10240.0)
    code = near.to(torch.float16).view(torch.int16) >> 7
    return torch.where(amax.isfinite(), code, 255).to(torch.uint8)


def _scale_of(code):
    return (code.to(torch.int16) << 7).view(torch.float16).float()


def _coded(x):
    """Rows of the cache for x [..., d]."""
    g = x.float().unflatten(-1, (-1, 16))
    code = _scale_code(g.abs().amax(-1))
    scale = _scale_of(code)[..., None]
    y = g.abs() / scale
    up = (y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5)
    up = up | torch.signbit(g).to(torch.uint8) << 3
    up = torch.where((scale > 0) & scale.isfinite(), up, torch.zeros_like(up)).flatten(-2)
    return torch.cat((up[..., 0::2] | up[..., 1::2] << 4, code), -1)


def _values(row):
    """Numbers of rows of the cache, fp32."""
    d = row.shape[-1] * 16 // 9
    codes = row[..., :d // 2]
    nibbles = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    table = torch.tensor(E2M1 + [-x for x in E2M1], device=row.device)
    return (table[nibbles].unflatten(-1, (-1, 16)) * _scale_of(row[..., d // 2:])[..., None]).flatten(-2)


def _places(s):
    """Page and slot of each row of the call."""
    row = torch.arange(s["rows"], device="cuda")
    start = s["row_start"].long()
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = s["held"].long()[seq] + row - start[seq]
    return s["page_table"].long()[seq, pos // s["page"]], pos % s["page"]


def _plain_store(s):
    page, slot = _places(s)
    out = []
    for x, cache in zip((s["k"], s["v"]), s["cache"]):
        cache[page, :, slot] = _coded(x)
        out.append(_values(cache[page, :, slot]).to(x.dtype))
    return out


def _by_seq(cache, s):
    """Numbers of the cache by sequence: [seqs, hkv, keys, d]."""
    x = _values(cache[s["page_table"].long().clamp(min=0)]).transpose(1, 2)
    return x.reshape(x.shape[0], s["hkv"], -1, s["d"])


def _scores(s):
    """Scores [seqs, hkv, longest, group, keys], -inf where a key is not seen."""
    kk = _by_seq(s["cache"][0], s)
    seqs, _, keys, _ = kk.shape
    t = torch.arange(s["longest"], device="cuda")
    row = (s["row_start"].long()[:-1, None] + t).clamp(max=max(0, s["rows"] - 1))
    q = s["q"].float()[row].reshape(seqs, s["longest"], s["hkv"], -1, s["d"]).permute(0, 2, 1, 3, 4)
    scores = q.reshape(seqs, s["hkv"], -1, s["d"]) @ kk.transpose(2, 3) / math.sqrt(s["d"])
    j = torch.arange(keys, device="cuda")
    seen = (j < s["held"].long()[:, None])[:, None, :]
    if s["q_first"] is not None:
        at = s["cp"] - 1 + s["cp"] * j
        seen = seen & (at <= (s["q_first"].long()[:, None] + t)[:, :, None])
    seen = seen & (t[None, :] < s["row_start"].diff()[:, None])[:, :, None]
    seen = seen.expand(seqs, s["longest"], keys)[:, None, :, None, :]
    return scores.reshape(seqs, s["hkv"], s["longest"], -1, keys).masked_fill(~seen, -math.inf)


def _row_places(s):
    """Sequence and number within it of each row of the call."""
    start = s["row_start"].long()
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(start[1:], row, right=True)
    return seq, row - start[seq]


def _by_row(s, x):
    """[seqs, hkv, longest, group, ...] as [rows, hq, ...]."""
    return x.transpose(1, 2)[_row_places(s)].flatten(1, 2)


def _plain_attn(s):
    scores = _scores(s)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1)
    o = (p.flatten(2, 3) @ _by_seq(s["cache"][1], s)).reshape(*p.shape[:-1], s["d"])
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    return _by_row(s, o).to(DTYPES[s["out"]]), _by_row(s, top[..., 0] + torch.log(total))


def _plain_weigh(s):
    scores = _scores(s)
    seq, t = _row_places(s)
    lse = torch.full((scores.shape[0], s["longest"], s["hq"]), math.inf, device="cuda")
    lse[seq, t] = torch.where(s["lse"].isfinite(), s["lse"], math.inf)
    lse = lse.unflatten(2, (s["hkv"], -1)).transpose(1, 2)
    new = torch.exp(scores - lse[..., None]).sum((2, 3))  # [seqs, hkv, keys]
    table = s["page_table"].long()
    j = torch.arange(new.shape[2], device="cuda")
    old = s["weight"][table.clamp(min=0)].transpose(1, 2).flatten(2) * s["decay"]
    new = new + torch.where(j < s["known"].long()[:, None, None], old, torch.zeros_like(old))
    seq, at = ((j < s["held"].long()[:, None]) & (s["row_start"].diff() > 0)[:, None]).nonzero(as_tuple=True)
    s["weight"][table[seq, at // s["page"]], :, at % s["page"]] = new[seq, :, at]
    return s["weight"]


def _plain_evict(s):
    weight = s["weight"].copy_(s["gathered"])
    table, n = s["page_table"].long(), s["held"].long()[:, None]
    seqs, keys = table.shape[0], table.shape[1] * s["page"]
    total = weight[table.clamp(min=0)].double().sum(2).float().flatten(1)  # [seqs, keys]
    j = torch.arange(keys, device="cuda")[None, :].expand(seqs, keys)
    after = n.clamp(max=s["keep"])
    old, most = n - s["recent"], after - s["recent"]  # tokens that may go; those of them that stay
    old = torch.where(n > s["keep"], old, n)
    most = torch.where(n > s["keep"], most, n)
    order = torch.where(j < old, total, -math.inf).sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j)
    stay = (rank < most) & (j < old)
    # tokens behind the first `most` slots that stay go, in order, where others leave room
    hole, mover = ~stay & (j < most), stay & (j >= most)
    seq, to = hole.nonzero(as_tuple=True)
    _, source = mover.nonzero(as_tuple=True)
    kept = torch.full((seqs, max(keys, s["keep"])), -1, device="cuda")
    kept[:, :keys] = torch.where(j < most, j, torch.where(j < after, j + n - after, -1))
    kept[seq, to] = source
    kept = kept[:, :s["keep"]]
    seq, to = ((kept >= 0) & (kept != torch.arange(s["keep"], device="cuda"))).nonzero(as_tuple=True)
    source = kept[seq, to]
    for x in (*s["cache"], weight):
        x[table[seq, to // s["page"]], :, to % s["page"]] = x[table[seq, source // s["page"]], :, source % s["page"]]
    return kept.to(torch.int32), after[:, 0].to(torch.int32), weight, *s["cache"]


# ------------------------------------------------------------------ the operators
def _own(s):
    import context_blockwise_attention_gb300 as cpa

    cache = cpa.Kv4Cache(*s["cache"])
    if s["op"] == "store":
        cpa.kv4_cache_write(cache, s["k"], s["v"], s["row_start"], s["held"], s["page_table"])
        return cpa.kv4_cache_read(cache, s["row_start"], s["held"], s["page_table"], s["rows"],
                                  dtype=DTYPES[s["dtype"]])
    if s["op"] == "evict":
        # a pass that is made again finds the weights as they were
        weight = s["weight"].copy_(s["gathered"])
        kept, lens = cpa.kv4_cache_evict(cache, weight, s["held"], s["page_table"], s["keep"], s["recent"])
        return kept, lens, weight, *s["cache"]
    pos = cpa.PosMap(s["cp"] - 1, s["cp"])
    if s["op"] == "weigh":
        return cpa.kv4_cache_weigh(s["q"], s["lse"], cache, s["weight"], s["row_start"], s["held"], s["page_table"],
                                   known=s["known"], q_first=s["q_first"], kv_pos=pos, decay=s["decay"])
    return cpa.kv4_cache_attn(s["q"], cache, s["row_start"], s["held"], s["page_table"], q_first=s["q_first"],
                              kv_pos=pos, o_dtype=DTYPES[s["out"]])


def run(state):
    if own:
        return _own(state)
    return {"store": _plain_store, "attn": _plain_attn, "weigh": _plain_weigh,
            "evict": _plain_evict}[state["op"]](state)


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "attn": _exact_attn, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _nearest(x, grid):
    """The index of the number of an increasing grid that is nearest to each x >= 0; ties to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - x, x - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


SCALES = [(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 15) for e in range(31) for m in range(8)]


def _exact_store(s):
    # every token of the call has a place of its own, so that what is read back is what it was coded to
    out = []
    for x in (s["k"], s["v"]):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for h in range(s["hkv"]):
            g = x[:, h].double().unflatten(-1, (-1, 16))
            scale = torch.tensor(SCALES, dtype=torch.float64, device="cuda")[_nearest(g.abs().amax(-1) / 6, SCALES)]
            scale = scale.clamp(max=10240.0)[..., None]
            code = _nearest(torch.where(scale > 0, g.abs() / scale, 0.0), E2M1)
            y[:, h] = (torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code] * scale * torch.sign(g)).flatten(-2)
        out.append(y)
    return out


def _exact_rows(s, which, b, h, m):
    """The first m tokens of a sequence and head, in 64 bits."""
    row = s["cache"][which][s["page_table"][b, :-(-m // s["page"])].long(), h].flatten(0, 1)[:m].long()
    d = s["d"]
    byte = row[:, d // 2:]
    e, f = byte >> 3, byte & 7
    scale = torch.where(e > 0, (8 + f).double() * 2.0 ** (e - 18).double(), f.double() * 2.0 ** -17)
    x = torch.empty((m, d), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        c = row[:, :d // 2] >> 4 * half & 15
        e, f = c >> 1 & 3, c & 1
        size = torch.where(e > 0, (2 + f).double() * 2.0 ** (e - 2).double(), f.double() / 2)
        x[:, half::2] = torch.where(c > 7, -size, size)
    return x * torch.repeat_interleave(scale, 16, 1)


def _exact_scores(s, b, h):
    """Scores of a sequence and KV head [rows, group, tokens], and which are seen."""
    m = int(s["held"][b])
    r0, r1 = int(s["row_start"][b]), int(s["row_start"][b + 1])
    group = s["hq"] // s["hkv"]
    seen = torch.ones((r1 - r0, m), dtype=torch.bool, device="cuda")
    if s["q_first"] is not None:
        key = s["cp"] * torch.arange(m, device="cuda") + s["cp"] - 1
        seen = key[None, :] <= (int(s["q_first"][b]) + torch.arange(r1 - r0, device="cuda"))[:, None]
    q = s["q"][r0:r1, h * group:(h + 1) * group].double()
    z = torch.einsum("ngd,md->ngm", q, _exact_rows(s, 0, b, h, m)) / math.sqrt(s["d"])
    return torch.where(seen[:, None, :], z, torch.full_like(z, -math.inf)), seen[:, None, :]


def _exact_attn(s):
    o = torch.zeros((s["rows"], s["hq"], s["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], s["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group, start = s["hq"] // s["hkv"], s["row_start"].tolist()
    for b, m in enumerate(s["held"].tolist()):
        if m == 0 or start[b] == start[b + 1]:
            continue
        for h in range(s["hkv"]):
            z, seen = _exact_scores(s, b, h)
            norm = torch.logsumexp(z, -1)
            weight = torch.where(seen & norm.isfinite()[..., None], torch.exp(z - norm[..., None]), torch.zeros_like(z))
            at = slice(start[b], start[b + 1]), slice(h * group, (h + 1) * group)
            o[at] = torch.einsum("ngm,md->ngd", weight, _exact_rows(s, 1, b, h, m))
            lse[at] = norm
    return o, lse


def _exact_weigh(s):
    weight = s["weight"].double()
    group, start = s["hq"] // s["hkv"], s["row_start"].tolist()
    for b, m in enumerate(s["held"].tolist()):
        if m == 0 or start[b] == start[b + 1]:
            continue
        at = torch.arange(m, device="cuda")
        page, slot = s["page_table"][b, at // s["page"]].long(), at % s["page"]
        for h in range(s["hkv"]):
            z, _ = _exact_scores(s, b, h)
            lse = s["lse"][start[b]:start[b + 1], h * group:(h + 1) * group].double()
            p = torch.where(lse.isfinite()[..., None], torch.exp(z - lse[..., None]), torch.zeros_like(z))
            old = torch.where(at < int(s["known"][b]), weight[page, h, slot] * s["decay"], 0.0)
            weight[page, h, slot] = old + p.sum((0, 1))
    return weight


def _exact_evict(s):
    # whole numbers and bytes that are moved have no value of another precision; the weights move with them
    weight = s["gathered"].double()
    for b, n in enumerate(s["held"].tolist()):
        if n <= s["keep"]:
            continue
        at = torch.arange(n, device="cuda")
        page, slot = s["page_table"][b, at // s["page"]].long(), at % s["page"]
        mine = weight[page, :, slot]
        total = mine.sum(1)[:n - s["recent"]].tolist()
        most = s["keep"] - s["recent"]
        stay = sorted(sorted(range(len(total)), key=lambda i: (-total[i], i))[:most])
        inside = set(i for i in stay if i < most)
        source, behind = list(range(most)) + list(range(n - s["recent"], n)), iter(i for i in stay if i >= most)
        for i in range(most):
            if i not in inside:
                source[i] = next(behind)
        to = slice(0, s["keep"])
        weight[page[to], :, slot[to]] = mine[torch.tensor(source, dtype=torch.long, device="cuda")]
    return None, None, weight, None, None

"""Cases of the operators of a rank that serves and trains over a sharded sequence: writing keys
and values into a paged 8-bit cache, reading them back, attention of new tokens over that cache,
and rotary positions with several axes.

``run`` computes each operator in its plain form (elementary torch operations, 32 bits), or, where
``own`` is true, by the calls that a program makes of the library.

The cache holds e4m3 values in pages ``[pages, kv_heads, page_size, head_dim]`` with one
power-of-two scale per page and head: the smallest 2^e at which the page's largest magnitude is at
most 448 (never below 2^-64).  A page that is written from its first slot on takes the scale of
what is written; one that is continued takes the larger of its own and the new tokens' scale, and
the values already in it are rounded once more at that scale.
"""

import math
import random

import torch

own = False

MIN_EXP = -64
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a prompt of several requests enters the cache; some pages are continued
        dict(name="write prompts", op="write", seqs=6, new_min=1000, new_max=9000, cached_min=0, cached_max=200,
             hkv=8, d=128, page=64, dtype="bf16", pick=1),
        # one decoding step of a batch: one token per request, in the middle of its last page
        dict(name="write one token each", op="write", seqs=128, new_min=1, new_max=1, cached_min=1, cached_max=8000,
             hkv=8, d=128, page=64, dtype="bf16", pick=2),
        # a cached prefix is read back as bf16 keys and values for a prompt's tensor-core attention
        dict(name="read prefixes", op="read", seqs=4, new_min=4000, new_max=16384, cached_min=0, cached_max=500,
             hkv=8, d=128, page=64, dtype="bf16", pick=3),
        # a few short ranges in fp32, small pages, ragged
        dict(name="read short ranges", op="read", seqs=5, new_min=0, new_max=300, cached_min=0, cached_max=100,
             hkv=8, d=64, page=16, dtype="fp32", pick=4),
        # one request, one token: latency
        dict(name="attend one token", op="attn", seqs=1, q_min=1, q_max=1, kv_min=1000, kv_max=1000, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", out="bf16", cp=1, causal=True, pick=5),
        # a batch of requests of uneven length, one token each
        dict(name="attend batch", op="attn", seqs=64, q_min=1, q_max=1, kv_min=256, kv_max=8192, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", out="bf16", cp=1, causal=True, pick=6),
        # one rank's share of very long requests: the (O, LSE) partial is merged with the other ranks'
        dict(name="attend long shard", op="attn", seqs=8, q_min=1, q_max=1, kv_min=90000, kv_max=131072, hq=64, hkv=8,
             d=64, page=128, dtype="bf16", out="fp32", cp=8, causal=True, pick=7),
        # several proposed tokens per request are checked in one pass
        dict(name="attend drafts", op="attn", seqs=16, q_min=2, q_max=6, kv_min=1000, kv_max=20000, hq=32, hkv=8,
             d=128, page=32, dtype="bf16", out="bf16", cp=1, causal=True, pick=8),
        # as many KV heads as query heads, small pages, fp32 partials, no causal limit
        dict(name="attend ungrouped", op="attn", seqs=7, q_min=1, q_max=2, kv_min=0, kv_max=8191, hq=32, hkv=32,
             d=128, page=16, dtype="fp32", out="fp32", cp=2, causal=False, pick=9),
        # a decoding step's queries and keys
        dict(name="rotate one step", op="rope", tokens=64, hq=64, hkv=8, d=64, rot=64, axes=1, interleaved=False,
             inverse=False, dtype="bf16", span=1000000, pick=10),
        # a shard of a video prompt: time, height and width, queries and keys in one call
        dict(name="rotate video shard", op="rope", tokens=32768, hq=32, hkv=8, d=128, rot=128, axes=3,
             interleaved=False, inverse=False, dtype="bf16", span=4096, pick=11),
        # gradients of rotated queries and keys, part of the head rotated, neighbours paired
        dict(name="rotate gradients back", op="rope", tokens=8191, hq=64, hkv=8, d=64, rot=32, axes=2,
             interleaved=True, inverse=True, dtype="fp32", span=262144, pick=12),
    ]


def _log(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "rope"])
    pick = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    page = rng.choice([16, 32, 64, 128])
    if op in ("write", "read"):
        seqs = _log(rng, 1, 128)
        most = max(1, min(16384, 60000 * 8 // (seqs * hkv)))
        new = _log(rng, 1, most)
        return dict(op=op, seqs=seqs, new_min=rng.choice([new, new // 2, 0 if seqs > 1 else new]), new_max=new,
                    cached_min=0, cached_max=_log(rng, 1, 2000), hkv=hkv, d=d, page=page, dtype=dtype, pick=pick)
    if op == "attn":
        group = rng.choice([1, 2, 4, 5, 8, 16])
        if hkv * group > 128:
            group = 128 // hkv
        seqs = _log(rng, 1, 64)
        q_max = rng.choice([1, 1, 1, 2, 4, _log(rng, 1, 16)])
        most = max(16, min(131072, 800000 * 512 // (seqs * hkv * d), 16000000 // (seqs * hkv * group * q_max)))
        kv = _log(rng, 1, most)
        return dict(op=op, seqs=seqs, q_min=1, q_max=q_max, kv_min=rng.choice([kv, kv // 3, 0]), kv_max=kv,
                    hq=hkv * group, hkv=hkv, d=d, page=page, dtype=dtype, out=rng.choice(["bf16", "fp32"]),
                    cp=rng.choice([1, 1, 2, 8]), causal=rng.random() < 0.8, pick=pick)
    group = rng.choice([1, 2, 4, 8])
    size = 4 if dtype == "fp32" else 2
    tokens = _log(rng, 1, max(1, min(32768, 800000000 // (2 * size * hkv * (group + 1) * d))))
    return dict(op="rope", tokens=tokens, hq=hkv * group, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]),
                axes=rng.choice([1, 2, 3, 4]), interleaved=rng.random() < 0.4, inverse=rng.random() < 0.4,
                dtype=dtype, span=_log(rng, 16, 1 << 30), pick=pick)


def _lengths(case, lo, hi, salt):
    """A length for each sequence, from the case alone: both ends of the range are among them."""
    r = random.Random(case["pick"] * 7 + salt)
    n = [r.randint(lo, hi) for _ in range(case["seqs"])]
    n[-1] = hi
    if len(n) > 1:
        n[r.randrange(len(n) - 1)] = lo
    return n


def _rows_of(case):
    """Rows of the call and cached tokens before them, for each sequence."""
    if case["op"] == "attn":
        return _lengths(case, case["q_min"], case["q_max"], 1), _lengths(case, case["kv_min"], case["kv_max"], 2)
    return (_lengths(case, case["new_min"], case["new_max"], 1),
            _lengths(case, case["cached_min"], case["cached_max"], 2))


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
    if case["op"] == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * n * case["d"] * size + 4 * case["axes"] * case["tokens"], "flops": 3 * n * case["rot"]}
    rows, held = _rows_of(case)
    if case["op"] == "attn":
        pairs, read = _visible(case)
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": 2 * read * case["hkv"] * case["d"] + sum(rows) * case["hq"] * (case["d"] * (size + out) + 4)
                + 8 * case["hkv"] * read // case["page"] + 4 * read // case["page"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    n = 2 * sum(rows) * case["hkv"] * case["d"]
    return {"bytes": n * (size + 1), "flops": 2 * n}


# ------------------------------------------------------------------ inputs
def _normal(shape, dtype, gen, outliers=False):
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:  # the spread that keys show: one value in a hundred is eight times larger
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, 8 * x, x)
    return x.to(dtype)


def _filled_cache(pages, case, gen):
    shape = (pages, case["hkv"], case["page"], case["d"])
    out = []
    for outliers in (True, False):
        x = _normal(shape, torch.float32, gen, outliers)
        scale = _scale_of(x.abs().amax((2, 3)))
        out.append((_round8(x / scale[:, :, None, None]), scale))
        del x
    return out[0][0], out[1][0], out[0][1], out[1][1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "rope":
        s["x"] = [_normal((case["tokens"], h, case["d"]), dt, gen) for h in (case["hq"], case["hkv"])]
        s["positions"] = torch.randint(0, case["span"], (case["axes"], case["tokens"]), generator=gen, device="cuda",
                                       dtype=torch.int32)
        half = case["rot"] // 2
        cut = [half // case["axes"]] * case["axes"]
        cut[0] += half - sum(cut)
        s["sections"] = tuple(cut)
        s["inv_freq"] = tuple(10000.0 ** (-i / half) for i in range(half))
        return s
    rows, held = _rows_of(case)
    reach = [m if case["op"] == "attn" else n + m for n, m in zip(rows, held)]
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
    if case["op"] == "write":
        s["k"] = _normal((s["rows"], case["hkv"], case["d"]), dt, gen, True)
        s["v"] = _normal((s["rows"], case["hkv"], case["d"]), dt, gen)
    if case["op"] == "attn":
        s["q"] = _normal((s["rows"], case["hq"], case["d"]), dt, gen)
        s["q_first"] = None
        if case["causal"]:
            s["q_first"] = torch.tensor(_first_query(case, rows, held), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _scale_of(amax):
    """The smallest power of two at which a magnitude is at most 448, in 32 bits."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _round8(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _values(b):
    return b.view(torch.float8_e4m3fn).float()


def _places(s):
    """Page, slot and sequence of each row of the call."""
    row = torch.arange(s["rows"], device="cuda")
    start = s["row_start"].long()
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = s["held"].long()[seq] + row - start[seq]
    return s["page_table"].long()[seq, pos // s["page"]], pos % s["page"], seq


def _plain_write_one(s, x, cache, scale, page, slot):
    new = torch.zeros_like(scale)
    token = x.float().abs().amax(2)
    new.scatter_reduce_(0, page[:, None].expand_as(token), token, "amax")
    first = torch.full((scale.shape[0],), s["page"], device="cuda").scatter_reduce_(0, page, slot, "amin")
    touched, fresh = first < s["page"], first == 0
    new = _scale_of(new)
    after = torch.where(touched[:, None], torch.where(fresh[:, None], new, torch.maximum(new, scale)), scale)
    go_on = (touched & ~fresh).nonzero()[:, 0]
    cache = cache.view(torch.uint8)
    held = cache[go_on].view(torch.float8_e4m3fn).float()
    again = _round8(held * (scale[go_on] / after[go_on])[:, :, None, None])
    kept = torch.arange(s["page"], device="cuda")[None, None, :, None] < first[go_on][:, None, None, None]
    cache[go_on] = torch.where(kept, again.view(torch.uint8), cache[go_on])
    cache[page, :, slot] = _round8(x.float() / after[page][:, :, None]).view(torch.uint8)
    scale.copy_(after)


def _plain_write(s):
    page, slot, _ = _places(s)
    k, v, ks, vs = s["cache"]
    _plain_write_one(s, s["k"], k, ks, page, slot)
    _plain_write_one(s, s["v"], v, vs, page, slot)
    return s["cache"]


def _plain_read(s):
    page, slot, _ = _places(s)
    k, v, ks, vs = s["cache"]
    dt = DTYPES[s["dtype"]]
    return ((_values(k.view(torch.uint8)[page, :, slot]) * ks[page][:, :, None]).to(dt),
            (_values(v.view(torch.uint8)[page, :, slot]) * vs[page][:, :, None]).to(dt))


def _plain_attn(s):
    k, v, ks, vs = s["cache"]
    table = s["page_table"].long().clamp(min=0)
    seqs, width = table.shape
    keys = width * s["page"]
    shape = (seqs, s["hkv"], keys, s["d"])
    kk = (_values(k.view(torch.uint8)[table]) * ks[table][..., None, None]).transpose(1, 2).reshape(shape)
    vv = (_values(v.view(torch.uint8)[table]) * vs[table][..., None, None]).transpose(1, 2).reshape(shape)
    start = s["row_start"].long()
    t = torch.arange(s["longest"], device="cuda")
    row = (start[:-1, None] + t).clamp(max=max(0, s["rows"] - 1))
    q = s["q"].float()[row].reshape(seqs, s["longest"], s["hkv"], -1, s["d"]).permute(0, 2, 1, 3, 4)
    group = q.shape[3]
    scores = q.reshape(seqs, s["hkv"], -1, s["d"]) @ kk.transpose(2, 3) / math.sqrt(s["d"])
    scores = scores.reshape(seqs, s["hkv"], s["longest"], group, keys)
    j = torch.arange(keys, device="cuda")
    seen = (j < s["held"].long()[:, None])[:, None, :]
    if s["causal"]:
        at = s["cp"] - 1 + s["cp"] * j
        seen = seen & (at <= (s["q_first"].long()[:, None] + t)[:, :, None])
    seen = seen.expand(seqs, s["longest"], keys)[:, None, :, None, :]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1)
    o = (p.reshape(seqs, s["hkv"], -1, keys) @ vv).reshape(seqs, s["hkv"], s["longest"], group, s["d"])
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    lse = top[..., 0] + torch.log(total)
    seq = torch.searchsorted(start[1:], torch.arange(s["rows"], device="cuda"), right=True)
    step = torch.arange(s["rows"], device="cuda") - start[seq]
    o = o.permute(0, 2, 1, 3, 4)[seq, step].reshape(s["rows"], -1, s["d"])
    lse = lse.permute(0, 2, 1, 3)[seq, step].reshape(s["rows"], -1)
    return o.to(DTYPES[s["out"]]), lse


def _plain_rope(s):
    half = s["rot"] // 2
    freq = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    axis = torch.repeat_interleave(torch.arange(s["axes"], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=half)
    angle = s["positions"].double()[axis].T * freq
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if s["inverse"]:
        sin = -sin
    return [_rotated(x.float(), cos, sin, half, s["interleaved"]).to(x.dtype) for x in s["x"]]


def _rotated(x, cos, sin, half, interleaved):
    rot = x[..., :2 * half]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :half], rot[..., half:])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


# ------------------------------------------------------------------ the operators
def _own(s):
    import context_blockwise_attention_gb300 as cpa

    if s["op"] == "rope":
        return cpa.rope_axes(s["x"], s["positions"], s["inv_freq"], s["sections"], interleaved=s["interleaved"],
                             inverse=s["inverse"])
    cache = cpa.KvCache(*s["cache"])
    if s["op"] == "write":
        cpa.kv_cache_write(cache, s["k"], s["v"], s["row_start"], s["held"], s["page_table"])
        return s["cache"]
    if s["op"] == "read":
        return cpa.kv_cache_read(cache, s["row_start"], s["held"], s["page_table"], s["rows"],
                                 dtype=DTYPES[s["dtype"]])
    return cpa.kv_cache_attn(s["q"], cache, s["row_start"], s["held"], s["page_table"], q_first=s["q_first"],
                             kv_pos=cpa.PosMap(s["cp"] - 1, s["cp"]), o_dtype=DTYPES[s["out"]])


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn, "rope": _plain_rope}[state["op"]](state)


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn, "rope": _exact_rope}[case["op"]](s)


def _nearest8(x):
    """The nearest e4m3 value, ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    step = ((e.long() - 1).clamp(min=-6) - 3 + 1023 << 52).view(torch.float64)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _smallest_scale(amax):
    e = MIN_EXP
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _spans(s):
    """(sequence, page, first slot, first row, rows) of every page that the call touches."""
    start, held, table = s["row_start"].tolist(), s["held"].tolist(), s["page_table"].tolist()
    for b in range(len(held)):
        row, pos = start[b], held[b]
        while row < start[b + 1]:
            n = min(s["page"] - pos % s["page"], start[b + 1] - row)
            yield b, table[b][pos // s["page"]], pos % s["page"], row, n
            row, pos = row + n, pos + n


def _exact_write(s):
    done = []
    spans = list(_spans(s))
    if len(spans) > 5000:
        return None
    for x, cache, scale in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        values, scales = cache.float().double(), scale.double().cpu()
        x = x.double()
        tops = x.abs().amax(2).cpu()
        for _, page, slot, row, n in spans:
            top = tops[row:row + n].amax(0).tolist()
            now = [_smallest_scale(a) for a in top]
            if slot:
                now = [max(a, b) for a, b in zip(now, scales[page].tolist())]
                ratio = (scales[page] / torch.tensor(now, dtype=torch.float64)).cuda()
                values[page, :, :slot] = _nearest8(values[page, :, :slot] * ratio[:, None, None])
            scales[page] = torch.tensor(now, dtype=torch.float64)
            mine = scales[page].cuda()[:, None, None]
            values[page, :, slot:slot + n] = _nearest8(x[row:row + n].transpose(0, 1) / mine)
        done.append((values, scales.cuda()))
    return done[0][0], done[1][0], done[0][1], done[1][1]


def _exact_read(s):
    out = []
    for cache, scale in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        x = torch.empty((s["rows"], s["hkv"], s["d"]), dtype=torch.float64, device="cuda")
        for _, page, slot, row, n in _spans(s):
            x[row:row + n] = (cache[page, :, slot:slot + n].float().double() * scale[page].double()[:, None, None]).transpose(0, 1)
        out.append(x)
    return out


def _exact_attn(s):
    start, held = s["row_start"].tolist(), s["held"].tolist()
    o = torch.zeros((s["rows"], s["hq"], s["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], s["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group = s["hq"] // s["hkv"]
    for b, m in enumerate(held):
        n = start[b + 1] - start[b]
        if n == 0 or m == 0:
            continue
        pages = s["page_table"][b, :-(-m // s["page"])].long()
        seen = torch.ones((n, m), dtype=torch.bool, device="cuda")
        if s["causal"]:
            key = s["cp"] * torch.arange(m, device="cuda") + s["cp"] - 1
            query = int(s["q_first"][b]) + torch.arange(n, device="cuda")
            seen = key[None, :] <= query[:, None]
        for h in range(s["hkv"]):
            k, v = ((c[:, h].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float().double() * f[pages, h].double()[:, None, None]).reshape(-1, s["d"])[:m]
                    for c, f in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
            q = s["q"][start[b]:start[b + 1], h * group:(h + 1) * group].double()
            z = torch.einsum("ngd,md->ngm", q, k) / math.sqrt(s["d"])
            z = torch.where(seen[:, None, :], z, torch.full_like(z, -math.inf))
            norm = torch.logsumexp(z, -1)
            weight = torch.where(seen[:, None, :], torch.exp(z - norm[..., None]), torch.zeros_like(z))
            o[start[b]:start[b + 1], h * group:(h + 1) * group] = torch.einsum("ngm,md->ngd", weight, v)
            lse[start[b]:start[b + 1], h * group:(h + 1) * group] = norm
    return o, lse


def _exact_rope(s):
    half, cuts = s["rot"] // 2, [0]
    for n in s["sections"]:
        cuts.append(cuts[-1] + n)
    turn = torch.empty((s["tokens"], half), dtype=torch.complex128, device="cuda")
    freq = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    for a in range(s["axes"]):
        angle = s["positions"][a].double()[:, None] * freq[cuts[a]:cuts[a + 1]]
        turn[:, cuts[a]:cuts[a + 1]] = torch.polar(torch.ones_like(angle), -angle if s["inverse"] else angle)
    out = []
    for x in s["x"]:
        y = x.double()
        lo, hi = (slice(0, s["rot"], 2), slice(1, s["rot"], 2)) if s["interleaved"] else (slice(0, half), slice(half, s["rot"]))
        z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn[:, None, :]
        y[..., lo], y[..., hi] = z.real, z.imag
        out.append(y)
    return out

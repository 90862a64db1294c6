"""Oracle: the paged 4-bit cache in float64 -- test infrastructure only.

A row of ``d`` numbers is ``d / 2`` bytes of codes (even elements in the low nibbles) and ``d / 16`` scale bytes.
Code: sign, two exponent bits (bias 1), one fraction bit.  Scale byte: five exponent bits (bias 15), three fraction
bits; the scale of a group is the byte nearest to amax / 6 (ties to the even byte), at most 226 (10240); a group with a
number that is not finite has the byte 255 and codes of 0, as codes of a group of scale 0 are.
"""

import numpy as np

from .cache import spans

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MOST = 226


def _table():
    out = np.full(256, np.nan)
    for b in range(248):
        e, f = b >> 3, b & 7
        out[b] = f / 8 * 2.0 ** -14 if e == 0 else (1 + f / 8) * 2.0 ** (e - 15)
    return out


SCALE = _table()


def _nearest(x, grid):
    """Index of the nearest number of an increasing grid to x >= 0; ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def encode(x):
    """Rows of bytes [..., d * 9 / 16] of x [..., d]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, 16)
    fine = np.isfinite(g).all(-1)
    a = np.where(fine[..., None], np.abs(np.where(np.isfinite(g), g, 0.0)), 0.0)
    scale = np.where(fine, _nearest(a.max(-1) / 6, SCALE[:MOST + 1]), 255).astype(np.uint8)
    live = fine & (scale > 0)
    s = np.where(live, SCALE[np.where(live, scale, 1)], 1.0)
    codes = _nearest(a / s[..., None], E2M1) + np.where(np.signbit(g), 8, 0)
    codes = np.where(live[..., None], codes, 0).reshape(x.shape).astype(np.uint8)
    return np.concatenate([codes[..., 0::2] | codes[..., 1::2] << 4, scale], -1)


def decode(rows):
    """Numbers of rows of bytes."""
    d = rows.shape[-1] * 16 // 9
    b = rows[..., :d // 2]
    codes = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], d)
    x = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return x * np.repeat(SCALE[rows[..., d // 2:]], 16, -1)


def cache_write(pool, x, row_start, cached, page_table):
    """Writes rows of x [rows, hkv, d] into pool [pages, hkv, P, bytes], in place."""
    for b in range(len(cached)):
        for page, slot, row, n in spans(row_start, cached, page_table, pool.shape[2], b):
            pool[page, :, slot:slot + n] = np.swapaxes(encode(x[row:row + n]), 0, 1)


def cache_tokens(pool, pages, n):
    """The first n tokens of the listed pages as float64 [n, hkv, d]."""
    if n == 0:
        return np.zeros((0, pool.shape[1], pool.shape[3] * 16 // 9))
    return np.concatenate([np.swapaxes(decode(pool[p]), 0, 1) for p in pages])[:n]


def evict(weight, n, keep, recent):
    """Slots that the tokens of a sequence had which afterwards stand in slots 0, 1, ..; weight [n] is what is gone by."""
    if n <= keep:
        return list(range(n))
    z, old = keep - recent, n - recent
    order = sorted(range(old), key=lambda i: ((1, 0.0, i) if np.isnan(weight[i]) else (0, -float(weight[i]), i)))
    stay = set(order[:z])
    behind = iter(i for i in range(z, old) if i in stay)
    return [i if i in stay else next(behind) for i in range(z)] + list(range(old, n))

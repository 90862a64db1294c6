"""Oracle: the paged 8-bit cache and rotary positions in float64 -- test infrastructure only.

Cache.  Page ``p`` and head ``h`` hold ``page_size`` tokens of ``d`` e4m3 numbers and one scale
``2^e``, ``e`` the smallest integer >= -64 with ``amax <= 448 * 2^e`` (amax over the finite values
written); the cached number is ``e4m3 * 2^e``.  Continuing a page at slot ``s > 0`` takes the larger
of the old and the new scale and rounds the slots before ``s`` again at it.

e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent 0 is subnormal (``f / 8 * 2^-6``);
0x7f and 0xff are NaN, so the largest number is 0x7e = 448; there is no infinity.
"""

import numpy as np

MIN_EXP = -64


def _table():
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[b] = (-x if b & 128 else x) if (b & 127) != 127 else np.nan
    return out


E4M3 = _table()


def e4m3_decode(b):
    return E4M3[np.asarray(b, dtype=np.uint8)]


def e4m3_encode(x):
    """Nearest e4m3 byte: ties to the even fraction, beyond 448 (infinity too) to 448, NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    grid = E4M3[:127]  # increasing
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(grid[hi] == a, hi, pick)
    out = pick + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, out).astype(np.uint8)


def scale_exponent(amax):
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def cache_write(pool, scale, x, row_start, cached, page_table):
    """Writes rows of ``x`` [rows, hkv, d] (float64) into ``pool`` (bytes [pages, hkv, P, d]) and
    ``scale`` [pages, hkv], in place, one token range of a page at a time."""
    P = pool.shape[2]
    for b in range(len(cached)):
        for page, slot, row, n in spans(row_start, cached, page_table, P, b):
            for h in range(pool.shape[1]):
                new = x[row:row + n, h]
                fin = np.abs(new[np.isfinite(new)])
                s = 2.0 ** scale_exponent(fin.max() if fin.size else 0.0)
                if slot > 0 and scale[page, h] >= s:
                    s = float(scale[page, h])
                elif slot > 0:
                    old = e4m3_decode(pool[page, h, :slot]) * (float(scale[page, h]) / s)
                    nan = np.isnan(old)
                    pool[page, h, :slot] = np.where(nan, pool[page, h, :slot] | 127, e4m3_encode(old))
                scale[page, h] = s
                pool[page, h, slot:slot + n] = e4m3_encode(new / s)


def spans(row_start, tokens, page_table, P, b):
    """(page, slot, row, count) of sequence b's rows, page by page."""
    row, token = int(row_start[b]), int(tokens[b])
    while row < row_start[b + 1]:
        n = min(P - token % P, int(row_start[b + 1]) - row)
        yield int(page_table[b][token // P]), token % P, row, n
        row, token = row + n, token + n


def cache_tokens(pool, scale, pages, n):
    """The first ``n`` tokens of the listed pages as float64 [n, hkv, d]."""
    if n == 0:
        return np.zeros((0, pool.shape[1], pool.shape[3]))
    x = np.concatenate([np.swapaxes(e4m3_decode(pool[p]) * np.asarray(scale[p], np.float64)[:, None, None], 0, 1)
                        for p in pages])
    return x[:n]


def rotate(x, positions, inv_freq, sections, interleaved=False, inverse=False):
    """Rotary positions of ``x`` [tokens, heads, d]: pair i turns by positions[axis(i)] * inv_freq[i]."""
    x = np.asarray(x, dtype=np.float64)
    half = len(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    y = x.copy()
    for i in range(half):
        w = (np.asarray(positions[axis[i]], dtype=np.longdouble) * np.longdouble(inv_freq[i])).astype(np.longdouble)
        c, s = np.cos(w).astype(np.float64)[:, None], np.sin(w).astype(np.float64)[:, None]
        if inverse:
            s = -s
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, :, ia] = x[:, :, ia] * c - x[:, :, ib] * s
        y[:, :, ib] = x[:, :, ia] * s + x[:, :, ib] * c
    return y

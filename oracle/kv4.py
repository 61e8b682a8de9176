"""The 4-bit key-value cache in plain numpy float64: its format, rows in and out, attention over it, eviction.

Written from the definitions (zl.h): a code is a sign, two bits of exponent, one of mantissa; a scale has five bits of
exponent and three of mantissa and serves 16 channels; a tile of 16 slots is the keys' codes, the values' codes, the
keys' scales, the values' scales.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every scale that is written, ascending: bits 0 .. 224 (2^13)
SCALES = np.array([m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18) for e in range(32) for m in range(8)])
WRITTEN = SCALES[:225]


def nearest(x, table):
    """Index of the entry of an ascending table nearest to x >= 0, ties to the even index, the last one for larger x."""
    x = np.minimum(x, table[-1])
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    below, above = x - table[hi - 1], table[hi] - x
    return np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)


def encode(x):
    """(codes 0 .. 15, scale bits) of [..., d] numbers; NaN is 0."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, x).reshape(*x.shape[:-1], -1, 16)
    bits = nearest(np.abs(x).max(-1) / 6, WRITTEN)
    s = WRITTEN[bits][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(x) / s, 0.0)
    codes = nearest(y, LEVELS) + 8 * ((x < 0) & (s > 0))
    return codes.reshape(*x.shape[:-2], -1).astype(np.uint8), bits.astype(np.uint8)


def decode(codes, bits):
    v = np.concatenate([LEVELS, -LEVELS])[codes].reshape(*codes.shape[:-1], -1, 16)
    return (v * SCALES[bits][..., None]).reshape(codes.shape)


def where(pages, page, b, slot):
    """(page, tile of the page, row of the tile) of a slot."""
    return pages[b, slot // page], slot % page // 16, slot % 16


def get_row(data, pages, b, h, slot):
    """(key codes, value codes, key scales, value scales) of a slot."""
    d, page = data.shape[3] // 18, data.shape[2] * 16
    p, t, r = where(pages, page, b, slot)
    tile, out = data[p, h, t], []
    for i in range(2):
        c = tile[8 * d * i + r * (d // 2): 8 * d * i + (r + 1) * (d // 2)]
        out.append(np.stack([c & 15, c >> 4], -1).reshape(-1))
    for i in range(2):
        at = 16 * d + i * d + r * (d // 16)
        out.append(tile[at:at + d // 16])
    return out


def put_row(data, pages, b, h, slot, row):
    d, page = data.shape[3] // 18, data.shape[2] * 16
    p, t, r = where(pages, page, b, slot)
    tile = data[p, h, t]
    for i in range(2):
        tile[8 * d * i + r * (d // 2): 8 * d * i + (r + 1) * (d // 2)] = row[i][0::2] + 16 * row[i][1::2]
        at = 16 * d + i * d + r * (d // 16)
        tile[at:at + d // 16] = row[2 + i]


def sequence(data, pages, b, h, length):
    """Keys and values [length, d] of a head; slots of a page that is none are NaN."""
    d, page = data.shape[3] // 18, data.shape[2] * 16
    k = np.full((length, d), np.nan)
    v = k.copy()
    for s in range(length):
        if 0 <= pages[b, s // page] < data.shape[0]:
            row = get_row(data, pages, b, h, s)
            k[s], v[s] = decode(row[0], row[2]), decode(row[1], row[3])
    return k, v


def write(data, pages, lens, starts, k, v):
    """New tokens into the last slots of their sequences, in place."""
    enc = [encode(k), encode(v)]
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            slot = lens[b] - n + i
            if slot >= 0:
                t = starts[b] + i
                for h in range(k.shape[1]):
                    put_row(data, pages, b, h, slot, (enc[0][0][t, h], enc[1][0][t, h], enc[0][1][t, h], enc[1][1][t, h]))


def attend_head(q, k, v, scale):
    """(P, O, LSE) of n queries over m slots, the last query seeing all; slots whose key is NaN are not there."""
    n, m = len(q), len(k)
    gone = np.isnan(k).any(1)
    s = q @ np.where(gone[:, None], 0.0, k).T * scale
    s[:, gone] = -np.inf
    s[np.arange(m) > m - n + np.arange(n)[:, None]] = -np.inf
    top = s.max(1, initial=-np.inf, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, top + np.log(total), -np.inf)[:, 0]
    p = e / np.where(total > 0, total, 1.0)
    return p, p @ np.where(gone[:, None], 0.0, v), lse


def keep_order(weights, positions, recent):
    """Slots in order of claim: the newest positions' first, then larger weights, then lower slots."""
    newest = max(int(x) for x in positions)
    w = [-np.inf if np.isnan(x) else float(x) for x in weights]
    low = [bool(np.isnan(x)) for x in weights]
    return sorted(range(len(w)), key=lambda i: (int(positions[i]) <= newest - recent, low[i], -w[i], i))


def evict_moves(weights, positions, keep, recent):
    """[(from, to)] of a head's slots."""
    n = len(weights)
    if n <= keep:
        return []
    kept = set(keep_order(weights, positions, recent)[:keep])
    return list(zip((s for s in range(keep, n) if s in kept), (s for s in range(keep) if s not in kept)))

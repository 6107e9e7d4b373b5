"""Oracle of the paged cache held in 4 bits — TEST INFRASTRUCTURE ONLY.

A plain transcription, in numpy, of what include/cachegen.h says of cg_quant_* and
cg_pages_slots_async.  A row is built and read number by number of its definition: the
scale is looked up among all binary16 numbers of at most 8 significant bits.
"""
from __future__ import annotations

import numpy as np

from oracle.paged_cache import BAD_PAGE, REFUSED, Cache, len_ok, row_ok


def _scales():
    x = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    m, _ = np.frexp(x)
    return np.concatenate([[0.0], x[(m * 256 == np.floor(m * 256)) & (x <= 9344)]])


SCALES = _scales()
# where channel e of the 8 of a word stands in it
SHIFT = np.array([16 * (e % 2) + 4 * (e // 2) for e in range(8)], np.uint32)


def sizes(C, d):
    """(bytes of a head's codes, groups of a head, where the scales begin, bytes of a row)"""
    groups = -(-d // 32)
    scales = C // d * groups * 16
    return 16 * groups, groups, scales, -(-(scales + 2 * (C // d) * groups) // 16) * 16


def quantise(x, d):
    """binary16 [..., C] -> (codes 1 .. 15 [..., heads, groups, 32], scales float64 [..., heads, groups])"""
    groups = -(-d // 32)
    y = np.zeros(x.shape[:-1] + (x.shape[-1] // d, groups * 32))
    y[..., :d] = x.astype(np.float64).reshape(x.shape[:-1] + (-1, d))
    y = y.reshape(y.shape[:-1] + (groups, 32))
    ok = np.isfinite(y).all(-1)
    y = np.where(ok[..., None], y, 0.0)
    a = np.abs(y).max(-1)
    s = SCALES[np.minimum(np.searchsorted(7 * SCALES, a), len(SCALES) - 1)]
    n = np.floor(y / np.where(s > 0, s, 1.0)[..., None] + 0.5)
    return (n + 8).astype(np.uint32), np.where(ok, s, np.nan)


def rows_of(x, d, rows):
    """The rows of binary16 numbers [..., C], over what `rows` (uint8 [..., row]) held before."""
    head, groups, at, row = sizes(x.shape[-1], d)
    n, s = quantise(x, d)
    words = (n.reshape(n.shape[:-3] + (-1, 8)) << SHIFT).sum(-1, dtype=np.uint32)
    out = rows.copy()
    out[..., :at] = np.ascontiguousarray(words).view(np.uint8)
    half = s.astype(np.float16).view(np.uint16)
    half[np.isnan(s)] = 0x7E00
    half = np.ascontiguousarray(half.reshape(half.shape[:-2] + (-1,)))
    out[..., at:at + 2 * half.shape[-1]] = half.view(np.uint8)
    return out


def numbers(rows, C, d):
    """What rows (uint8 [..., row]) stand for, binary16 [..., C]."""
    head, groups, at, _ = sizes(C, d)
    words = np.ascontiguousarray(rows[..., :at]).view(np.uint32)
    n = ((words[..., None] >> SHIFT) & 15).astype(np.float64) - 8
    s = np.ascontiguousarray(rows[..., at:at + 2 * (C // d) * groups]).view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        y = n.reshape(n.shape[:-2] + (-1, groups, 32)) * s.reshape(s.shape[:-1] + (-1, groups, 1))
        y = y.reshape(y.shape[:-2] + (-1,))[..., :d]
        return y.reshape(y.shape[:-2] + (C,)).astype(np.float16)


def raw(c: Cache):
    """The pools' bytes [L][N][P][row] of a cache whose rows are held as binary16 units."""
    return c.k.view(np.uint8), c.v.view(np.uint8)


def write(c: Cache, C, d, layer0, slots, k_new, v_new):
    """Returns (status, numbers held of k_new, of v_new)."""
    status, held = 0, []
    for pool, new in zip(raw(c), (k_new, v_new)):
        L = new.shape[0]
        some = rows_of(new, d, np.zeros(new.shape[:2] + (pool.shape[3],), np.uint8))
        held.append(numbers(some, C, d))
        for t, s in enumerate(slots):
            if 0 <= s < c.N * c.P:
                at = pool[layer0:layer0 + L, s // c.P, s % c.P]
                at[:] = rows_of(new[:, t], d, at)
            elif s != -1:
                status |= BAD_PAGE
    return status, held[0], held[1]


def read(c: Cache, C, d, layer0, slots, k_out, v_out):
    status = 0
    for pool, out in zip(raw(c), (k_out, v_out)):
        for t, s in enumerate(slots):
            if 0 <= s < c.N * c.P:
                out[:, t] = numbers(pool[layer0:layer0 + out.shape[0], s // c.P, s % c.P], C, d)
            elif s != -1:
                status |= BAD_PAGE
    return status


def slots(c: Cache, rows, firsts, starts, n_tokens):
    """Returns (status, slots)."""
    status, out = 0, np.full(n_tokens, -1, np.int64)
    for i, r in enumerate(rows):
        a, b, f = int(starts[i]), int(starts[i + 1]), 0 if firsts is None else int(firsts[i])
        if (not row_ok(c, r) or not len_ok(c, c.lens[r]) or not 0 <= a <= b <= n_tokens or f < 0
                or f + b - a > c.lens[r]):
            status |= REFUSED
            continue
        for t in range(a, b):
            pos = f + t - a
            p = int(c.tables[r, pos // c.P])
            if 0 <= p < c.N:
                out[t] = p * c.P + pos % c.P
            else:
                status |= BAD_PAGE
    return status, out


def held(c: Cache, C, d):
    """The same cache with the numbers that its rows stand for, for paged_cache.attention."""
    k, v = (numbers(x, C, d) for x in raw(c))
    return Cache(k, v, c.tables, c.lens, c.refs)

"""Plain fp64 oracle of the attention calls, in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  bfloat16 arrays are
``uint16`` bit patterns (see :func:`widen` and :func:`round_bf16`).

* :func:`rope` -- pair i of a head at position p turns by p * f_i.
* :func:`append` -- rows scattered into a paged cache.
* :func:`gather` -- one request's keys or values out of a paged cache.
* :func:`attend` -- softmax(scale q.k) v over the seen keys, with what the
  error bounds of a bfloat16 kernel need.
"""
from __future__ import annotations

import numpy as np


def widen(bits) -> np.ndarray:
    """bfloat16 bit patterns as float64."""
    bits = np.ascontiguousarray(bits, np.uint16)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def round_bf16(x) -> np.ndarray:
    """float64 values rounded to bfloat16 (nearest even), as float64."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def rope(x, pos, inv_freq, interleaved: bool) -> np.ndarray:
    """x [rows, heads, D] float64; pos [rows]; inv_freq [rot/2] radians."""
    y = np.array(x, np.float64)
    inv_freq = np.asarray(inv_freq, np.float64)
    half = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None, None] * inv_freq
    c, s = np.cos(a), np.sin(a)
    if interleaved:
        i0, i1 = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        i0, i1 = slice(0, half), slice(half, 2 * half)
    x0, x1 = np.array(y[..., i0]), np.array(y[..., i1])
    y[..., i0] = x0 * c - x1 * s
    y[..., i1] = x1 * c + x0 * s
    return y


def append(cache, rows, row_req, pos, block_table) -> None:
    """Scatter rows [n, heads, D] into cache [pages, slots, heads, D] in
    place; rows of no request and positions of no page are dropped."""
    pages, slots = cache.shape[:2]
    for r in range(len(rows)):
        b, p = int(row_req[r]), int(pos[r])
        if b < 0 or p // slots >= block_table.shape[1]:
            continue
        page = int(block_table[b, p // slots])
        if 0 <= page < pages:
            cache[page, p % slots] = rows[r]


def gather(cache, table_row, n: int):
    """(entries [n, heads, D] of positions 0..n-1, valid [n])."""
    pages, slots = cache.shape[:2]
    out = np.zeros((n,) + cache.shape[2:], cache.dtype)
    valid = np.zeros(n, bool)
    for p in range(n):
        if p // slots >= len(table_row):
            continue
        page = int(table_row[p // slots])
        if 0 <= page < pages:
            out[p] = cache[page, p % slots]
            valid[p] = True
    return out, valid


def attend(q, k, v, first_pos: int, scale: float, window: int = 0, valid=None):
    """Rows q [n, Hq, D] at positions first_pos + j over keys k, v
    [m, Hkv, D] at positions 0..m-1 (all float64).

    Returns (o, spread, ds): o [n, Hq, D] the outputs (0 where a row sees no
    key); spread [n, Hq, D] = sum p |v| / sum p; ds [n, Hq] the largest
    scale * sum |q_i k_i| over the seen keys."""
    n, Hq, D = q.shape
    m, Hkv = k.shape[:2]
    pos = first_pos + np.arange(n)[:, None]
    t = np.arange(m)[None, :]
    seen = t <= pos
    if window > 0:
        seen &= t > pos - window
    if valid is not None:
        seen &= valid[None, :]
    o, spread, ds = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        for j in range(n):
            s = np.nonzero(seen[j])[0]
            if len(s) == 0:
                continue
            kk, vv = k[s, kv], v[s, kv]
            x = scale * (kk @ q[j, h])
            p = np.exp(x - x.max())
            total = p.sum()
            o[j, h] = p @ vv / total
            spread[j, h] = p @ np.abs(vv) / total
            ds[j, h] = scale * (np.abs(kk) @ np.abs(q[j, h])).max()
    return o, spread, ds

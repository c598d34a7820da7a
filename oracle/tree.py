"""Plain oracle of the calls on drafted trees and on the caches' pages, in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

* :func:`walk` -- the walk that a target goes down one drafted tree.
* :func:`commit` -- an accepted path's entries move to their places.
* :func:`update_pages` -- the pages of a batch's next step, one request and
  one page after the other.
"""
from __future__ import annotations

import numpy as np


def walk(logits, parent, ids):
    """(path, tokens) of one request: logits [n, V], parent and ids [n].  No rows: ([], [])."""
    n = len(parent)
    if n == 0:
        return [], []
    path, tokens = [0], []
    while True:
        at = path[-1]
        tokens.append(int(np.argmax(logits[at])))  # the lowest id on ties
        nxt = [j for j in range(at + 1, n) if parent[j] == at and ids[j] == tokens[-1]]
        if not nxt:
            return path, tokens
        path.append(nxt[0])


def commit(cache, table_row, start: int, path) -> None:
    """Moves one request's entries in place: cache [layers, pages, slots, ...]."""
    pages, slots = cache.shape[1:3]

    def place(p):
        page = int(table_row[p // slots]) if p // slots < len(table_row) else -1
        return (page, p % slots) if 0 <= page < pages else None

    old = cache.copy()
    for j, x in enumerate(path):
        if x < 0:
            return
        src, dst = place(start + x), place(start + j)
        if x > j and src and dst:
            cache[:, dst[0], dst[1]] = old[:, src[0], src[1]]


def update_pages(table_in, parent, keep, want, page: int, num_pages: int, first=None, sinks: int = 0,
                 held=None):
    """(table_out, granted, tail_src, tail_dst, totals) as the call leaves them."""
    B, width = len(keep), table_in.shape[1]
    cap = width * page
    parent = [int(p) for p in (range(B) if parent is None else parent)]
    keep = [min(max(int(x), 0), cap) if 0 <= p < table_in.shape[0] else 0 for x, p in zip(keep, parent)]
    want = [min(max(int(w), k), cap) for w, k in zip(want, keep)]
    first = [0] * B if first is None else [max(int(x), 0) for x in first]
    held = np.zeros(num_pages, bool) if held is None else np.asarray(held) != 0
    drops = lambda b, i: (i + 1) * page <= first[b] and i * page >= sinks  # noqa: E731
    out = np.full((B, width), -1, np.int32)
    readers, writers = set(), {}
    for b in range(B):
        p = parent[b]
        for i in range(-(-keep[b] // page)):
            x = int(table_in[p, i])
            if drops(b, i) or not 0 <= x < num_pages:
                continue
            out[b, i] = x
            if (i + 1) * page > keep[b] and want[b] > keep[b]:
                writers.setdefault(x, []).append(b)
            else:
                readers.add(x)
    free = [x for x in range(num_pages) if x not in readers and x not in writers and not held[x]]
    n_free, asked = len(free), 0
    granted, src, dst = list(want), [-1] * B, [-1] * B
    for b in range(B):
        at = keep[b] // page
        if want[b] > keep[b] and keep[b] % page and not drops(b, at) and out[b, at] < 0:
            granted[b] = keep[b]  # the page that keep lies inside is missing
        for i in range(-(-want[b] // page)):
            x = int(out[b, i])
            own = x >= 0 and (i + 1) * page > keep[b] and want[b] > keep[b]
            shared = own and (x in readers or writers[x][0] != b or held[x])
            new = i * page >= keep[b] and not drops(b, i)
            if not (shared or new):
                continue
            asked += 1
            if not free:
                granted[b] = min(granted[b], max(i * page, keep[b]))
                continue
            out[b, i] = free.pop(0)
            if shared:
                src[b], dst[b] = x, out[b, i]
    i32 = lambda v: np.array(v, np.int32)  # noqa: E731
    return out, i32(granted), i32(src), i32(dst), i32([max(n_free - asked, 0), max(asked - n_free, 0)])

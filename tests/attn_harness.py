"""Inputs, calls and error bounds shared by the tests of the attention calls.

Bounds.  The kernels round a softmax weight to bfloat16 (half a step:
2^-8 relative) and normalise by the sum of the rounded weights, so a weight's
share is off by at most a factor (1 + 2^-8) / (1 - 2^-8); scores are fp32
sums of D exact products, each addition off by 2^-24 of what it adds to, so a
score is off by ds * (D + 4) * 2^-24 (ds = scale * sum |q_i k_i|; 4 more for
the scale, the maximum's subtraction and the exponential), and a share by twice
that.  With A = sum p |v| / sum p and one rounding of the output o:

    |out - o| <= 2^-8 |o| + A (2.02 * 2^-8 + 2 ds (D + 4) 2^-24 + n 2^-24)

n 2^-24 covers the fp32 sums over n keys.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import attention as oa

EPS = 2.0 ** -8


def bits(t) -> np.ndarray:
    """A bfloat16 tensor's bit patterns on the host."""
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def wide(t) -> np.ndarray:
    return oa.widen(bits(t))


def bound(o, spread, ds, n_keys: int) -> np.ndarray:
    D = o.shape[-1]
    f = 2.02 * EPS + 2 * ds[..., None] * (D + 4) * 2.0 ** -24 + n_keys * 2.0 ** -24
    return EPS * np.abs(o) * 1.0001 + spread * f + 1e-30


def assert_close(got, o, spread, ds, n_keys, what=""):
    tol = bound(o, spread, ds, n_keys)
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.nanmax(np.abs(got - o) / tol)))


def offsets(n) -> np.ndarray:
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def packed(ctx, n, rows):
    """(row_off, row_req, packed_pos) of a batch, padded to ``rows`` slots."""
    req = [b for b in range(len(n)) for _ in range(n[b])]
    pos = [ctx[b] + j for b in range(len(n)) for j in range(n[b])]
    pad = rows - len(req)
    return (offsets(n), np.array(req + [-1] * pad, np.int32), np.array(pos + [0] * pad, np.int32))


def make_cache(num_pages, page, Hkv, D, heads_first, gen, fill=None):
    """A [pages, slots, heads, D] view of a cache in either memory order."""
    shape = (num_pages, Hkv, page, D) if heads_first else (num_pages, page, Hkv, D)
    if fill is None:
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    else:
        t = torch.full(shape, fill, device="cuda", dtype=torch.bfloat16)
    return t.transpose(1, 2) if heads_first else t


def make_table(need, num_pages, max_pages, rng, unused=-1):
    """A block table [B, max_pages]: pages in random order, ``unused`` elsewhere."""
    table = np.full((len(need), max_pages), unused, np.int32)
    order, at = rng.permutation(num_pages), 0
    for b, k in enumerate(need):
        table[b, :k] = order[at: at + k]
        at += k
    return table


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).cuda()

"""The attention half of the verify forward (oracle).  TEST INFRASTRUCTURE ONLY.

The pages leave the forward to the model; they fix what it works on: every
cached row has its position ([Forensics] 3, 3.1), the forward's slots follow
the cached rows (App. D), and a tree verifier records positions and a
visibility mask ([Walkthrough] 5.2).  Plain definitions in float64:

  tree_paths      positions and visibility of a tree's nodes, from its links;
  norm_rope       per-head root-mean-square norm and position rotation;
  cache_rows      a sequence's rows of one (layer, K/V) of a cache, in order;
  attend          softmax attention of query rows over the rows they see.
"""
from __future__ import annotations

import numpy as np

from .status import ST_BAD_STATE


def tree_paths(first_child, next_sibling, kv_len):
    """first_child, next_sibling [B, N]; kv_len [B].  Returns positions [B, N],
    see [B, N, N] bool (row i: the nodes on the path from the root to i, i
    included; none for a node that no path reaches) and status [B]."""
    fc, ns = np.asarray(first_child), np.asarray(next_sibling)
    B, N = fc.shape
    pos = np.zeros((B, N), np.int32)
    see = np.zeros((B, N, N), bool)
    status = np.zeros(B, np.int32)
    for b in range(B):
        pos[b] = kv_len[b]
        links = [(i, int(x[b, i])) for i in range(N) for x in (fc, ns) if x[b, i] != -1]
        to = [c for _, c in links]
        wrong = any(not i < c < N for i, c in links) or len(set(to)) < len(to)
        if wrong or kv_len[b] < 0:
            status[b] = ST_BAD_STATE
        if wrong:
            continue
        paths = {0: [0]}
        for i in range(N):
            if i not in paths:
                continue
            c = int(fc[b, i])
            while c != -1:
                paths[c] = paths[i] + [c]
                c = int(ns[b, c])
        for i, path in paths.items():
            see[b, i, path] = True
            pos[b, i] = kv_len[b] + len(path) - 1
    return pos, see, status


def mask_words(see) -> np.ndarray:
    """Visibility [..., N] as bit words [..., ceil(N / 32)] (uint32)."""
    N = see.shape[-1]
    out = np.zeros(see.shape[:-1] + ((N + 31) // 32,), np.uint32)
    for j in range(N):
        out[..., j // 32] |= (see[..., j].astype(np.uint32) << np.uint32(j % 32))
    return out


def norm_rope(x, weight, eps: float, positions, inv_freq, interleaved: bool = False) -> np.ndarray:
    """x [T, heads, D]; weight [D] or None; positions [T]; inv_freq [rot / 2]."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out = y.copy()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = (np.asarray(positions, np.float64) * float(inv_freq[i]))[:, None]
        out[..., a] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t)
        out[..., b] = y[..., b] * np.cos(t) + y[..., a] * np.sin(t)
    return out


def row_places(b: int, rows: int, n: int, E=None, table=None, page: int = 0):
    """(plane, column) of each of the first `rows` rows of sequence b, which has
    n cached rows: in the left-padded rectangle that ends at column E, or in
    pages."""
    if table is None:
        return [(b, E - n + r) for r in range(rows)]
    return [(int(table[b][r // page]), r % page) for r in range(rows)]


def cache_rows(planes, places) -> np.ndarray:
    """planes [planes, H, cols, D] -> [H, rows, D]."""
    return np.stack([planes[p, :, c, :] for p, c in places], axis=1)


def attend(q, k, v, see, scale: float):
    """q [R, D], k and v [C, D], see [R, C] bool -> out [R, D], lse [R].  Rows
    that are not seen take no part, whatever they hold; a row that sees
    nothing, or only scores of -inf, gives zeros and -inf."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    out = np.zeros((q.shape[0], v.shape[1]))
    lse = np.full(q.shape[0], -np.inf)
    for r in range(q.shape[0]):
        at = np.nonzero(see[r])[0]
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (k[at] @ q[r])
            m = s.max(initial=-np.inf)
            if m == -np.inf:
                continue
            w = np.exp(s - m)
            out[r] = w @ v[at] / w.sum()
            lse[r] = m + np.log(w.sum())
    return out, lse

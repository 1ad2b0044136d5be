"""Inputs, oracle runs and tolerances of the attention tests."""
import numpy as np
import torch

import oracle
from tests._gpu import DEV, i32

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}     # half a step of a stored value, relative
EPS32 = 2.0 ** -24


def f64(t) -> np.ndarray:
    return t.detach().to("cpu").double().numpy()


def randn(rng, dt, *shape, sd=1.0):
    """A host tensor of dt."""
    return torch.from_numpy((rng.standard_normal(shape) * sd).astype(np.float32)).to(TDT[dt])


class Cache:
    """One call's cache on the host: L layers, every cell NaN but the rows that
    sequences hold; rows [0, rows_b) of sequence b, which has n_b rows before E
    (rectangle) or in its pages (page > 0, shuffled, with spare pages)."""

    def __init__(self, rng, dt, L, H, D, rows, n, page=0, spare=3, slack=2):
        rows, n = np.asarray(rows, np.int64), np.asarray(n, np.int64)
        B = len(rows)
        self.dt, self.L, self.H, self.D, self.rows, self.n, self.page, self.B = dt, L, H, D, rows, n, page, B
        if page:
            per = (rows + page - 1) // page
            order = rng.permutation(int(per.sum()) + spare)
            self.table = np.full((B, max(1, int(per.max()))), -5, np.int32)   # unused entries: no page
            at = 0
            for b in range(B):
                self.table[b, :per[b]] = order[at:at + per[b]]
                at += int(per[b])
            self.E, planes, cols = None, len(order), page
        else:
            self.table, self.E, planes = None, int(n.max()) + slack, B
            cols = self.E + int((rows - n).max()) + slack
        self.kv = torch.full((L, 2, planes, H, cols, D), float("nan"), dtype=TDT[dt])
        self.places = [oracle.row_places(b, int(rows[b]), int(n[b]), self.E, self.table, page) for b in range(B)]
        for b in range(B):
            for p, c in self.places[b]:
                self.kv[:, :, p, :, c] = randn(rng, dt, L, 2, H, D)

    def where(self):
        """The device argument after the layer: end_col, or the block table."""
        return i32(self.table) if self.page else i32([self.E])

    def max_rows(self):
        return self.table.shape[1] * self.page if self.page else self.kv.shape[4]

    def layer_rows(self, layer, b):
        """K and V rows of sequence b, [H, rows, D] each, in float64."""
        return [oracle.cache_rows(f64(self.kv[layer, j]), self.places[b]) for j in (0, 1)]


def attend_all(q, cache, layer, tokens, see, scale):
    """q host tensor [sum tokens, H * G, D]; see[b] [tokens_b, rows_b] bool.
    Returns out and lse in float64 and the tolerances of both.

    Tolerance.  With P_j = exp(s_j - m) / sum and A = sum_j P_j |v_j|:
    a float32 score is off by ds = (D + 4) 2^-24 scale max sum |q k| at most (a
    sum of D exact or once-rounded products, then a scaling and a subtraction
    of the size of the scores), which moves every P by 2 ds relatively; sums
    over C rows add (C + 16) 2^-24 A; P rounded to bf16 for the matrix product
    adds half a bf16 step of A; the stored result half a step of itself."""
    H, D = cache.H, cache.D
    G = q.shape[1] // H
    q64 = f64(q)
    out, lse = np.zeros(q64.shape), np.zeros(q64.shape[:2])
    tol, tol_l = np.zeros(q64.shape), np.zeros(q64.shape[:2])
    t0 = 0
    for b, len_b in enumerate(tokens):
        if not len_b:
            continue
        k, v = cache.layer_rows(layer, b)
        for h in range(H):
            seen_any = see[b].any(0)
            C = int(seen_any.sum())
            for g in range(G):
                at = (slice(t0, t0 + len_b), h * G + g)
                qh = q64[at]
                out[at], lse[at] = oracle.attend(qh, k[h], v[h], see[b], scale)
                size, _ = oracle.attend(qh, k[h], np.abs(v[h]), see[b], scale)
                big = (np.abs(qh) @ np.abs(np.nan_to_num(k[h][seen_any], posinf=0, neginf=0)).T).max(initial=0.0)
                ds = (D + 4) * EPS32 * scale * big
                rel = 2 * ds + (C + 16) * EPS32 + (HALF["bf16"] if cache.dt == "bf16" else 0.0)
                tol[at] = rel * size + 1.01 * HALF[cache.dt] * np.abs(out[at]) + 1e-30
                tol_l[at] = ds + (C + 16) * EPS32 + 4 * EPS32 * np.abs(np.nan_to_num(lse[at], neginf=0)) + 1e-30
        t0 += len_b
    return out, lse, tol, tol_l


def assert_within(got, want, tol, what=""):
    got = f64(got) if torch.is_tensor(got) else np.asarray(got, np.float64)
    got = got.reshape(want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    over = np.abs(got[fine] - want[fine]) - tol[fine]
    assert (over <= 0).all(), f"{what}: worst excess {over.max()}"


def dev(t):
    return t.to(DEV)

"""A cache of 4-bit numbers on the host, for the tests of its calls."""
import numpy as np
import torch

import oracle
from oracle import mx
from tests._gpu import DEV, i32


class MxCache:
    """As tests._attn.Cache: every cell that no sequence's row uses holds random
    codes under a scale that stands for NaN; rows hold codes of normal numbers."""

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
        self.codes = rng.integers(0, 256, (L, 2, planes, H, cols, D // 2)).astype(np.uint8)
        self.scales = rng.integers(253, 256, (L, 2, planes, H, cols, D // 32)).astype(np.uint8)
        self.places = [oracle.row_places(b, int(rows[b]), int(n[b]), self.E, self.table, page) for b in range(B)]
        for b in range(B):
            for p, c in self.places[b]:
                x = rng.standard_normal((L, 2, H, D))
                self.codes[:, :, p, :, c], self.scales[:, :, p, :, c] = mx.pack(x)

    def where(self):
        """The device argument after the layer: end_col, or the block table."""
        return i32(self.table) if self.page else i32([self.E])

    def max_rows(self):
        return self.table.shape[1] * self.page if self.page else self.codes.shape[4]

    def layer_rows(self, layer, b):
        """K and V rows of sequence b, [H, rows, D] each, in float64."""
        at = [np.array([pc[i] for pc in self.places[b]], int) for i in (0, 1)]
        return [np.moveaxis(mx.unpack(self.codes[layer, j][at[0], :, at[1]], self.scales[layer, j][at[0], :, at[1]]),
                            0, 1) for j in (0, 1)]

    def on_device(self):
        return torch.from_numpy(self.codes).to(DEV), torch.from_numpy(self.scales).to(DEV)


def as_bf16(x):
    """Codes or scales as the calls that move rows take them."""
    return x.view(torch.bfloat16)

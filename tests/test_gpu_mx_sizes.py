"""Attention over caches of 4-bit numbers whose queries are small or large and whose keys
make up for it, and with values of any size: results do not depend on where in the range
of float32 the operands lie."""
import numpy as np
import pytest

from tests import test_gpu_mx_attention as base

pytestmark = base.pytestmark


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("keys,values", [(100, 0), (118, 110), (-100, 0), (-118, 60)])
@pytest.mark.parametrize("n,N,H,G,D", [([70, 3], 1, 2, 4, 128), ([40], 5, 1, 7, 64), ([33, 90], 9, 1, 3, 256), ([60], 3, 1, 12, 192),
                                       ([100], 40, 1, 3, 128)])
def test_small_queries_and_large_keys(dt, keys, values, n, N, H, G, D):
    def spoil(cache, see):
        for b in range(cache.B):
            for p, c in cache.places[b]:
                for j, by in ((0, keys), (1, values)):
                    cache.scales[:, j, p, :, c] = np.clip(cache.scales[:, j, p, :, c].astype(int) + by, 2, 252)
    base._check(abs(keys) + N, dt, n, N, H, G, D, 0, "tree", sd=2.0 ** -keys, spoil=spoil)

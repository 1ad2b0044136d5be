"""Attention over caches of 4-bit numbers whose queries are small or large and whose keys
make up for it, and with values of any size: results do not depend on where in the range
of float32 the operands lie."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_04_amd as sv
from oracle import mx
from tests import test_gpu_mx_attention as base
from tests._attn import TDT, f64
from tests._gpu import DEV, i32, note

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


@pytest.mark.parametrize("byte", [0, 1, 2])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_smallest_scales_are_exact(byte, dt):
    """Under byte 1 (and 0, which counts as 1) code 0.5 is 2^-127, below the smallest normal number: readers
    hold it all the same."""
    note(f"mx smallest scales {byte} {dt}")
    codes = torch.zeros(1, 2, 1, 1, 1, 32, dtype=torch.uint8)
    codes[..., :16] = torch.arange(16, dtype=torch.uint8)
    scales = torch.full((1, 2, 1, 1, 1, 2), byte, dtype=torch.uint8)
    want = mx.unpack(codes.numpy(), scales.numpy())[0, 0, 0, 0, 0]
    k, v = (torch.empty(1, 1, 64, dtype=TDT[dt], device=DEV) for _ in range(2))
    sv.spec_unpack_kv_mx(codes.to(DEV), scales.to(DEV), 0, i32([0]), i32([0]), k, v)
    torch.cuda.synchronize()
    assert np.array_equal(f64(k)[0, 0], want) and np.array_equal(f64(v)[0, 0], want)
    assert np.array_equal(np.signbit(f64(k)[0, 0]), np.signbit(want))
    # one row, and a query of 2^126 at its first element: the lse is their product, exactly
    for G in (1, 40, 70):
        for code in range(16):
            one = torch.zeros_like(codes)
            one[0, 0, ..., 0] = code
            q = torch.zeros(1, 1, G, 64, dtype=TDT[dt], device=DEV)
            q[..., 0] = 2.0 ** 126
            out, lse = torch.empty_like(q), torch.empty(1, 1, G, device=DEV)
            need = sv.spec_tree_attention_mx_workspace_bytes(1, 1, 1, G, 64, 1, sv.SPEC_BF16 if dt == "bf16" else sv.SPEC_F32)
            sv.spec_tree_attention_mx(q, one.to(DEV), scales.to(DEV), 0, i32([0]), i32([0]), out, sv.workspace(need, DEV),
                                      scale=1.0, lse=lse)
            assert f64(lse).tolist() == [[[want[2 * code] * 2.0 ** 126] * G]], (G, code)

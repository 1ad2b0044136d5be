"""Queries that hold NaNs of any payload, over caches of 4-bit numbers."""
import pytest
import torch

import speculative_decoding_verification_04_amd as sv
from tests._attn import TDT
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

NANS = {"f32": [0x7f800001, 0x7f80ffff, 0x7fc00000, 0x7f810000, 0x7fffffff], "bf16": [0x7f81, 0x7fc0, 0x7fff]}


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("dt,nan,sign", [(dt, x, s) for dt in NANS for x in NANS[dt] for s in (0, 1)])
@pytest.mark.parametrize("nodes,G", [(1, 1), (3, 12), (5, 14)])
def test_a_nan_in_a_query_gives_nan(dt, nan, sign, nodes, G, D):
    """Every key holds -1 (+1 for negative payloads) where the query holds its NaN, and 0 elsewhere: taken for
    an infinity it would give scores of -inf only, and zeros."""
    note(f"mx NaN query {dt} {nan:x} sign={sign} N={nodes} G={G} D={D}")
    C, n, at = 48, 40, 37 if D == 64 else D - 3
    codes = torch.zeros(1, 2, 1, 1, C, D // 2, dtype=torch.uint8)
    codes[0, 0, :, :, :, at // 2] = (0x2 if sign else 0xA) << (4 * (at % 2))
    codes[0, 1] = 0x44                                    # values of 2
    scales = torch.full((1, 2, 1, 1, C, D // 32), 127, dtype=torch.uint8)
    q = torch.ones(1, nodes, G, D, dtype=TDT[dt])
    bits = torch.int32 if dt == "f32" else torch.int16
    width = 32 if dt == "f32" else 16
    q.view(bits)[0, 0, 0, at] = nan - (sign << (width - 1))    # as a signed whole number
    assert bool(q[0, 0, 0, at].isnan())
    out = torch.full((1, nodes, G, D), 9.0, dtype=q.dtype, device=DEV)
    lse = torch.full((1, nodes, G), 9.0, device=DEV)
    code = sv.SPEC_BF16 if dt == "bf16" else sv.SPEC_F32
    ws = sv.workspace(sv.spec_tree_attention_mx_workspace_bytes(1, nodes, 1, G, D, C, code), DEV)
    sv.spec_tree_attention_mx(q.to(DEV), codes.to(DEV), scales.to(DEV), 0, i32([n]), i32([n]), out, ws, lse=lse)
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    assert bool(out[0, 0, 0].isnan().all()) and bool(lse[0, 0, 0].isnan())
    rest = torch.ones(nodes, G, dtype=torch.bool)
    rest[0, 0] = False
    # the others' weights are all 1: their sums are exact, and the quotient and joins round a few times
    assert bool(((out[0][rest].float() - 2.0).abs() <= 2 * 16 * 2.0 ** -24).all()) and bool(lse[0][rest].isfinite().all())

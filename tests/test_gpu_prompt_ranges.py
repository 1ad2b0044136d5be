"""Packed ranges that reach past the call's tokens: the sequence's own tokens get zeros and a status, the
others are served, tokens of no sequence keep their bits."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_04_amd as sv
from tests._attn import TDT, Cache, dev, randn
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

BAD = sv.SPEC_ST_BAD_STATE


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("H,G", [(2, 2), (32, 8)])        # the larger grid exceeds the chip
@pytest.mark.parametrize("tail", [0, 70])                 # with it: more than 64 sequences
@pytest.mark.parametrize("cu,status", [
    ([0, 60, 85, 130], [0, 0, BAD]),                      # past the last token
    ([-7, 12, 40, 85], [BAD, 0, 0]),                      # before the first
    ([0, 25, 25, 2 ** 31 - 1], [0, 0, BAD]), ([-2 ** 31, 25, 50, 101], [BAD, 0, BAD]),
    ([-9, 130, 130, 140], [BAD, BAD, BAD]),               # every token is the first one's
    ([5, 100, 100, 100], [0, 0, 0])])                     # up to the last token: good; 0 .. 4 are nobody's
def test_ranges_past_the_tokens(dt, page, H, G, tail, cu, status):
    rng = np.random.default_rng(len(cu) + abs(cu[0]) % 97)
    T, D, B = 100, 64, 3 + tail
    lens = np.array([100] * B)
    cache = Cache(rng, dt, 1, H, D, lens, lens, page)
    q, kv = dev(randn(rng, dt, T, H * G, D)), dev(cache.kv)
    cu_all, end = cu + [cu[-1]] * tail, cu[-1] if cu[-1] <= T else None
    note(f"prompt ranges {dt} page={page} H={H} tail={tail} cu={cu}")
    f = sv.spec_prompt_attention_paged if page else sv.spec_prompt_attention

    def call(ranges, st):
        out = torch.full((T, H * G, D), 7.0, dtype=TDT[dt], device=DEV)
        l = torch.full((T, H * G), 7.0, device=DEV)
        f(q, kv, 0, i32(ranges), cache.where(), i32(lens), out, lse=l, status=st)
        return out, l

    st = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    out, l = call(cu_all, st)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == status + [0 if end is not None else BAD] * tail
    held = np.zeros(T, bool)
    for b in range(3):
        lo, hi = max(cu[b], 0), min(cu[b + 1], T)
        if lo >= hi:
            continue
        held[lo:hi] = True
        if status[b]:
            assert float(out[lo:hi].float().abs().max()) == 0.0 and bool((l[lo:hi] == -np.inf).all())
        else:                                             # as where every range is inside the call
            alone, al = call([lo] * (b + 1) + [hi] * (B - b), st)
            assert torch.equal(out[lo:hi], alone[lo:hi]) and torch.equal(l[lo:hi], al[lo:hi])
    free = torch.from_numpy(~held).to(DEV)
    assert bool((out[free] == 7.0).all()) and bool((l[free] == 7.0).all())
    again, _ = call(cu_all, None)                         # without a status too
    assert torch.equal(again, out)

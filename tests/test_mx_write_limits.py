"""How many tokens the write into a cache of 4-bit numbers takes at once: what passes the checks
would be launched, so these run only where no GPU is."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_04_amd as sv

try:
    LIB = sv.library()
except RuntimeError:
    LIB = None

pytestmark = pytest.mark.skipif(LIB is None or torch.cuda.is_available(), reason="needs the library, and no GPU")

# fake addresses 16 TB apart, never dereferenced
FAR = [ctypes.c_void_p((i + 1) << 44) for i in range(9)]


@pytest.mark.parametrize("T,st,code", [(1 << 24, None, sv.SPEC_EHIP), ((1 << 26) - 4, None, sv.SPEC_EHIP),
                                       ((1 << 26) - 4, FAR[8], sv.SPEC_EINVAL), (1 << 26, None, sv.SPEC_EINVAL)])
@pytest.mark.parametrize("heads", [1, 30, 254])
def test_tokens_of_a_call(T, st, code, heads):
    """Four tokens a workgroup of 256 lanes, whatever their heads, and one workgroup more for the status; without
    a GPU a call that passes ends at its launch."""
    rope = (None, None, None, None, 1e-6, None, 0, 0, FAR[7], st, None)    # after kv_len
    head = (FAR[0], 64 * heads, FAR[1], 64, FAR[2], 64, FAR[3], FAR[4], sv.SPEC_BF16, 1)
    assert LIB.spec_norm_rope_kv_mx(*head, 1, 1, T, 64, 0, T, T, heads, FAR[5], FAR[6], *rope) == code
    assert LIB.spec_norm_rope_kv_mx_paged(*head, T // 4, 1, 4, 64, 0, T, 1, T, heads, FAR[5], T // 4, FAR[6], *rope) == code

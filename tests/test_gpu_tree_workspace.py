"""Where the tree attention call keeps its records in the workspace."""
import pytest
import torch

import speculative_decoding_verification_04_amd as sv
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("B,H", [(1, 1), (3, 1), (1, 5), (2, 1)])
def test_the_groups_records_are_aligned(B, H):
    """Each group's record is two 32-bit numbers that the kernels read and write as one value of 8 bytes.
    With one tile a group nothing else in the workspace is written, so the records are what changes."""
    D, n = 64, 9
    kv = torch.zeros(1, 2, B, H, 32, D, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device=DEV)
    need = sv.spec_tree_attention_workspace_bytes(B, 1, H, 1, D, 32, sv.SPEC_BF16)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device=DEV)
    note(f"tree attention workspace records B={B} H={H}")
    sv.spec_tree_attention(q, kv, 0, i32([n]), i32([n] * B), torch.empty_like(q), ws)
    torch.cuda.synchronize()
    words = ws.view(torch.int32).cpu()
    at = (words != 0x5A5A5A5A).nonzero().flatten().tolist()
    slots = B * H                                         # a slot and a piece for each group
    assert len(at) == 2 * slots and at == list(range(at[0], at[0] + 2 * slots))
    assert at[0] * 4 % 8 == 0
    assert words[at].view(slots, 2).tolist() == [[i, 1] for i in range(slots)]

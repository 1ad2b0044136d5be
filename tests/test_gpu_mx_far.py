"""Calls on caches of 4-bit numbers and the tree commit over pages where offsets pass 32 bits and where calls
are large: the same bits as in a small cache, or in several calls."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_04_amd as sv
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _normal(seed, shape, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, dtype=torch.float32, device=DEV, generator=g).to(dtype)


def _write(qkv, H, G, codes, scales, table, n, cu=None):
    D = qkv.shape[-1]
    q_out = torch.empty(qkv.shape[0], G * H, D, dtype=qkv.dtype, device=DEV)
    st = torch.full((table.shape[0],), -7, dtype=torch.int32, device=DEV)
    freq = torch.from_numpy((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)).to(DEV)
    w = _normal(3, (D,), qkv.dtype)
    sv.spec_norm_rope_kv_mx_paged(qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:], codes, scales, 0, table, n,
                                  q_out, cu_seqlens=cu, q_weight=w, k_weight=w, inv_freq=freq, status=st)
    return q_out, st


def test_offsets_past_32_bits():
    """A layer of 2^22 + 7 pages of 16 rows of 2 heads of 64: 4.3 GB of K's codes, of which the last pages are used."""
    pages, H, G, D, page, rows, N = (1 << 22) + 7, 2, 2, 64, 16, 150, 5
    per = (rows + N + page - 1) // page
    far = (torch.empty(1, 2, pages, H, page, D // 2, dtype=torch.uint8, device=DEV),
           torch.empty(1, 2, pages, H, page, D // 32, dtype=torch.uint8, device=DEV))
    near = tuple(torch.zeros(1, 2, 2 * per, H, page, x.shape[-1], dtype=torch.uint8, device=DEV) for x in far)
    tables = i32(pages - 1 - np.arange(2 * per).reshape(2, per)), i32(np.arange(2 * per).reshape(2, per))
    qkv = _normal(1, (2 * rows, (G + 2) * H, D), torch.bfloat16)
    more = _normal(2, (2 * N, (G + 2) * H, D), torch.bfloat16)
    n, cu = i32([rows, rows]), i32([0, rows, 2 * rows])
    got = []
    for (codes, scales), table in ((far, tables[0]), (near, tables[1])):
        note(f"mx far pages {codes.shape[2]}: write")
        out = [*_write(qkv, H, G, codes, scales, table, n, cu), *_write(more, H, G, codes, scales, table, n)]
        k, v = (torch.empty(2 * rows, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        note("mx far: unpack")
        sv.spec_unpack_kv_mx_paged(codes, scales, 0, table, n, k, v, cu_seqlens=cu)
        note("mx far: prompt")
        o = torch.empty_like(out[0])
        sv.spec_prompt_attention_mx_paged(out[0], codes, scales, 0, cu, table, n, o)
        note("mx far: tree")
        q = out[2].view(2, N, G * H, D)
        t = torch.empty_like(q)
        ws = torch.empty(sv.spec_tree_attention_mx_workspace_bytes(2, N, H, G, D, per * page, sv.SPEC_BF16),
                         dtype=torch.uint8, device=DEV)
        sv.spec_tree_attention_mx_paged(q, codes, scales, 0, table, n, t, ws)
        note("mx far: commit")
        path, kept = i32([[0, 2, 4, -1, -1], [0, 1, 3, 4, -1]]), i32([3, 4])
        for x in (codes, scales):
            sv.spec_compact_tree_paged(x.view(torch.bfloat16), table, n, path, kept)
        used = [x[:, :, table.long().flatten()] for x in (codes, scales)]
        rows_used = torch.cat([used[0], used[1]], -1).view(2, 2, per, H, page, -1).transpose(3, 4).flatten(2, 3)
        torch.cuda.synchronize()
        got.append([*out, k, v, o, t, rows_used[:, :, :rows + 3]])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    assert got[0][6].float().abs().sum() > 0 and got[0][7].float().abs().sum() > 0


@pytest.mark.parametrize("H,G,D,dtype,lens", [
    (1, 1, 64, torch.bfloat16, (130, 500)),              # two waves a token, four where called alone
    (1, 1, 64, torch.float32, (250, 1900)),              # one wave a token, four and two
    (16, 8, 256, torch.float32, (460, 459))])            # more bytes than the Infinity Cache holds: 271 MB
def test_a_batch_writes_what_its_sequences_write_alone(H, G, D, dtype, lens):
    page, lens = 32, np.asarray(lens)
    per = int(lens.max() + page - 1) // page
    table, cu = i32(2 * per - 1 - np.arange(2 * per).reshape(2, per)), np.array([0, lens[0], lens.sum()])
    qkv = _normal(7, (int(lens.sum()), (G + 2) * H, D), dtype)
    pools = [[torch.full((1, 2, 2 * per, H, page, w), 7, dtype=torch.uint8, device=DEV) for w in (D // 2, D // 32)]
             for _ in range(2)]
    note(f"mx batch H={H} G={G} D={D} lens={lens.tolist()}")
    q_out, st = _write(qkv, H, G, *pools[0], table, i32(lens), i32(cu))
    alone = [_write(qkv[cu[b]:cu[b + 1]], H, G, *pools[1], table[b:b + 1], i32(lens[b:b + 1]), i32([0, lens[b]]))[0]
             for b in range(2)]
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0, 0]
    assert torch.equal(q_out, torch.cat(alone))
    for a, b in zip(*pools):
        assert torch.equal(a, b) and not bool((a == 7).all())

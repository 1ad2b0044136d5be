"""Positions and visibility bits of candidate trees against the oracle: equal."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_04_amd as sv
import workloads as W
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _run(fc, ns, n):
    B, N = fc.shape
    pos = torch.full((B, N), -9, dtype=torch.int32, device=DEV)
    bits = torch.full((B, N, (N + 31) // 32), -9, dtype=torch.int32, device=DEV)
    st = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    sv.spec_tree_mask(i32(fc), i32(ns), i32(n), pos, bits, status=st)
    torch.cuda.synchronize()
    return pos.cpu().numpy(), bits.cpu().numpy().view(np.uint32), st.cpu().numpy()


def _check(fc, ns, n):
    fc, ns, n = np.asarray(fc), np.asarray(ns), np.asarray(n)
    pos, see, st = oracle.tree_paths(fc, ns, n)
    got = _run(fc, ns, n)
    for a, b in zip(got, (pos, oracle.mask_words(see), st)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("N", [1, 2, 3, 31, 32, 33, 63, 64, 65, 100, 255, 256])
def test_random_trees(N):
    rng = np.random.default_rng(N)
    B = 9
    fc, ns = np.full((B, N), -1, np.int32), np.full((B, N), -1, np.int32)
    for b in range(B):
        used = N if b % 3 else int(rng.integers(1, N + 1))
        _, fc[b, :used], ns[b, :used] = W.random_tree(rng, used, 1 + b)
    note(f"tree mask N={N}")
    _check(fc, ns, rng.integers(0, 5000, B))


def test_chain_and_star_of_256():
    fc, ns = np.full((2, 256), -1, np.int32), np.full((2, 256), -1, np.int32)
    fc[0, :-1] = np.arange(1, 256)
    fc[1, 0], ns[1, 1:-1] = 1, np.arange(2, 256)
    note("tree mask chain and star")
    _check(fc, ns, [0, 7])


def test_bad_links_and_states():
    fc = np.array([[1, 2, -1, -1], [0, -1, -1, -1], [4, -1, -1, -1], [1, -1, -1, -1], [1, 3, -1, -1],
                   [1, -1, -1, -1], [-2, -1, -1, -1], [1, 2, -1, -1]])
    ns = np.array([[-1, -1, -1, -1], [-1, -1, -1, -1], [-1, -1, -1, -1], [-1, 1, -1, -1], [-1, 2, 3, -1],
                   [2, -1, 3, -1], [-1, -1, -1, -1], [-1, -1, -1, -1]])
    # fine; to itself; past the end; backwards; two links to node 3; the root has siblings (which no path
    # reaches); below -1; negative length
    note("tree mask bad links")
    _check(fc, ns, [3, 3, 3, 3, 3, 3, 3, -1])


def test_status_is_optional_and_replay_is_equal():
    rng = np.random.default_rng(2)
    _, fc, ns = W.random_tree(rng, 40, 3)
    f, s, n = i32(fc[None]), i32(ns[None]), i32([6])
    pos = torch.empty(1, 40, dtype=torch.int32, device=DEV)
    bits = torch.empty(1, 40, 2, dtype=torch.int32, device=DEV)
    note("tree mask graph")
    sv.spec_tree_mask(f, s, n, pos, bits)
    want = pos.clone(), bits.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_tree_mask(f, s, n, pos, bits)
    for _ in range(3):
        pos.fill_(-1)
        bits.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pos, want[0]) and torch.equal(bits, want[1])

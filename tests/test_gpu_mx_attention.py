"""Attention over caches of 4-bit numbers against the oracle in float64, for
trees, chains, single tokens and prompts.  Every cell of a cache that no
sequence's rows use stands for NaN.

The tolerance is that of the caches of bf16 and float32 (tests/_attn.py): codes
times scales are exact in both types, so nothing is added to it."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_04_amd as sv
import workloads as W
from tests._attn import TDT, assert_within, attend_all, dev, randn
from tests._gpu import DEV, i32, note, requires_gpu
from tests._mx import MxCache

pytestmark = [pytest.mark.gpu, requires_gpu]


def _see(rng, kind, B, N):
    """[B, N, N] visibility among the nodes; kind: chain (no mask), tree, any."""
    if kind == "chain":
        return np.tril(np.ones((N, N), bool))[None].repeat(B, 0)
    if kind == "any":
        return rng.random((B, N, N)) < 0.3               # some rows may be empty
    see = np.zeros((B, N, N), bool)
    for b in range(B):
        _, fc, ns = W.random_tree(rng, N, 1 + b % 5)
        see[b] = oracle.tree_paths(fc[None], ns[None], [0])[1][0]
    return see


def _whole(see, n):
    """Visibility over the cached rows and the nodes; a row of no bits sees nothing."""
    return [np.concatenate([np.repeat(s.any(1)[:, None], int(x), 1), s], 1) for s, x in zip(see, n)]


def _tree(q, cache, kv, layer, n, mask, B, N, scale=None, lse=True, stream=None, ws=None, out=None, where=None):
    H, D, G = cache.H, cache.D, q.shape[-2] // cache.H
    out = torch.full((B, N, H * G, D), 7.0, dtype=q.dtype, device=DEV) if out is None else out
    l = torch.full((B, N, H * G), 7.0, device=DEV) if lse else None
    st = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    need = sv.spec_tree_attention_mx_workspace_bytes(B, N, H, G, D, cache.max_rows(),
                                                     sv.SPEC_BF16 if q.dtype == torch.bfloat16 else sv.SPEC_F32)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws
    f = sv.spec_tree_attention_mx_paged if cache.page else sv.spec_tree_attention_mx
    f(q, *kv, layer, cache.where() if where is None else where, i32(n), out, ws, mask=mask, scale=scale, lse=l, status=st,
      stream=stream)
    return out, l, st


def _check(seed, dt, n, N, H, G, D, page, kind, L=2, sd=1.0, scale=None, spoil=None, strided=False):
    rng = np.random.default_rng(seed)
    n = np.asarray(n, np.int64)
    B = len(n)
    cache = MxCache(rng, dt, L, H, D, n + N, n, page)
    see = _see(rng, kind, B, N)
    q = randn(rng, dt, B * N, H * G, D, sd=sd)
    if spoil:
        spoil(cache, see)
    layer = L - 1
    s = 1.0 / np.sqrt(D) if scale is None else scale
    want, want_l, tol, tol_l = attend_all(q, cache, layer, [N] * B, _whole(see, n), s)
    mask = None if kind == "chain" else i32(oracle.mask_words(see).view(np.int32))
    qd = dev(q).view(B, N, H * G, D)
    if strided:
        wide = torch.full((B, N, H * G + 2 * H, D), float("nan"), dtype=qd.dtype, device=DEV)
        wide[:, :, :H * G] = qd
        qd = wide[:, :, :H * G]
    note(f"mx tree attention {dt} n={n[:6].tolist()} N={N} H={H} G={G} D={D} page={page} {kind}")
    out, l, st = _tree(qd, cache, cache.on_device(), layer, n, mask, B, N, scale)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * B
    assert_within(out, want, tol, "out")
    assert_within(l, want_l, tol_l, "lse")
    return out, want


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16, 5])
@pytest.mark.parametrize("n,N,H,G,D,kind", [
    ([0], 1, 1, 1, 64, "chain"), ([1, 0, 700], 1, 2, 4, 128, "chain"), ([31, 32, 33, 63, 64, 65, 127], 1, 1, 8, 64, "chain"),
    ([300, 12], 5, 2, 7, 128, "chain"), ([40, 0, 129], 9, 4, 2, 128, "tree"), ([33, 200], 16, 2, 4, 128, "tree"),
    ([500, 31], 33, 1, 5, 64, "tree"), ([64, 10], 70, 2, 1, 64, "any"), ([150], 16, 1, 3, 256, "tree"),
    ([90, 2], 40, 1, 4, 192, "tree"), ([17], 64, 1, 8, 64, "any"), ([200, 3], 1, 3, 1, 192, "chain"),
    ([95, 130], 7, 1, 9, 256, "any"), ([77], 13, 1, 5, 128, "any"), ([64], 130, 1, 2, 128, "tree")])
def test_trees_match_the_oracle(dt, page, n, N, H, G, D, kind):
    _check(len(n) * 1000 + N, dt, n, N, H, G, D, page, kind)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_largest_tree(dt):
    _check(9, dt, [130, 0], 256, 1, 2, 64, 0, "tree", L=1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_long_caches_in_many_pieces(dt):
    _check(2, dt, [9001], 3, 1, 4, 128, 0, "chain", L=1)
    _check(3, dt, [7003, 5], 11, 1, 7, 64, 64, "tree", L=1)
    _check(4, dt, [6001], 2, 1, 2, 256, 0, "chain", L=1)
    _check(5, dt, [3000, 100, 2000, 0], 16, 2, 4, 128, 16, "tree", L=1)


def test_many_sequences():
    rng = np.random.default_rng(21)
    _check(21, "bf16", rng.integers(0, 90, 150), 2, 1, 2, 64, 0, "chain", L=1)
    _check(22, "f32", rng.integers(0, 90, 70), 3, 2, 1, 64, 8, "any", L=1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,N,G,D,page,longest", [
    (64, 5, 2, 2, 64, 16, 6500),                         # more groups than workgroups, cut
    (60, 3, 16, 4, 128, 32, 6100),                       # groups for over half of the workgroups, cut
    (70, 1, 1, 3, 128, 16, 5400),                        # more sequences than lanes
    (30, 5, 9, 4, 64, 0, 700), (90, 3, 12, 5, 128, 8, 300)])   # one launch, below and above the chip's workgroups
def test_one_long_sequence_among_many(dt, B, H, N, G, D, page, longest):
    rng = np.random.default_rng(B)
    n = rng.integers(0, 40, B)
    n[B // 3], n[B // 2] = longest, 0
    _check(B, dt, n, N, H, G, D, page, "chain", L=1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,G", [(8, 4), (11, 3), (16, 4), (13, 5), (64, 1), (65, 1)])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_around_32_and_64_query_rows(dt, N, G, D):
    _check(N * G + D, dt, [257, 30], N, 2, G, D, 0, "tree", L=1)


def test_sharp_scores_and_scales():
    _check(5, "bf16", [200, 31], 8, 2, 4, 128, 0, "tree", sd=60.0)      # scores of several hundreds
    _check(6, "f32", [200, 31], 8, 2, 4, 64, 16, "tree", sd=60.0)
    _check(7, "bf16", [100], 4, 1, 2, 64, 0, "chain", scale=1e-6)
    _check(8, "f32", [100], 4, 1, 2, 64, 0, "chain", scale=3.0)


def test_strided_queries():
    _check(11, "bf16", [70, 3], 6, 2, 2, 64, 0, "tree", strided=True)
    _check(12, "f32", [70, 3], 40, 2, 2, 128, 7, "tree", strided=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,G,D", [(6, 2, 128), (16, 4, 64), (40, 4, 128), (5, 3, 256)])
def test_rows_that_some_do_not_see_may_stand_for_nan(dt, N, G, D):
    """Node 2's K and V, one block each: whoever sees it gets NaN there, and nobody else."""
    def spoil(cache, see):
        p, c = cache.places[0][int(cache.n[0]) + 2]
        cache.scales[:, 0, p, :, c, 0] = 255
        see[0, :, 2] = False
        see[0, 4, 1] = True
    _check(31, dt, [50, 9], N, 1, G, D, 0, "any", spoil=spoil)

    def spoil_v(cache, see):
        p, c = cache.places[0][int(cache.n[0]) + 2]
        cache.scales[:, 1, p, :, c, 1] = 254
        see[0, :, 2] = False
        see[0, 3, 2] = True
    out, want = _check(32, dt, [50, 9], N, 1, G, D, 4, "any", spoil=spoil_v)
    assert np.isnan(want.reshape(2, N, G, D)[0, 3, :, 32:64]).all()
    assert np.isfinite(want.reshape(2, N, G, D)[0, 3, :, 64:]).all() and np.isfinite(want.reshape(2, N, G, D)[0, :3]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,N", [(20, 3), (300, 3), (300, 33)])
def test_a_cached_row_that_stands_for_nan_reaches_everyone(dt, n, N):
    def spoil(cache, see):
        p, c = cache.places[0][7]
        cache.scales[:, 1, p, :, c, 0] = 255
    out, want = _check(33, dt, [n], N, 1, 4, 128, 0, "chain", spoil=spoil)
    assert np.isnan(want[..., :32]).all() and np.isfinite(want[..., 32:]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_far_apart_scales(dt):
    """Rows of very large and very small numbers beside each other."""
    def spoil(cache, see):
        for r, byte in ((3, 252 - 40), (4, 2), (9, 20), (11, 1)):
            p, c = cache.places[0][r]
            cache.scales[:, 1, p, :, c] = byte
        for r, byte in ((5, 2), (6, 100), (12, 1)):
            p, c = cache.places[0][r]
            cache.scales[:, 0, p, :, c] = byte
    _check(34, dt, [40], 3, 1, 4, 128, 0, "chain", spoil=spoil)


@pytest.mark.parametrize("page", [0, 8])
@pytest.mark.parametrize("N,G", [(3, 2), (20, 4)])
def test_bad_sequences_give_zeros(page, N, G):
    rng = np.random.default_rng(41)
    n = np.array([30, 25, 60, 40])
    cache = MxCache(rng, "bf16", 1, 2, 128, n + N, n, page)
    q = dev(randn(rng, "bf16", 4, N, 2 * G, 128))
    kv = cache.on_device()
    where = cache.where()
    good, gl, _ = _tree(q, cache, kv, 0, n, None, 4, N)
    said = n.copy()
    said[1] = -4
    want = [0, 16, 0, 0]
    if page:
        table = cache.table.copy()
        table[3, 2] = cache.codes.shape[2] + 7
        where = i32(table)
        want[3] = 16
        said[2] = cache.max_rows()
        want[2] = 32
    else:
        said[2] = cache.E + 1
        want[2] = 16
    note(f"mx bad sequences page={page}")
    out, l, st = _tree(q, cache, kv, 0, said, None, 4, N, where=where)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == want
    for b in (1, 2):
        assert bool((out[b] == 0).all()) and bool((l[b] == float("-inf")).all())
    assert float((out[0].float() - good[0].float()).abs().max()) <= 2 * (4 * 2.0 ** -8 + 4 * 2.0 ** -8)
    assert bool(torch.isfinite(out).all())


def test_calls_repeat_bit_for_bit_on_streams_and_in_graphs():
    rng = np.random.default_rng(51)
    n, N = np.array([900, 40, 333]), 5
    cache = MxCache(rng, "bf16", 1, 2, 128, n + N, n, 16)
    q = dev(randn(rng, "bf16", 3, N, 8, 128))
    kv, where = cache.on_device(), cache.where()
    note("mx tree repeats")
    first, l0, _ = _tree(q, cache, kv, 0, n, None, 3, N)
    torch.cuda.synchronize()
    # two streams at once, each with its own outputs and workspace, all of them there before either starts
    need = sv.spec_tree_attention_mx_workspace_bytes(3, N, 2, 4, 128, cache.max_rows(), sv.SPEC_BF16)
    nd, side = i32(n), torch.cuda.Stream()
    outs, lses, spaces = ([make() for _ in range(2)] for make in (
        lambda: torch.empty_like(first), lambda: torch.empty_like(l0), lambda: sv.workspace(need, DEV)))
    torch.cuda.synchronize()
    for i, stream in enumerate((side, None)):
        sv.spec_tree_attention_mx_paged(q, *kv, 0, where, nd, outs[i], spaces[i], lse=lses[i], stream=stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(first, outs[i]) and torch.equal(l0, lses[i]), i
    out, ws = outs[0], spaces[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_tree_attention_mx_paged(q, *kv, 0, where, nd, out, ws)
    for lens in ([900, 40, 333], [10, 0, 300], [899, 39, 1], [900, 40, 333]):
        nd.copy_(i32(lens))
        want, _, _ = _tree(q, cache, kv, 0, np.array(lens), None, 3, N)
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,G", [(3, 2), (16, 4), (40, 4)])
def test_bad_sequences_beside_one_that_is_cut(dt, N, G):
    """A long cache in pieces: one page of it is missing, and of its neighbours one has no length, one no room."""
    rng = np.random.default_rng(43)
    n = np.array([6500, 25, 60, 40])
    cache = MxCache(rng, dt, 1, 2, 128, n + N, n, 32)
    q = randn(rng, dt, 4 * N, 2 * G, 128)
    see = _see(rng, "chain", 4, N)
    want, want_l, tol, tol_l = attend_all(q, cache, 0, [N] * 4, _whole(see, n), 1.0 / np.sqrt(128))
    kv, qd = cache.on_device(), dev(q).view(4, N, 2 * G, 128)
    said, table = n.copy(), cache.table.copy()
    said[1], said[2] = -1, cache.max_rows()
    note(f"mx bad sequences, cut {dt} N={N}")
    for page, status in ((None, 0), (150, 16)):
        if page is not None:
            table[0, page] = -1
        out, l, st = _tree(qd, cache, kv, 0, said, None, 4, N, where=i32(table))
        torch.cuda.synchronize()
        assert st.cpu().tolist() == [status, 16, 32, 0]
        for b in (1, 2):
            assert bool((out[b] == 0).all()) and bool((l[b] == float("-inf")).all())
        for b in (0, 3) if page is None else (3,):
            at = slice(b * N, (b + 1) * N)
            shape = (4 * N, 2 * G, 128)
            assert_within(out[b], want.reshape(shape)[at], tol.reshape(shape)[at], f"out {b}")
            assert_within(l[b], want_l.reshape(shape[:2])[at], tol_l.reshape(shape[:2])[at], f"lse {b}")
        assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_cut_call_repeats_on_streams_and_in_graphs(dt):
    rng = np.random.default_rng(52)
    n, N = np.array([7000, 40, 3333]), 5
    cache = MxCache(rng, dt, 1, 2, 128, n + N, n, 64)
    q = dev(randn(rng, dt, 3, N, 8, 128))
    kv, where = cache.on_device(), cache.where()
    need = sv.spec_tree_attention_mx_workspace_bytes(3, N, 2, 4, 128, cache.max_rows(),
                                                     sv.SPEC_BF16 if dt == "bf16" else sv.SPEC_F32)
    nd, side = i32(n), torch.cuda.Stream()
    note(f"mx cut tree repeats {dt}")
    first, _, _ = _tree(q, cache, kv, 0, n, None, 3, N)
    outs, spaces = ([make() for _ in range(2)] for make in (lambda: torch.empty_like(first), lambda: sv.workspace(need, DEV)))
    torch.cuda.synchronize()
    for i, stream in enumerate((side, None)):
        sv.spec_tree_attention_mx_paged(q, *kv, 0, where, nd, outs[i], spaces[i], stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(first, outs[0]) and torch.equal(first, outs[1])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]   # of one workspace, replayed one after the other
    for graph, out in zip(graphs, outs):
        with torch.cuda.graph(graph):
            sv.spec_tree_attention_mx_paged(q, *kv, 0, where, nd, out, spaces[0])
    for lens in ([7000, 40, 3333], [10, 0, 3000], [6999, 39, 1], [7000, 40, 3333]):
        nd.copy_(i32(lens))
        want, _, _ = _tree(q, cache, kv, 0, np.array(lens), None, 3, N)
        for out in outs:
            out.fill_(3.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


# ------------------------------------------------------------------- prompts ----
def _prompt(q, cache, kv, layer, cu, n, scale=None, stream=None):
    B, T, Hq = len(n), q.shape[0], q.shape[1]
    out = torch.full((T, Hq, cache.D), 7.0, dtype=q.dtype, device=DEV)
    l = torch.full((T, Hq), 7.0, device=DEV)
    st = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    f = sv.spec_prompt_attention_mx_paged if cache.page else sv.spec_prompt_attention_mx
    f(q, *kv, layer, i32(cu), cache.where(), i32(n), out, scale=scale, lse=l, status=st, stream=stream)
    return out, l, st


def _check_prompt(seed, dt, lens, H, G, D, page, before=0, L=2, sd=1.0, behind=0, spoil=None, strided=False):
    """before: cached rows in front of every prompt's; behind: tokens of no sequence."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    n = lens + before
    T = int(lens.sum())
    cache = MxCache(rng, dt, L, H, D, n, n, page)
    q = randn(rng, dt, T + behind, H * G, D, sd=sd)
    if spoil:
        spoil(cache)
    see = [np.tril(np.ones((x, x + before), bool), before) for x in lens]
    want, want_l, tol, tol_l = attend_all(q[:T], cache, L - 1, lens.tolist(), see, 1.0 / np.sqrt(D))
    qd = dev(q)
    if strided:
        wide = torch.full((T + behind, H * G + 2 * H, D), float("nan"), dtype=qd.dtype, device=DEV)
        wide[:, :H * G] = qd
        qd = wide[:, :H * G]
    note(f"mx prompt attention {dt} lens={lens[:6].tolist()} before={before} H={H} G={G} D={D} page={page}")
    out, l, st = _prompt(qd, cache, cache.on_device(), L - 1, np.concatenate([[0], np.cumsum(lens)]), n)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * len(lens)
    assert_within(out[:T], want, tol, "out")
    assert_within(l[:T], want_l, tol_l, "lse")
    assert bool((out[T:] == 7.0).all()) and bool((l[T:] == 7.0).all())
    return out, want


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16, 7])
@pytest.mark.parametrize("lens,H,G,D,before", [
    ([1], 1, 1, 64, 0), ([5, 0, 1, 33], 2, 2, 128, 0), ([64, 63, 65], 1, 4, 64, 0), ([130, 17], 2, 7, 128, 0),
    ([200], 1, 3, 192, 0), ([100, 31], 1, 1, 256, 0), ([40, 9, 1], 2, 2, 64, 77), ([129], 4, 1, 128, 300),
    ([16, 30], 1, 8, 64, 1)])
def test_prompts_match_the_oracle(dt, page, lens, H, G, D, before):
    _check_prompt(sum(lens) + D, dt, lens, H, G, D, page, before)


def test_many_prompts_and_tokens_of_no_sequence():
    rng = np.random.default_rng(3)
    _check_prompt(4, "bf16", rng.integers(0, 9, 150), 1, 2, 64, 0, behind=37)
    _check_prompt(5, "f32", rng.integers(0, 9, 70), 1, 2, 64, 4, behind=3)


def test_longer_prompts_sharp_scores_and_strides():
    _check_prompt(6, "bf16", [700, 3], 1, 2, 128, 0, L=1, strided=True)
    _check_prompt(7, "bf16", [150], 1, 2, 64, 0, sd=60.0)
    _check_prompt(8, "f32", [150], 1, 2, 64, 16, sd=60.0)
    _check_prompt(9, "bf16", [400, 390], 8, 4, 64, 16, L=1)         # tiles of 128 rows
    _check_prompt(10, "bf16", [300, 200], 8, 16, 256, 0, L=1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_prompts_row_that_stands_for_nan_reaches_its_followers(dt):
    def spoil(cache):
        for r in (20, 90):
            p, c = cache.places[0][r]
            cache.scales[:, 1, p, :, c, 1] = 255
    out, want = _check_prompt(11, dt, [120], 1, 2, 128, 0, spoil=spoil)
    assert np.isfinite(want[:20]).all() and np.isnan(want[20:, :, 32:64]).all() and np.isfinite(want[20:, :, :32]).all()


@pytest.mark.parametrize("page", [0, 4])
def test_bad_prompts_give_zeros(page):
    rng = np.random.default_rng(61)
    lens = np.array([9, 7, 12])
    cache = MxCache(rng, "bf16", 1, 1, 64, lens, lens, page)
    q = dev(randn(rng, "bf16", 28, 2, 64))
    kv = cache.on_device()
    cu = np.array([0, 9, 16, 28])
    good, _, _ = _prompt(q, cache, kv, 0, cu, lens)
    note("mx bad prompts")
    out, l, st = _prompt(q, cache, kv, 0, cu, [9, 5, 12])
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0, 16, 0]
    assert bool((out[9:16] == 0).all()) and torch.equal(out[:9], good[:9]) and torch.equal(out[16:], good[16:])
    out, l, st = _prompt(q, cache, kv, 0, [0, 9, 9, 40], lens)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0, 0, 16]
    assert bool((out[9:] == 0).all()) and torch.equal(out[:9], good[:9])

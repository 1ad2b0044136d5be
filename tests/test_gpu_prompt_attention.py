"""Causal attention of packed prompts over the cache against the oracle in
float64.  Every cell of a cache that no sequence's rows use holds NaN."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_04_amd as sv
from tests._attn import Cache, assert_within, attend_all, dev, randn
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _call(q, cache, kv, layer, cu, n, scale=None, out=None, stream=None):
    B, T, Hq = len(n), q.shape[0], q.shape[1]
    out = torch.full((T, Hq, cache.D), 7.0, dtype=q.dtype, device=DEV) if out is None else out
    l = torch.full((T, Hq), 7.0, device=DEV)
    st = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    f = sv.spec_prompt_attention_paged if cache.page else sv.spec_prompt_attention
    f(q, kv, layer, i32(cu), cache.where(), i32(n), out, scale=scale, lse=l, status=st, stream=stream)
    return out, l, st


def _check(seed, dt, lens, H, G, D, page, before=0, L=2, sd=1.0, behind=0, spoil=None, strided=False):
    """before: cached rows in front of every prompt's; behind: tokens of no sequence."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    n = lens + before
    T = int(lens.sum())
    cache = Cache(rng, dt, L, H, D, n, n, page)
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
    note(f"prompt attention {dt} lens={lens[:6].tolist()} before={before} H={H} G={G} D={D} page={page}")
    out, l, st = _call(qd, cache, dev(cache.kv), L - 1, np.concatenate([[0], np.cumsum(lens)]), n)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * len(lens)
    assert_within(out[:T], want, tol, "out")
    assert_within(l[:T], want_l, tol_l, "lse")
    assert bool((out[T:] == 7.0).all()) and bool((l[T:] == 7.0).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16, 7])
@pytest.mark.parametrize("lens,H,G,D,before", [
    ([1], 1, 1, 64, 0), ([5, 0, 1, 33], 2, 2, 128, 0), ([64, 63, 65], 1, 4, 64, 0), ([130, 17], 2, 7, 128, 0),
    ([200], 1, 3, 80, 0), ([100, 31], 1, 1, 256, 0), ([40, 9, 1], 2, 2, 64, 77), ([129], 4, 1, 96, 300),
    ([16, 30], 1, 8, 8, 1)])
def test_matches_oracle(dt, page, lens, H, G, D, before):
    if dt == "f32" and D == 8:
        D = 4
    _check(sum(lens) + D, dt, lens, H, G, D, page, before)


def test_many_prompts_and_tokens_of_no_sequence():
    rng = np.random.default_rng(3)
    _check(4, "bf16", rng.integers(0, 9, 150), 1, 2, 64, 0, behind=37)
    _check(5, "f32", rng.integers(0, 9, 70), 1, 2, 64, 4, behind=3)


def test_longer_prompt_sharp_scores_and_strides():
    _check(6, "bf16", [700, 3], 1, 2, 128, 0, L=1, strided=True)
    _check(7, "bf16", [150], 1, 2, 64, 0, sd=60.0)
    _check(8, "f32", [150], 1, 2, 64, 16, sd=60.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16])
def test_infinities_and_nans_reach_only_later_tokens(dt, page):
    def spoil(cache):
        p, c = cache.places[0][90]
        cache.kv[:, 1, p, :, c, 1::3] = np.inf
        p, c = cache.places[0][100]
        cache.kv[:, :, p, :, c] = np.nan
        p, c = cache.places[1][0]
        cache.kv[:, 1, p, :, c, 2] = -np.inf
    _check(9, dt, [140, 20], 2, 2, 64, page, spoil=spoil)


def test_states_out_of_range():
    rng = np.random.default_rng(11)
    lens = np.array([9, 20, 5])
    cache = Cache(rng, "bf16", 1, 2, 64, lens, lens)
    q, kv = dev(randn(rng, "bf16", 40, 4, 64)), dev(cache.kv)
    cu = [0, 9, 29, 34]
    note("prompt attention bad states")
    good, _, _ = _call(q, cache, kv, 0, cu, lens)
    out, l, st = _call(q, cache, kv, 0, cu, [9, 19, 5])                    # fewer rows than tokens
    assert st.cpu().tolist() == [0, sv.SPEC_ST_BAD_STATE, 0]
    assert torch.equal(out[:9], good[:9]) and torch.equal(out[29:34], good[29:34])
    assert float(out[9:29].float().abs().max()) == 0.0 and bool((l[9:29] == -np.inf).all())
    out, _, st = _call(q, cache, kv, 0, cu, [9, cache.E + 1, 5])
    assert st.cpu().tolist() == [0, sv.SPEC_ST_BAD_STATE, 0]
    out, _, st = _call(q, cache, kv, 0, [0, 9, 4, 41], lens)               # backwards, and past T
    assert st.cpu().tolist() == [0, sv.SPEC_ST_BAD_STATE, sv.SPEC_ST_BAD_STATE]
    assert torch.equal(out[:9], good[:9]) and bool((out[9:] == 7.0).all())
    cache.E = cache.kv.shape[4] + 1
    _, _, st = _call(q, cache, kv, 0, cu, lens)
    assert st.cpu().tolist() == [sv.SPEC_ST_CAPACITY] * 3
    paged = Cache(rng, "bf16", 1, 2, 64, lens, lens, 4)
    kvp = dev(paged.kv)
    good, _, _ = _call(q, paged, kvp, 0, cu, lens)
    paged.table[1, 2] = -3
    out, _, st = _call(q, paged, kvp, 0, cu, [9, 20, paged.max_rows() + 1])
    assert st.cpu().tolist() == [0, sv.SPEC_ST_BAD_STATE, sv.SPEC_ST_CAPACITY]
    assert torch.equal(out[:9], good[:9]) and float(out[29:34].float().abs().max()) == 0.0


def test_offsets_past_32_bits():
    rng = np.random.default_rng(12)
    H, D, page = 4, 128, 64
    small = Cache(rng, "bf16", 1, H, D, [150], [150], page)
    q = dev(randn(rng, "bf16", 150, H * 2, D))
    note("prompt attention far pages")
    want, _, _ = _call(q, small, dev(small.kv), 0, [0, 150], [150])
    pages = (5 << 30) // (H * page * D * 2) + 8
    pool = torch.zeros(1, 2, pages, H, page, D, dtype=torch.bfloat16, device=DEV)
    far = np.array([[pages - 1, 3, pages - 2, 0]], np.int32)[:, :small.table.shape[1]]
    for i in range(far.shape[1]):
        pool[0, :, int(far[0, i])] = dev(small.kv)[0, :, int(small.table[0, i])]
    small.table = far
    got, _, _ = _call(q, small, pool, 0, [0, 150], [150])
    assert torch.equal(got, want)


def test_graph_replay_and_side_stream():
    rng = np.random.default_rng(13)
    lens = np.array([70, 200])
    c = Cache(rng, "bf16", 1, 2, 64, lens, lens, 16)
    q, kv, cu, t, n = dev(randn(rng, "bf16", 270, 4, 64)), dev(c.kv), i32([0, 70, 270]), c.where(), i32(lens)
    out = torch.empty(270, 4, 64, dtype=torch.bfloat16, device=DEV)
    call = lambda s=None: sv.spec_prompt_attention_paged(q, kv, 0, cu, t, n, out, stream=s)  # noqa: E731
    note("prompt attention graph")
    call()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("H,G,tail", [(2, 2, 0), (32, 8, 0), (2, 2, 70)])
def test_ranges_that_fall_have_no_tokens(H, G, tail):
    """From where cu_seqlens falls on, ranges would hold other sequences' tokens: no sequence there has any,
    and those before it are served.  With 32 heads the grid exceeds the chip; tail: more than 64 sequences."""
    rng = np.random.default_rng(14)
    lens = np.array([60, 0, 5, 90] + [1] * tail)
    cache = Cache(rng, "bf16", 1, H, 64, lens, lens)
    q, kv = dev(randn(rng, "bf16", 150, H * G, 64)), dev(cache.kv)
    note(f"prompt attention falling ranges H={H} tail={tail}")
    good, _, st = _call(q, cache, kv, 0, [0, 60, 60, 65, 65] + [65] * tail, [60, 0, 5, 90] + [1] * tail)
    assert st.cpu().tolist() == [0] * (4 + tail)
    out, l, st = _call(q, cache, kv, 0, [0, 60, 30, 35, 125] + [125] * tail, lens)
    bad = sv.SPEC_ST_BAD_STATE
    assert st.cpu().tolist() == [0] + [bad] * (3 + tail)
    assert torch.equal(out[:60], good[:60]) and bool((out[60:] == 7.0).all()) and bool((l[60:] == 7.0).all())
    # all of the tokens twice: no workgroup is missing
    out, _, st = _call(q, cache, kv, 0, [0, 60, 60, 0, 60] + [60] * tail, lens)
    assert st.cpu().tolist() == [0, 0] + [bad] * (2 + tail)
    assert torch.equal(out[:60], good[:60]) and bool((out[60:] == 7.0).all())


def test_equal_and_empty_prompts_in_a_grid_past_the_chip():
    """Many sequences of equal and of no length, in a grid that exceeds the chip."""
    _check(15, "bf16", [130, 0, 130, 64, 1, 0, 130], 16, 8, 64, 16)


def test_two_graphs_and_two_streams_on_the_rectangle():
    rng = np.random.default_rng(16)
    lens = np.array([33, 150])
    c = Cache(rng, "f32", 2, 2, 128, lens, lens)
    kv, cu, E, n = dev(c.kv), i32([0, 33, 183]), c.where(), i32(lens)
    qs = [dev(randn(rng, "f32", 183, 6, 128)) for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    call = lambda i, s=None: sv.spec_prompt_attention(qs[i], kv, i, cu, E, n, outs[i], stream=s)  # noqa: E731
    note("prompt attention two graphs")
    for i in (0, 1):
        call(i)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for i in (0, 1):
        call(i, sides[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        call(rep % 2)

"""Writing rows into a cache of 4-bit numbers and reading them back, against the
oracle in float64; every byte that a call does not own keeps its value."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_04_amd as sv
from oracle import mx
from tests._attn import EPS32, HALF, TDT, assert_within, dev, f64, randn
from tests._gpu import DEV, i32, note, requires_gpu
from tests._mx import MxCache

pytestmark = [pytest.mark.gpu, requires_gpu]

# Keys are computed in float64 here and there: D squares, a root, an angle's sine and cosine and three
# products are off by (D + 32) 2^-53 of the head's largest element at most, which can be 2^10 times a
# small element.  Within 2^-36 of a border either side of it is right.
BORDER = 2.0 ** -36


def _freq(half):
    return (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def _same_codes(codes, scales, x, what):
    """Bytes [..., D / 2], [..., D / 32] are x's [..., D], but where x is next to a border."""
    want_c, want_s = mx.pack(x)
    differ = (mx.unpack(codes, scales) != mx.unpack(want_c, want_s))
    differ &= ~(np.isnan(mx.unpack(codes, scales)) & np.isnan(mx.unpack(want_c, want_s)))
    if differ.any():
        near = mx.border_distance(x).reshape(-1, 32).min(-1) < BORDER
        assert np.repeat(near, 32).reshape(differ.shape)[differ].all(), what
    else:
        assert np.array_equal(scales, want_s), what


def _case(seed, dt, H, G, D, lens, new, page, rot, near=False, norm=True, packed=False, positions=None, L=2, fused=True,
          eps=1e-5, spoil=None, stream=None):
    """lens: cached rows (packed: rows with the prompt); new: tokens per sequence."""
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    B, T = len(lens), int(new.sum())
    rows = lens if packed else lens + new
    cache = MxCache(rng, dt, L, H, D, rows, lens, page)
    layer = L - 1
    seq = np.repeat(np.arange(B), new)
    row = np.concatenate([rows[b] - new[b] + np.arange(new[b]) for b in range(B)]).astype(np.int64)
    qkv = randn(rng, dt, T, (G + 2) * H, D, sd=3.0)
    if spoil:
        spoil(qkv)
    wq, wk = (randn(rng, dt, D), randn(rng, dt, D)) if norm else (None, None)
    freq = _freq(rot // 2)
    at = row if positions is None else positions[:T]
    d = dev(qkv)
    q, k, v = d[:, :G * H], d[:, G * H:(G + 1) * H], d[:, (G + 1) * H:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    codes, scales = cache.on_device()
    q_out = torch.full((T, G * H, D), 9.0, dtype=qkv.dtype, device=DEV)
    st = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    cu = i32(np.concatenate([[0], np.cumsum(new)])) if packed else None
    where, n = cache.where(), i32(lens)
    note(f"mx rows {dt} H={H} G={G} D={D} lens={lens[:5].tolist()} new={new[:5].tolist()} page={page} rot={rot}")
    f = sv.spec_norm_rope_kv_mx_paged if page else sv.spec_norm_rope_kv_mx
    f(q, k, v, codes, scales, layer, where, n, q_out, cu_seqlens=cu,
      positions=None if positions is None else i32(positions[:T]), eps=eps, interleaved=near, status=st,
      q_weight=None if wq is None else dev(wq), k_weight=None if wk is None else dev(wk),
      inv_freq=torch.from_numpy(freq).to(DEV) if rot else None)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * B
    x = f64(qkv)
    # queries: as in spec_norm_rope_kv's tests
    want = oracle.norm_rope(x[:, :G * H], None if wq is None else f64(wq), eps, at, freq, near)
    size = np.abs(oracle.norm_rope(x[:, :G * H], None if wq is None else f64(wq), eps, at, freq[:0], near)).max(-1, keepdims=True)
    assert_within(q_out, want, (D + 32) * EPS32 * size + 1.01 * HALF[dt] * np.abs(want), "q")
    keys = oracle.norm_rope(x[:, G * H:(G + 1) * H], None if wk is None else f64(wk), eps, at, freq, near)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    plane, col = (np.array([cache.places[b][r][i] for b, r in zip(seq, row)], int) for i in (0, 1))
    for i, y in ((0, keys), (1, x[:, (G + 1) * H:])):
        _same_codes(c[layer, i][plane, :, col], s[layer, i][plane, :, col], y, "kv"[i])
    # nothing else has changed
    for got, had in ((c, cache.codes), (s, cache.scales)):
        expect = had.copy()
        expect[layer][:, plane, :, col] = got[layer][:, plane, :, col]
        assert np.array_equal(expect, got)
    # and the rows come back as their values
    k_out, v_out = (torch.full((T, H, D), 9.0, dtype=qkv.dtype, device=DEV) for _ in range(2))
    st.fill_(-7)
    f = sv.spec_unpack_kv_mx_paged if page else sv.spec_unpack_kv_mx
    f(codes, scales, layer, where, n, k_out, v_out, cu_seqlens=cu, status=st)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * B
    for i, got in ((0, k_out), (1, v_out)):
        assert np.array_equal(f64(got), mx.unpack(c[layer, i][plane, :, col], s[layer, i][plane, :, col]), equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,D,rot", [(1, 1, 64, 64), (2, 3, 64, 32), (8, 4, 128, 128), (2, 7, 128, 96), (2, 2, 192, 96),
                                       (1, 8, 256, 256), (3, 1, 128, 22), (4, 2, 64, 0), (2, 2, 192, 128), (5, 1, 256, 64)])
def test_slots_of_the_verify_forward(dt, H, G, D, rot):
    for page in (0, 7):
        _case(D + G, dt, H, G, D, [0, 5, 33], [3, 3, 3], page, rot)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 40), (192, 22), (256, 128)])
def test_neighbouring_pairs(dt, D, rot):
    _case(D, dt, 2, 2, D, [4, 1], [5, 5], 4, rot, near=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16])
def test_packed_prompts(dt, page):
    # a whole prompt, one of no tokens, one token, a chunk behind cached rows
    _case(3, dt, 2, 4, 128, [50, 9, 1, 40], [50, 0, 1, 13], page, 128, packed=True)


def test_many_sequences_are_found():
    rng = np.random.default_rng(5)
    new = rng.integers(0, 4, 200)
    _case(4, "bf16", 1, 1, 64, new + rng.integers(0, 3, 200) + (new == 0), new, 0, 64, packed=True)


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_far_positions(fused, norm):
    pos = np.array([0, 1, 1 << 20, (1 << 20) + 1, 2 ** 31 - 1, 12345, 7, 8])
    _case(6, "f32", 2, 2, 64, [3, 9], [4, 4], 0, 64, norm=norm, positions=pos, fused=fused)


def test_one_token():
    _case(7, "bf16", 8, 4, 128, [900], [1], 0, 128)
    _case(8, "f32", 1, 1, 64, [0], [1], 1, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_values_on_borders_and_at_the_ends_of_the_range(dt):
    """Without norm and rotation the inputs are what is packed: ties of codes and of scales, powers of two,
    zeros, the largest and smallest numbers."""
    tiny = [2.0 ** -120, 2.0 ** -124, 2.0 ** -125, 2.0 ** -126, 1.5 * 2.0 ** -126]
    heads = [[6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5], [7, .5, 1.5, 2.5, 3.5, 5, 6.96875, 7], [3.5, 3.484375, .125],
             [1.75, 1.7421875, -1.75], [2.0 ** 127, 1.5 * 2.0 ** 127, -1.75 * 2.0 ** 127, 2.0 ** 124],
             [3.38e38, -3.38e38, 1e38], tiny, [-0.0, 0.0], [-1, 2, -4, 8, -16, 32], [2.0 ** -127 * 3, 2.0 ** -130]]

    def spoil(qkv):
        for j, head in enumerate(heads):
            for kv in (2, 3):
                x = torch.zeros(64)
                x[:len(head)] = torch.tensor(head, dtype=torch.float64).float()
                x[40:40 + len(head)] = -x[:len(head)]
                qkv[j, kv] = x.to(qkv.dtype)
    _case(9, dt, 1, 2, 64, [2, 0], [5, 5], 0, 0, norm=False, spoil=spoil)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_blocks_that_are_not_finite(dt):
    def spoil(qkv):
        qkv[0, 2, 3] = float("inf")
        qkv[1, 2, 70] = float("nan")
        qkv[2, 3, 0] = float("-inf")
        qkv[3, 3, 127] = float("nan")
    _case(10, dt, 1, 2, 128, [2], [4], 3, 0, norm=False, spoil=spoil)


def test_every_code_under_every_scale():
    """All 256 bytes of two codes under all 256 scales (byte 0 counts as 1)."""
    note("mx unpack all codes")
    B, D = 256, 512 // 2                                   # a row of 256 elements: 128 bytes
    codes = torch.arange(256, dtype=torch.uint8).view(2, 1, 1, 128).expand(2, B, 1, 128)[None, :, :, :, None]
    scales = torch.arange(256, dtype=torch.uint8).view(1, B, 1, 1).expand(2, B, 1, 8)[None, :, :, :, None]
    codes, scales = codes.contiguous(), scales.contiguous()
    want = mx.unpack(codes.numpy(), scales.numpy())
    for dt in ("bf16", "f32"):
        out = [torch.empty(B, 1, D, dtype=TDT[dt], device=DEV) for _ in range(2)]
        sv.spec_unpack_kv_mx(codes.to(DEV), scales.to(DEV), 0, i32([0]), i32([0] * B), *out)
        torch.cuda.synchronize()
        for i in (0, 1):
            got, w = f64(out[i]), want[0, i, :, :, 0]
            assert np.array_equal(np.isnan(got), np.isnan(w))
            fine = np.isfinite(w)
            # below the smallest normal number a value may be taken for 0
            small = np.abs(w) < 2.0 ** -126
            assert np.array_equal(got[fine & ~small], w[fine & ~small])
            assert (np.abs(got[fine & small]) <= 2.0 ** -126).all()


def _states(packed):
    """Three sequences, the middle one's state out of range."""
    return dict(cu=[0, 4, 8, 12], n=[4, 2, 4]) if packed else dict(cu=None, n=[0, -3, 2])


@pytest.mark.parametrize("page", [0, 4])
@pytest.mark.parametrize("packed", [False, True])
def test_a_bad_sequence_is_not_written_and_reads_as_zeros(page, packed):
    note(f"mx bad sequence page={page} packed={packed}")
    rng = np.random.default_rng(12)
    s = _states(packed)
    rows = [4, 4, 6]
    cache = MxCache(rng, "bf16", 1, 2, 64, rows, [4, 4, 6] if packed else [0, 0, 2], page)
    if packed:
        s["n"] = [4, 2, 6]                                # shorter than its range
    codes, scales = cache.on_device()
    qkv = dev(randn(rng, "bf16", 12, 4 * 2, 64))
    q_out, st = torch.empty(12, 4, 64, dtype=torch.bfloat16, device=DEV), torch.full((3,), -7, dtype=torch.int32, device=DEV)
    cu = None if s["cu"] is None else i32(s["cu"])
    names = ("spec_norm_rope_kv_mx_paged", "spec_unpack_kv_mx_paged") if page else ("spec_norm_rope_kv_mx", "spec_unpack_kv_mx")
    getattr(sv, names[0])(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], codes, scales, 0, cache.where(), i32(s["n"]), q_out,
                          cu_seqlens=cu, status=st)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0, sv.SPEC_ST_BAD_STATE, 0]
    c = codes.cpu().numpy()
    for b in range(3):
        same = all(np.array_equal(c[0, :, p, :, col], cache.codes[0, :, p, :, col]) for p, col in cache.places[b])
        assert same == (b == 1)
    out = [torch.full((12, 2, 64), 9.0, device=DEV) for _ in range(2)]
    getattr(sv, names[1])(codes, scales, 0, cache.where(), i32(s["n"]), *out, cu_seqlens=cu, status=st.fill_(-7))
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0, sv.SPEC_ST_BAD_STATE, 0]
    for x in out:
        assert bool((x[4:8] == 0).all()) and not bool((x[:4] == 9).any()) and not bool((x[8:] == 9).any())
        assert float(x[:4].abs().max()) > 0 and float(x[8:].abs().max()) > 0


def test_bad_pages_and_capacity():
    note("mx bad pages")
    rng = np.random.default_rng(13)
    cache = MxCache(rng, "f32", 1, 1, 64, [6, 6, 6], [4, 4, 4], 4)
    table = cache.table.copy()
    planes = cache.codes.shape[2]
    table[0, 1], table[1, 1] = planes, -1
    codes, scales = cache.on_device()
    qkv = dev(randn(rng, "f32", 6, 3, 64))
    q_out, st = torch.empty(6, 1, 64, device=DEV), torch.full((3,), -7, dtype=torch.int32, device=DEV)
    for n, want in (([4, 4, 4], [16, 16, 0]), ([3, 7, 4], [16, 32, 0])):
        sv.spec_norm_rope_kv_mx_paged(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], codes, scales, 0, i32(table), i32(n), q_out, status=st)
        out = [torch.full((6, 1, 64), 9.0, device=DEV) for _ in range(2)]
        sv.spec_unpack_kv_mx_paged(codes, scales, 0, i32(table), i32(n), *out, status=st)
        torch.cuda.synchronize()
        assert st.cpu().tolist() == want
        y = mx.unpack(*(a.astype(np.uint8) for a in mx.pack(f64(qkv[:, 2:]))))
        assert np.array_equal(f64(out[1][4:]), y[4:])
        assert bool((out[1][1:4] == 0).all())              # the bad pages' rows, and a sequence of a status
        assert np.array_equal(f64(out[1][0]), y[0]) == (n[0] == 3)


def test_ranges_past_the_tokens_and_tokens_of_no_sequence():
    note("mx ranges")
    rng = np.random.default_rng(14)
    cache = MxCache(rng, "bf16", 1, 1, 64, [8, 8, 8], [8, 8, 8], 0)
    codes, scales = cache.on_device()
    big = 2 ** 31 - 1
    for cu, left, zeros in (([2, 5, 5, 7], [0, 1, 7, 8, 9], []), ([0, 3, 6, 12], [], [6, 7, 8, 9]),
                            ([0, 4, 2, 9], [4, 5, 6, 7, 8, 9], []), ([-2, 1, 3, 4], [4, 5, 6, 7, 8, 9], [0]),
                            ([-big - 1, big, 0, 1], [], list(range(10)))):
        out = [torch.full((10, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        sv.spec_unpack_kv_mx(codes, scales, 0, i32([10]), i32([8, 8, 8]), *out, cu_seqlens=i32(cu))
        torch.cuda.synchronize()
        for x in out:
            for t in range(10):
                assert bool((x[t] == 9).all()) == (t in left), (cu, t)
                assert bool((x[t] == 0).all()) == (t in zeros), (cu, t)


def test_two_streams_and_a_graph():
    note("mx rows graph")
    rng = np.random.default_rng(15)
    cache = MxCache(rng, "bf16", 1, 2, 128, [40, 30], [36, 26], 16)
    qkv = dev(randn(rng, "bf16", 8, 8, 128))
    codes, scales = cache.on_device()
    table, n = cache.where(), i32([36, 26])
    q_out = torch.empty(8, 4, 128, dtype=torch.bfloat16, device=DEV)
    k_out, v_out = (torch.empty(8, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def both(stream=None):
        sv.spec_norm_rope_kv_mx_paged(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], codes, scales, 0, table, n, q_out, stream=stream)
        sv.spec_unpack_kv_mx_paged(codes, scales, 0, table, n, k_out, v_out, stream=stream)
    both()
    torch.cuda.synchronize()
    want = [x.clone() for x in (q_out, k_out, v_out, codes, scales)]
    side = torch.cuda.Stream()
    for x in (q_out, k_out, v_out):
        x.zero_()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (q_out, k_out, v_out, codes, scales)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    base = qkv.clone()
    for i in range(4):
        qkv.copy_(base * (1 + i))
        both()
        torch.cuda.synchronize()
        want = [x.clone() for x in (q_out, k_out, v_out, codes, scales)]
        for x in (q_out, k_out, v_out, codes):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (q_out, k_out, v_out)]
        assert all(torch.equal(a, b) for a, b in zip(want[:3], got)), i

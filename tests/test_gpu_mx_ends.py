"""Writing rows into a cache of 4-bit numbers where exponents and angles leave the
ordinary: sizes of keys, queries and weights, positions far from 0, the largest numbers."""
from fractions import Fraction
from functools import cache

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_04_amd as sv
from oracle import mx
from tests._attn import EPS32, HALF, assert_within, dev, f64, randn
from tests._gpu import DEV, i32, note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _write(q, k, v, positions=None, **more):
    """T tokens of one sequence: codes and scales of K and V [T, H, ..], and q_out."""
    T, H, D = k.shape
    codes = torch.full((1, 2, 1, H, T, D // 2), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((1, 2, 1, H, T, D // 32), 0x5A, dtype=torch.uint8, device=DEV)
    q_out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    st = torch.full((1,), -7, dtype=torch.int32, device=DEV)
    sv.spec_norm_rope_kv_mx(dev(q), dev(k), dev(v), codes, scales, 0, i32([0]), i32([0]), q_out, status=st,
                            positions=None if positions is None else i32(positions),
                            **{n: dev(x) if torch.is_tensor(x) else x for n, x in more.items()})
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0]
    c, s = (x[0, :, 0].permute(0, 2, 1, 3).cpu().numpy() for x in (codes, scales))
    return c, s, q_out


def _freq(half):
    return (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def _times(x, power):
    """x times 2^power, rounded to its type once."""
    return (x.double() * 2.0 ** power).to(x.dtype)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rot,near", [(0, False), (64, False), (22, False), (64, True)])
@pytest.mark.parametrize("key,weight,eps", [(100, 30, 1e-5), (60, 90, 0.0), (-100, -40, 0.0), (-90, 100, 0.0), (-70, -60, 0.0),
                                            (120, -110, 1e-6), (3, -122, 1e-6)])
def test_sizes_of_keys_and_weights(dt, rot, near, key, weight, eps):
    """The product of a key and its weight may leave float32 where the normed key does not.  Keys are float64:
    codes are the definition's byte for byte (no element of these is within 2^-36 of a border)."""
    note(f"mx sizes of keys {dt} rot={rot} near={near} 2^{key} 2^{weight}")
    rng = np.random.default_rng(abs(key) + rot)
    T, H, D = 6, 3, 64
    k, v = _times(randn(rng, dt, T, H, D), key), randn(rng, dt, T, H, D)
    w = _times(randn(rng, dt, D), weight)
    want = oracle.norm_rope(f64(k), f64(w), eps, np.arange(T), _freq(rot // 2), near)
    assert mx.border_distance(want).min() > 2.0 ** -36
    c, s, _ = _write(randn(rng, dt, T, H, D), k, v, k_weight=w, eps=eps, interleaved=near,
                     inv_freq=torch.from_numpy(_freq(rot // 2)) if rot else None)
    want_c, want_s = mx.pack(want)
    assert np.array_equal(s[0], want_s)
    assert np.array_equal(c[0], want_c)

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679, 10 ** 100)


def _turned(pos, freq):
    """Cosine and sine of pos * freq: the angle is reduced exactly, so they are float64's nearest but for 2^-52."""
    turns = Fraction(int(pos)) * Fraction(float(freq)) / (2 * PI)
    t = float((turns - round(turns)) * 2 * PI)
    return np.cos(t), np.sin(t)


@cache
def _cases(pos, freq):
    """(border, side, pair) for keys that turn by pos * freq, and that angle's cosine and sine."""
    rng = np.random.default_rng(pos % 1000)
    cos, sin = _turned(pos, freq)
    cases = [(b, side, _pair_next_to(rng, b, cos, sin, side)) for b in (0.75, 1.25, 1.75, 2.5, 3.5) for side in (-1, 1)]
    return [x for x in cases if x[2]], cos, sin


def _pair_next_to(rng, border, cos, sin, side):
    """float32 a and m with a cos - m sin between 2^-44 and 2^-42 from the border, on the given side."""
    other = rng.uniform(2.0, 5.8, 1 << 22)                # its partner: what an error of the angle is multiplied by
    a = (border * cos + other * sin).astype(np.float32).astype(np.float64)
    m = ((a * cos - border) / sin).astype(np.float32).astype(np.float64)
    off = (a * cos - m * sin - border) * side
    good = np.nonzero((off > 2.0 ** -44) & (off < 2.0 ** -42) & (np.abs(m * cos + a * sin) < 5.9))[0]
    return (a[good[0]], m[good[0]]) if len(good) else None


@pytest.mark.parametrize("rot,near", [(64, False), (2, False), (64, True)])
@pytest.mark.parametrize("pos,freq", [(1, 1.0), (2000, 1.0), (2000, 0.7), (131071, 1.0), (131071, 0.9), ((1 << 20) + 1, 0.7),
                                      ((1 << 24) + 3, 0.3), ((1 << 29) + 1, 0.9), (2 ** 31 - 1, 1.0), (2 ** 31 - 1, 0.7)])
def test_angles_decide_no_code(pos, freq, rot, near):
    """Keys whose rotated element lies 2^-44 to 2^-42 from a border, on either side.  An angle that is off by
    2^-54 of a turn moves it by 2 pi 2^-54 times its partner (below 6), and the sine, the cosine and the products
    by 2^-49 at most: 2^-48 together."""
    note(f"mx angles pos={pos} freq={freq} rot={rot} near={near}")
    freq = np.float32(freq)
    cases, cos, sin = _cases(pos, freq)
    assert len(cases) >= 4
    D, half = 64, rot // 2
    T, lo, hi = len(cases), 0, 1 if near else half
    k = np.zeros((T, 1, D), np.float32)
    want = np.zeros((T, 1, D))
    still = 10 if rot > 2 else 4                          # a pair that does not turn, in both blocks: the largest elements
    k[:, 0, still] = k[:, 0, still + 32] = want[:, 0, still] = want[:, 0, still + 32] = 6.0
    for t, (border, side, (a, m)) in enumerate(cases):
        k[t, 0, lo], k[t, 0, hi] = a, m
        want[t, 0, lo], want[t, 0, hi] = a * cos - m * sin, m * cos + a * sin
    inv_freq = np.zeros(half, np.float32)
    inv_freq[0] = freq
    x = torch.from_numpy(k)
    c, s, _ = _write(x, x, x, positions=[pos] * T, inv_freq=torch.from_numpy(inv_freq), interleaved=near)
    want_c, want_s = mx.pack(want)
    assert np.array_equal(s[0], want_s)
    assert np.array_equal(c[0], want_c), [x[:2] for x, g, w in zip(cases, c[0], want_c) if not np.array_equal(g, w)]


def test_keys_next_to_the_largest_number():
    """As float32 a key of 2^128 - 2^103 and more is infinite, and one below it the largest number."""
    note("mx largest keys")
    largest, t = float(np.finfo(np.float32).max), 2.0 ** -20
    k = np.zeros((5, 1, 64), np.float32)
    for i, steps in enumerate((0.0, 0.9, 0.99, 1.01, 1.5)):   # of 2^103 above the largest number
        k[i, 0, 0], k[i, 0, 32] = largest, -steps * 2.0 ** 103 / t
    freq = np.zeros(32, np.float32)
    freq[0] = t
    want = oracle.norm_rope(k.astype(np.float64), None, 0.0, [1] * 5, freq)
    x = torch.from_numpy(k)
    c, s, _ = _write(x, x, x, positions=[1] * 5, inv_freq=torch.from_numpy(freq))
    want_c, want_s = mx.pack(want)
    assert want_s[:, 0, 0].tolist() == [252, 252, 252, 255, 255]
    assert np.array_equal(s[0], want_s)
    assert np.array_equal(c[0], want_c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rot,near", [(0, False), (64, False), (22, False), (64, True)])
@pytest.mark.parametrize("query,weight,eps", [(50, 90, 1e-5), (-50, -90, 0.0), (-50, 110, 0.0), (-64, 0, 0.0), (-64, 100, 0.0),
                                              (40, -110, 1e-6)])
def test_sizes_of_queries_and_weights(dt, rot, near, query, weight, eps):
    """As spec_norm_rope_kv's queries: statistics in float32, the norm before the weight.  Squares of 2^-64 are
    below the smallest normal number and off by 2^-150 each, 2^-22 of themselves, and the root by half of it:
    two EPS32 more."""
    note(f"mx sizes of queries {dt} rot={rot} near={near} 2^{query} 2^{weight}")
    rng = np.random.default_rng(abs(query) + rot)
    T, Hq, H, D = 6, 6, 3, 64
    q, kv = _times(randn(rng, dt, T, Hq, D), query), randn(rng, dt, T, H, D)
    w = _times(randn(rng, dt, D), weight)
    want = oracle.norm_rope(f64(q), f64(w), eps, np.arange(T), _freq(rot // 2), near)
    size = np.abs(oracle.norm_rope(f64(q), f64(w), eps, np.arange(T), _freq(0), near)).max(-1, keepdims=True)
    _, _, got = _write(q, kv, kv, q_weight=w, eps=eps, interleaved=near,
                       inv_freq=torch.from_numpy(_freq(rot // 2)) if rot else None)
    # results below the smallest normal number have an absolute step, 2^-133 in bf16
    tol = (D + 34) * EPS32 * size + 1.01 * HALF[dt] * np.abs(want) + 2.0 ** (-133 if dt == "bf16" else -149)
    assert_within(got, want, tol)



@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,near", [(64, 64, False), (128, 40, False), (192, 96, True), (256, 256, False)])
def test_bytes_of_codes_and_scales(dt, D, rot, near):
    """Every byte, signs of zeros and the codes of blocks that are not finite among them."""
    note(f"mx bytes {dt} D={D} rot={rot} near={near}")
    rng = np.random.default_rng(D)
    T, H = 7, 3
    k, v = randn(rng, dt, T, H, D, sd=3.0), randn(rng, dt, T, H, D, sd=3.0)
    for x in (k, v):
        x[0, 0, 5::7] = -0.0
        x[2, 2, D - 1] = float("nan")
        x[3, 0] = 0.0
        x[4, 1] = -0.0
        x[5, 2, 10:20] *= 2.0 ** -9                       # codes of 0 with either sign
    v[1, 1, 3], v[1, 2, D - 1] = float("inf"), float("-inf")
    w = randn(rng, dt, D)
    with np.errstate(invalid="ignore"):
        keys = oracle.norm_rope(f64(k), f64(w), 1e-5, np.arange(T), _freq(rot // 2), near)
    c, s, _ = _write(randn(rng, dt, T, H, D), k, v, k_weight=w, eps=1e-5, interleaved=near,
                     inv_freq=torch.from_numpy(_freq(rot // 2)))
    for i, y in ((0, keys), (1, f64(v))):
        want_c, want_s = mx.pack(y)
        assert i == 1 or np.nanmin(mx.border_distance(y)) > 2.0 ** -36
        assert np.array_equal(s[i], want_s), "kv"[i]
        assert np.array_equal(c[i], want_c), "kv"[i]
        assert (s[i] == 255).any() and (np.repeat(s[i] == 255, 16, axis=-1) <= (c[i] == 0)).all()


def test_streams_and_replays_write_codes_and_scales():
    """A call on another stream and each replay of a captured one fill the cache themselves."""
    note("mx rows again")
    rng = np.random.default_rng(16)
    T, H, D = 5, 2, 128
    q, k, v = (dev(randn(rng, "bf16", T, h, D)) for h in (4, H, H))
    codes = torch.empty(1, 2, 1, H, 16, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(1, 2, 1, H, 16, D // 32, dtype=torch.uint8, device=DEV)
    E, n, q_out = i32([4]), i32([3]), torch.empty_like(q)
    rows = [codes, scales, q_out]

    def write(stream=None):
        sv.spec_norm_rope_kv_mx(q, k, v, codes, scales, 0, E, n, q_out, stream=stream)

    def marked():
        for x in rows:
            x.view(torch.uint8).fill_(0x5A)

    def result():
        torch.cuda.synchronize()
        return [x.clone() for x in rows]
    marked()
    write()
    want = result()
    assert int((want[0] != 0x5A).sum()) > 2 * H * T * D // 4 and int((want[1] != 0x5A).sum()) == 2 * H * T * D // 32
    side = torch.cuda.Stream()
    marked()
    side.wait_stream(torch.cuda.current_stream())
    write(side)
    assert all(torch.equal(a, b) for a, b in zip(want, result()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        write()
    base = [x.clone() for x in (q, k, v)]
    for i in range(4):
        for x, y in zip((q, k, v), base):
            x.copy_(y * (1 + i))
        marked()
        write()
        want = result()
        marked()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, result())), i

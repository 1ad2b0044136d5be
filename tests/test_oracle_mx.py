"""Pins of the 4-bit format's oracle: the format's own numbers, and what the
choice of scale and code promises."""
import numpy as np
import pytest

from oracle import mx


def _block(*head):
    x = np.zeros(32)
    x[:len(head)] = head
    return x


def test_every_code_and_where_it_lies():
    values = [0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6]
    codes, scales = mx.pack(_block(*values))
    assert scales.tolist() == [127]
    want = [0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11, 12, 13, 14, 15]
    nibbles = np.stack([codes & 15, codes >> 4], -1).reshape(-1)
    assert nibbles[:15].tolist() == want and not nibbles[15:].any()
    assert codes[0] == 0x10 and codes[1] == 0x32          # the even element in the low half
    assert mx.unpack(codes, scales)[:15].tolist() == values


def test_ties_go_to_the_even_code():
    ties = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0]
    codes, scales = mx.pack(_block(6.0, *ties))
    assert mx.unpack(codes, scales)[1:8].tolist() == [0, 1, 1, 2, 2, 4, 4]


@pytest.mark.parametrize("top,e", [(1.0, -2), (1.74, -2), (1.75, -1), (1.99, -1), (2.0, -1), (3.49, -1), (3.5, 0),
                                   (6.99, 0), (7.0, 1), (8.0, 1), (0.0, -125), (2.0 ** -140, -125), (3e38, 125)])
def test_the_scale_of_a_largest_element(top, e):
    assert mx.scale_exponents(_block(top, -top / 3)).tolist() == [e]


def test_no_element_is_off_by_more_than_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((500, 64)) * 10.0 ** rng.uniform(-20, 20, (500, 1))
    codes, scales = mx.pack(x)
    y = mx.unpack(codes, scales)
    unit = 2.0 ** np.repeat(scales.astype(float) - 127, 32, axis=-1)
    step = np.where(np.abs(x) < 2 * unit, .5, np.where(np.abs(x) < 4 * unit, 1, 2)) * unit
    assert (np.abs(x - y) <= step / 2).all()
    top = np.abs(y).reshape(500, 2, 32).max(-1) / unit[:, ::32]
    assert np.isin(top, [4, 6]).all()


def test_packing_values_gives_their_codes_again():
    rng = np.random.default_rng(2)
    codes, scales = mx.pack(rng.standard_normal((40, 128)))
    again = mx.pack(mx.unpack(codes, scales))
    assert np.array_equal(again[1], scales) and np.array_equal(again[0], codes)


@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan, 3.5e38])
def test_what_is_not_finite(odd):
    x = np.ones(64)
    x[40] = odd
    codes, scales = mx.pack(x)
    assert scales.tolist() == [125, 255] and not codes[16:].any()
    y = mx.unpack(codes, scales)
    assert np.isnan(y[32:]).all() and (y[:32] == 1).all()
    assert np.isnan(mx.unpack(np.zeros(16, np.uint8), np.array([253], np.uint8))).all()


def test_distance_from_a_border():
    d = mx.border_distance(_block(4.0, 1.2, 0.75))
    assert np.isclose(d[1], min(.05 / 1.2, .125)) and d[2] == 0 and np.isinf(d[3:]).sum() == 0
    assert np.isclose(d[0], min(.5 / 4, .125))

"""Pins of the attention oracle: what ties it to something other than itself."""
import numpy as np
import pytest

import oracle
import workloads as W


def test_tree_paths_hand_worked():
    # 0 -> 1, 2 (siblings); 1 -> 3; node 4 is linked to nothing
    fc, ns = np.array([[1, 3, -1, -1, -1]]), np.array([[-1, 2, -1, -1, -1]])
    pos, see, status = oracle.tree_paths(fc, ns, [5])
    assert pos.tolist() == [[5, 6, 6, 7, 5]] and status.tolist() == [0]
    assert oracle.mask_words(see)[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0]


def test_tree_paths_follow_the_generators_parents():
    rng = np.random.default_rng(3)
    for N in (1, 2, 33, 70):
        parent, fc, ns = W.random_tree(rng, N, 4)
        pos, see, _ = oracle.tree_paths(fc[None], ns[None], [11])
        for i in range(N):
            path, x = [], i
            while x != -1:
                path.append(x)
                x = int(parent[x])
            assert sorted(path) == np.nonzero(see[0, i])[0].tolist()
            assert pos[0, i] == 11 + len(path) - 1


@pytest.mark.parametrize("fc,ns", [([0, -1], [-1, -1]), ([2, -1], [-1, -1]), ([1, -1, -1], [1, -1, -1])])
def test_tree_paths_bad_links(fc, ns):
    pos, see, status = oracle.tree_paths(np.array([fc]), np.array([ns]), [4])
    assert status.tolist() == [oracle.ST_BAD_STATE] and not see.any() and (pos == 4).all()


def test_rotation_keeps_lengths_and_depends_on_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 16))
    freq = 10.0 ** -np.arange(8)
    for near in (False, True):
        at = lambda x, p: oracle.norm_rope(x, None, 0.0, [p], freq, near)[0, 0]  # noqa: E731
        assert np.allclose(at(q, 7) @ at(q, 7), q.ravel() @ q.ravel())
        assert np.allclose(at(q, 107) @ at(k, 100), at(q, 12) @ at(k, 5))
        assert np.allclose(at(q, 0), q.ravel())


def test_rotation_by_a_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    freq = [np.pi / 2, 0.0]
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [1], freq)[0, 0], [-3, 2, 1, 4])
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [1], freq, True)[0, 0], [-2, 1, 3, 4])


def test_norm_of_a_known_head():
    y = oracle.norm_rope(np.array([[[3.0, 4.0]]]), np.array([1.0, 10.0]), 0.0, [0], [])
    assert np.allclose(y, [[[3 / np.sqrt(12.5), 40 / np.sqrt(12.5)]]])


def test_attend_closed_forms():
    k = np.zeros((4, 2))
    v = np.arange(8.0).reshape(4, 2)
    see = np.array([[1, 1, 0, 0], [1, 1, 1, 1], [0, 0, 0, 0]], bool)
    out, lse = oracle.attend(np.ones((3, 2)), k, v, see, 1.0)     # equal scores: the mean of the rows seen
    assert np.allclose(out, [[1, 2], [3, 4], [0, 0]])
    assert np.allclose(lse[:2], np.log([2, 4])) and lse[2] == -np.inf
    k2 = np.array([[0.0], [np.log(3.0)]])                          # weights 1 : 3
    out, lse = oracle.attend(np.ones((1, 1)), k2, np.array([[0.0], [4.0]]), np.ones((1, 2), bool), 1.0)
    assert np.allclose(out, 3.0) and np.allclose(lse, np.log(4.0))


def test_attend_ignores_what_is_not_seen():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 5, 4))
    see = np.tril(np.ones((5, 5), bool))
    want, _ = oracle.attend(q, k, v, see, 0.5)
    k[4], v[4] = np.nan, np.inf
    got, _ = oracle.attend(q, k, v, see, 0.5)
    assert np.array_equal(got[:4], want[:4]) and np.isnan(got[4]).all()


def test_row_places():
    assert oracle.row_places(1, 4, 3, E=10) == [(1, 7), (1, 8), (1, 9), (1, 10)]
    assert oracle.row_places(0, 5, 3, table=[[9, 4, 7]], page=2) == [(9, 0), (9, 1), (4, 0), (4, 1), (7, 0)]

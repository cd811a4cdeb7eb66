"""Pins of the float64 reference of drafted trees: closed forms and invariants."""
import numpy as np
import pytest

from oracle import scored, tree


def _normal(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_lineages():
    assert tree.lineages([-1, 0, 0, 1, 3, -1, -2, 6, 8, 20]) == [
        [0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [5], [], [], [], []]


def test_a_chain_is_the_decoding_step():
    """A chain's nodes are the newest tokens of a cache that holds them."""
    B, h, n, L, d = 2, 4, 3, 9, 8
    q, k, v = _normal(B, h, n, d), _normal(B, 2, L + n, d, seed=1), _normal(B, 2, L + n, d, seed=2)
    lens = [L, 4]
    kt = np.stack([k[b, :, lens[b]:lens[b] + n] for b in range(B)])
    vt = np.stack([v[b, :, lens[b]:lens[b] + n] for b in range(B)])
    slopes = np.array([0.5, 0.25, 0.1, 0.0])
    for window in (None, 0, 2, 5):
        got = tree.attention(q, kt, vt, k, v, [[-1, 0, 1]] * B, lens, 0.3, 5.0, slopes, window)
        want = scored.decode(q, k, v, [x + n for x in lens], 0.3, 5.0, slopes, window)
        for x, y in zip(got, want):
            assert np.allclose(x, y, atol=1e-12)


def test_each_node_sees_its_own_branch_only():
    """A tree's node has the answer of its branch alone, as a chain."""
    n, L, d = 7, 5, 4
    parents = [-1, 0, 0, 1, 1, 2, -1]
    q, kt, vt = _normal(1, 1, n, d), _normal(1, 1, n, d, seed=1), _normal(1, 1, n, d, seed=2)
    k, v = _normal(1, 1, L, d, seed=3), _normal(1, 1, L, d, seed=4)
    o, lse = tree.attention(q, kt, vt, k, v, [parents], [L], 0.5)
    for i, line in enumerate(tree.lineages(parents)):
        m = len(line)
        one = tree.attention(q[:, :, line], kt[:, :, line], vt[:, :, line], k, v,
                             [list(range(-1, m - 1))], [L], 0.5)
        assert np.allclose(one[0][0, 0, -1], o[0, 0, i], atol=1e-12)
        assert np.allclose(one[1][0, 0, -1], lse[0, 0, i], atol=1e-12)


def test_no_node_sees_nothing():
    o, lse = tree.attention(_normal(1, 1, 2, 4), _normal(1, 1, 2, 4), np.full((1, 1, 2, 4), 3.0),
                            _normal(1, 1, 3, 4), _normal(1, 1, 3, 4), [[-2, 0]], [3], 1.0)
    assert (o == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("with_draft", [True, False])
def test_what_is_kept_is_distributed_as_the_target(with_draft):
    """Sum over every outcome of the draft and of the tests: the first token after
    the root has the target's probabilities."""
    p = np.array([0.5, 0.25, 0.125, 0.125])
    q = np.array([0.125, 0.125, 0.25, 0.5])
    got = np.zeros(4)
    if with_draft:
        draws = [((x, y), q[x] * q[y]) for x in range(4) for y in range(4)]
    else:
        draws = [((3, 0), 1.0)]
    parents = [-1, 0, 0]
    # a border between the midpoints of a grid of 64 is off by 1/128 at most, for each
    # of the two numbers
    grid = (np.arange(64) + 0.5) / 64
    for (x, y), chance in draws:
        for u1 in grid:
            for u2 in grid:
                target = np.stack([p, np.eye(4)[0], np.eye(4)[0]])
                path, r, _ = tree.verify(target, [0, x, y], parents, [0.0, u1, u2],
                                         np.stack([q, q, q]) if with_draft else None)
                w = chance / len(grid) ** 2
                if len(path) > 1:
                    got[[0, x, y][path[1]]] += w
                else:
                    got += w * r / r.sum()
    assert np.allclose(got, p, atol=1 / 64)


def test_walk_goes_on_from_the_child_that_stands():
    target = np.full((4, 3), 1 / 3)
    tokens, parents = [0, 2, 1, 0], [-1, 0, 0, 1]
    assert tree.verify(target, tokens, parents, [0.0, 0.9, 0.0, 0.1])[0] == [0, 2]
    assert tree.verify(target, tokens, parents, [0.0, 0.1, 0.0, 0.1])[0] == [0, 1, 3]
    path, r, _ = tree.verify(target, tokens, parents, [0.0, 0.9, 0.9, 0.1])
    assert path == [0] and r.tolist() == [1 / 3, 0.0, 0.0]


def test_next_tokens():
    r = np.array([0.0, 0.25, 0.0, 0.25])
    assert tree.next_tokens(r, 0.0, 0.0) == {1} and tree.next_tokens(r, 0.4999, 0.0) == {1}
    assert tree.next_tokens(r, 0.5, 0.0) == {3} and tree.next_tokens(r, 0.5, 1e-3) == {1, 3}
    assert tree.next_tokens(np.zeros(3), 0.5, 0.0) == {-1}


def test_append_path_cuts_at_a_bad_node():
    cache, nodes = np.zeros((1, 1, 1, 4, 2)), _normal(1, 1, 1, 3, 2)
    tree.append_path(cache, None, nodes, [[0, 2, 7]], [3], [1], 16, False)
    assert np.array_equal(cache[0, 0, 0, 1:3], nodes[0, 0, 0, [0, 2]])
    assert (cache[0, 0, 0, [0, 3]] == 0).all()

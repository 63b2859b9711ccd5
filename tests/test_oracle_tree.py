"""The drafted-tree oracle's pins: a chain is causal attention, verification reproduces the target's
distribution, kept paths move the records they name."""

import itertools

import numpy as np
import pytest

from oracle import paged, tree
from oracle.formats import Codec


def test_lines_and_positions():
    parents = [-1, 0, 0, 1, 1, -1, 5]
    assert tree.lines(parents) == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [5], [5, 6]]
    assert list(tree.positions([10], [0, 7], parents)) == [3, 4, 4, 5, 5, 3, 4]


def test_a_chain_is_causal():
    rng = np.random.default_rng(1)
    c = Codec("turbo4", rotation="wht", rot_seed=3)
    pages = rng.integers(0, 256, (4, 2, 16, 68), dtype=np.uint8)
    pages[..., :4] = np.frombuffer(np.float32(1.5).tobytes(), np.uint8)
    table, lens, cu = np.array([[2, 0, 3]]), [40], np.array([0, 5])
    q = rng.standard_normal((5, 4, 128))
    got = tree.attention(c, c, pages, pages, table, lens, cu, [-1, 0, 1, 2, 3], q, 5)
    want = paged.attention(c, c, pages, pages, table, lens, cu, q, 5)
    assert np.allclose(got, want, atol=1e-14)
    # siblings do not see one another: the second of two roots is a one-row batch without the first
    both = tree.attention(c, c, pages, pages, table, lens, cu, [-1, -1, 1, 1, 0], q, 5)
    assert np.allclose(both[0], got[0], atol=1e-14) and not np.allclose(both[1], got[1], atol=1e-3)


# Dyadic probabilities and random numbers on a grid whose cells no border crosses: the outcome's
# distribution is then an exact count.
P = np.array([[4, 2, 1, 1], [1, 1, 4, 2], [2, 2, 2, 2]]) / 8
Q = np.array([[2, 4, 1, 1], [4, 2, 1, 1], [1, 1, 2, 4]]) / 8


def outcomes(parents, tokens, target, draft, grid):
    count = {}
    u = (np.arange(grid) + 0.5) / grid
    for us in itertools.product(u, repeat=len(parents)):
        path, w = tree.verify(parents, tokens, target, np.array((0.0, *us[:-1])), us[-1], draft)
        said = tuple(int(tokens[c]) for c in path[1:]) + (w,)
        count[said[0]] = count.get(said[0], 0) + 1
    return count


def test_verify_chain_gives_the_targets_distribution():
    """One drafted token, each drawn with its draft probability: the first token said is p's."""
    grid, got = 64, np.zeros(4)
    for x in range(4):
        n = outcomes([-1, 0], [0, x], P, Q, grid)
        got += Q[0, x] * np.array([n.get(w, 0) for w in range(4)]) / grid ** 2
    assert np.allclose(got, P[0], atol=2e-2)  # cells of 1/64 in two numbers


def test_verify_siblings_give_the_targets_distribution():
    """Two tokens drawn independently behind the root."""
    grid, got = 16, np.zeros(4)
    for x, y in itertools.product(range(4), repeat=2):
        n = outcomes([-1, 0, 0], [0, x, y], P, Q, grid)
        got += Q[0, x] * Q[0, y] * np.array([n.get(w, 0) for w in range(4)]) / grid ** 3
    assert np.allclose(got, P[0], atol=8e-2)  # cells of 1/16 in three numbers


@pytest.mark.parametrize("tokens", [[0, 1, 2], [0, 3, 0], [0, 2, 2]])
def test_verify_without_a_draft_gives_the_targets_distribution(tokens):
    grid = 16
    n = outcomes([-1, 0, 0], tokens, P, None, grid)
    got = np.array([n.get(w, 0) for w in range(4)]) / grid ** 3
    assert np.allclose(got, P[0], atol=8e-2)


def test_verify_walks():
    one = np.eye(4)[[1, 2, 3, 0]]  # the target's choices: 1, then 2, then 3
    assert tree.verify([-1, 0, 1, 0], [9, 1, 2, 0], one[[0, 1, 2, 3]], np.full(4, 0.5), 0.5) == ([0, 1, 2], 3)
    assert tree.verify([-1, 0, 0, 2], [9, 0, 1, 2], one[[0, 3, 1, 2]], np.full(4, 0.5), 0.5) == ([0, 2, 3], 3)
    assert tree.verify([-1], [9], np.zeros((1, 4)), [0.0], 0.5) == ([0], -1)
    assert tree.verify([-1, 0], [9, 7], one[:2], [0.0, 0.0], 0.5) == ([0], 1)  # a token outside


def test_keep_moves_what_the_path_names():
    pages = np.arange(3 * 1 * 16 * 68).astype(np.uint8).reshape(3, 1, 16, 68)
    pages[:, :, :, 0] = np.arange(48).reshape(3, 1, 16)
    table = np.array([[2, 0, 1], [1, 1, 1]])
    out, lens = tree.keep(pages, table, [20, 0], [0, 6, 6], [[0, 2, 5], []])  # slots 14 .. 19
    assert lens == [17, 0]
    slots = lambda p: [int(p[table[0, t // 16], 0, t % 16, 0]) for t in range(20)]  # noqa: E731
    a, b = slots(pages), slots(out)
    assert b[14:17] == [a[14], a[16], a[19]] and b[:14] == a[:14] and b[17:] == a[17:]


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "no-draft"])
def test_whole_multiples_change_ordinary_walks_nowhere(draft):
    """2^-62 is far below any border that random rows put next to a random number."""
    rng = np.random.default_rng(9)
    for _ in range(60):
        T, V = int(rng.integers(1, 9)), int(rng.integers(2, 40))
        p, q = (rng.dirichlet(np.full(V, 0.3), T).astype(np.float32) for _ in range(2))
        parents = [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, T)]
        args = (parents, rng.integers(0, V, T), p, rng.random(T).astype(np.float32), np.float32(rng.random()), q if draft else None)
        assert tree.verify_fixed(*args) == tree.verify(*args)


def test_whole_multiples_round_down():
    """p(1) = 3.99 x 2^-62 holds three of them; 3.5 x 2^-62 of Z = 1 is three as well, so the child is not taken where
    the exact numbers take it.  A weight below 2^-62 is none."""
    p = np.array([[1.0, 3.99 * 2.0 ** -62], [2.0 ** -63, 2.0 ** -62]], np.float32)
    u = np.array([0.0, 3.5 * 2.0 ** -62], np.float32)
    assert tree.verify([-1, 0], [0, 1], p, u, 0.5) == ([0, 1], 1)
    assert tree.verify_fixed([-1, 0], [0, 1], p, u, 0.5) == ([0], 0)
    assert tree.verify_fixed([-1], [0], p[1:], u, 0.0) == ([0], 1) and tree.verify([-1], [0], p[1:], u, 0.0) == ([0], 0)
    assert list(tree.fixed([np.nan, -1.0, 0.5, 2.0, np.inf])) == [0, 0, 1 << 61, 1 << 62, 1 << 62]

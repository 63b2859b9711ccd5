"""The dense rotations that are held from one use of a seed to the next."""

import threading

import numpy as np
import pytest

from oracle.formats import Codec


@pytest.fixture(scope="module")
def tq():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_attention_gb300 as m
    return m


@pytest.mark.parametrize("d", [128, 256])
def test_a_seed_gives_its_matrix_whatever_was_made_between(tq, d):
    """More seeds than are held, in both dimensions; the same bits each time, and the matrix of the definition
    (fp64 factorisations in another order of sums, rounded to fp32: a step of 2^-24 of the largest element)."""
    first = {s: tq.tq_make_rotation("dense", s, d) for s in range(3)}
    for s in range(20):
        tq.tq_make_rotation("dense", 100 + s, 128 if s % 2 else d)
    for s, m in first.items():
        again = tq.tq_make_rotation("dense", s, d)
        assert np.array_equal(m, again)
        again[:] = 0  # the caller's copy
        assert np.array_equal(m, tq.tq_make_rotation("dense", s, d))
        assert np.abs(m - Codec("turbo4", d=d, rotation="dense", rot_seed=s).rot.R).max() <= 2.0 ** -24
    assert not np.array_equal(first[0], first[1])


def test_threads_get_their_own_seeds(tq):
    want = {s: tq.tq_make_rotation("dense", s) for s in range(12)}
    wrong = []

    def work(k):
        for i in range(30):
            s = (5 * k + 7 * i) % 12
            if not np.array_equal(tq.tq_make_rotation("dense", s), want[s]):
                wrong.append(s)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong

"""Pins of the sampling oracle (no GPU): closed forms of the filters, and that verification gives
the target's distribution whatever the drafter's."""
import itertools

import numpy as np
import pytest

from oracle import peagle_oracle as O
from oracle import sample_oracle as S

X = np.log([0.4, 0.1, 0.2, 0.2, 0.05, 0.05])


def test_filters_on_a_row_that_can_be_done_by_hand():
    assert np.allclose(S.distribution(X), [0.4, 0.1, 0.2, 0.2, 0.05, 0.05])
    assert np.allclose(S.distribution(X, top_k=2), [2 / 3, 0, 1 / 3, 0, 0, 0])  # the lower of two
    assert np.allclose(S.distribution(X, top_p=0.39), [1, 0, 0, 0, 0, 0])
    assert np.allclose(S.distribution(X, top_p=0.59), [2 / 3, 0, 1 / 3, 0, 0, 0])
    assert np.allclose(S.distribution(X, top_k=4, top_p=0.88), [0.5, 0, 0.25, 0.25, 0, 0])  # of 0.9
    assert np.allclose(S.distribution(X, min_p=0.3), [0.5, 0, 0.25, 0.25, 0, 0])
    assert np.allclose(S.distribution(X, temperature=0.5),
                       np.square([0.4, 0.1, 0.2, 0.2, 0.05, 0.05]) / 0.255)
    for T in (0.0, 1e-30):
        assert np.array_equal(S.distribution(X, temperature=T), [1, 0, 0, 0, 0, 0])
    assert np.array_equal(S.distribution(np.zeros(3), top_k=1), [1, 0, 0])
    assert np.allclose(S.distribution(np.zeros(4), top_p=0.5), [0.5, 0.5, 0, 0])
    assert np.array_equal(S.distribution(X, top_p=-1.0), [1, 0, 0, 0, 0, 0])
    assert np.array_equal(S.distribution(X, min_p=5.0), [1, 0, 0, 0, 0, 0])


def test_rows_without_a_distribution():
    assert S.distribution([0, np.nan]) is None and S.distribution([0, np.inf]) is None
    assert S.distribution([-np.inf] * 3) is None and S.distribution([0.0], temperature=-1) is None
    assert S.sample([np.nan], 0.5)[0] == -1
    assert np.array_equal(S.distribution([-np.inf, 2.0]), [0, 1])


def test_pick():
    p = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [S.pick(p, u) for u in (0.0, 0.2499, 0.25, 0.7499, 0.75, 1.0, 2.0)] == [1, 1, 3, 3, 4, 4, 4]
    assert S.pick(p, np.nan) == 1 and S.pick(p, -3.0) == 1
    assert S.sample(np.zeros(4), 0.6, d2t=[5, 5, 7, 9]) == (9, 0.25, 2)


@pytest.mark.parametrize("seed", range(6))
def test_verification_gives_the_targets_distribution(seed):
    """Two drafts over five tokens, every pair of drafts weighted with q: the first two tokens that
    come out have the target's joint distribution.  The random numbers are integrated over: a draft
    is accepted with its probability, the bonus drawn from what is left."""
    r = np.random.default_rng(seed)
    n = 5
    p = [r.dirichlet(np.full(n, 0.7)) for _ in range(1 + n)]  # p[0], and p[1 + x] after token x
    q0, q1 = r.dirichlet(np.full(n, 0.7), 2)  # (the drafts are drawn without one another)
    if seed % 2:
        p[0][1] = 0.0
        p[0] /= p[0].sum()
    joint, first = np.zeros((n, n)), np.zeros(n)
    for x, y in itertools.product(range(n), repeat=2):
        _, _, prob = S.verify([x, y], [p[0], p[1 + x], p[0]], [q0, q1], [0.0, 0.0], 0.5)
        w = q0[x] * q1[y]
        left = S.left_over(p[0], q0)
        first += w * (1 - prob[0]) * left / left.sum()
        left = S.left_over(p[1 + x], q1)
        joint[x] += w * prob[0] * (1 - prob[1]) * left / left.sum()
        joint[x, y] += w * prob[0] * prob[1]
    assert np.allclose(joint.sum(1) + first, p[0], atol=1e-12)
    for x in range(n):  # given that the first draft was accepted
        if joint[x].sum() > 0:
            assert np.allclose(joint[x] / joint[x].sum(), p[1 + x], atol=1e-12)


def test_greedy_distributions_verify_greedily():
    r = np.random.default_rng(3)
    K, n = 4, 6
    target = r.integers(0, n, (8, K + 1))
    draft = np.where(r.random((8, K)) < 0.7, target[:, :K], r.integers(0, n, (8, K)))
    want = O.verify_greedy(draft, target)
    for b in range(8):
        p = list(np.eye(n)[target[b]])
        m, x, _ = S.verify(draft[b], p, list(np.eye(n)[draft[b]]), r.random(K), r.random())
        assert (m, x) == (want[0][b], want[1][b])


def test_bad_drafts_and_rows():
    p = [np.array([0.5, 0.5])] * 3
    assert S.verify([0, 7], p, p[:2], [0, 0], 0.9)[:2] == (1, 1)
    assert S.verify([0, 1], [p[0], None, p[0]], p[:2], [0, 0], 0.9)[:2] == (1, -1)
    assert S.verify([0, 1], p, [None, p[0]], [0, 0], 0.2)[:2] == (0, 0)
    assert np.array_equal(S.spread(np.array([0.25, 0.75]), [2, 0], 4), [0, 0.75, 0.25, 0])

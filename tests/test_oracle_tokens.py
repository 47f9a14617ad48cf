"""Pins of the oracle of the steps over several new tokens against closed forms."""

import math

import numpy as np

from oracle.tokens import rope_f64, softmax_f64, verify_f64, visible_slots


def test_rope_turns_by_the_angle():
    # a quarter turn of (1, 0) is (0, 1); a half turn is (-1, 0); behind n_rot nothing turns
    x = np.array([[[1.0, 5.0, 0.0, 7.0, 9.0]]])
    out = rope_f64(x, [[1]], [math.pi / 2, math.pi])
    assert np.allclose(out, [[[0.0, -5.0, 1.0, -7.0, 9.0]]])
    out = rope_f64(np.array([[[1.0, 0.0, 5.0, 7.0]]]), [[2]], [math.pi / 4, math.pi / 2], halves=False)
    assert np.allclose(out, [[[0.0, 1.0, -5.0, -7.0]]])


def test_rope_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 8))
    f = 10000.0 ** (-np.arange(4) / 4)
    def dot(a, b):
        return float((rope_f64(q, [[a]], f) * rope_f64(k, [[b]], f)).sum())
    assert np.isclose(dot(7, 3), dot(1004, 1000))   # only the distance counts
    assert np.allclose(np.square(rope_f64(q, [[99]], f)).sum(), np.square(q).sum())


def test_rope_axes_norm_and_magnitude():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    out = rope_f64(x, [[0], [1]], [math.pi / 2, math.pi / 2], axes=[0, 1], halves=True)
    assert np.allclose(out, [[[3.0, 0.0, 0.0, 4.0]]])   # pair 0 on axis 0 (position 0), pair 1 on axis 1
    out = rope_f64(x, [[0]], [1.0, 1.0], axes=[0, 9], magnitude=2.0, norm=[1.0, 2.0, 1.0, 1.0])
    assert np.allclose(out, [[[2 * 3 / 2.5, 2 * 8 / 2.5, 0.0, 0.0]]])


def test_visible_slots():
    assert visible_slots(5, 2, 0).tolist() == [0, 1, 2, 3] and visible_slots(5, 2, 1).tolist() == [0, 1, 2, 3, 4]
    assert visible_slots(10, 1, 0, window=3).tolist() == [7, 8, 9]
    assert visible_slots(10, 1, 0, window=3, sinks=2).tolist() == [0, 1, 7, 8, 9]
    assert visible_slots(4, 1, 0, window=3, sinks=9).tolist() == [0, 1, 2, 3]
    assert visible_slots(1, 3, 0).tolist() == [] and visible_slots(1, 3, 2).tolist() == [0]
    assert visible_slots(0, 1, 0, window=4, sinks=4).tolist() == []


def test_verify_hand_examples():
    p, q = np.log([[0.1, 0.6, 0.3]] * 2), np.log([[0.5, 0.25, 0.25]] * 2)
    # token 0: accepted with probability 0.1 / 0.5
    for u, want in ((0.19, 1), (0.21, 0)):
        acc, nxt, prob = verify_f64(p, q, [0, 0], [u, 0], [0.5], [0, 2])
        assert acc.tolist() == [want] and np.allclose(prob, [0.2, 1.0])
    # the rest is (0, 0.35, 0.05): token 1 up to 7/8 of it
    assert verify_f64(p, q, [0, 0], [0.9, 0], [0.87], [0, 2])[1].tolist() == [1]
    assert verify_f64(p, q, [0, 0], [0.9, 0], [0.88], [0, 2])[1].tolist() == [2]
    # all accepted: the last row's own probabilities
    assert verify_f64(p, q, [1, 0], [0.99, 0], [0.05], [0, 2])[:2] == (np.array([1]), np.array([0]))
    # one-hot draft: token 1 refused, the rest is p without it
    acc, nxt, prob = verify_f64(p, None, [1, 0], [0.7, 0], [0.2], [0, 2])
    assert acc[0] == 0 and nxt[0] == 0 and np.isclose(prob[0], 0.6)
    assert verify_f64(p, None, [1, 0], [0.7, 0], [0.3], [0, 2])[1][0] == 2
    # greedy
    acc, nxt, prob = verify_f64(p, q, [1, 0], [0.99, 0], [0.0], [0, 2], [0.0])
    assert acc[0] == 1 and nxt[0] == 1 and prob.tolist() == [1.0, 1.0]


def test_verify_leaves_the_target_distribution():
    # over the drafts and numbers, the first token is distributed as the target says
    rng = np.random.default_rng(5)
    x, y = rng.standard_normal((2, 1, 6))
    p, q = softmax_f64(x[0]), softmax_f64(y[0])
    n = 200
    got = np.zeros(6)
    for t in range(6):
        for i in range(n):
            for j in (0.1, 0.3, 0.5, 0.7, 0.9):
                acc, nxt, _ = verify_f64(np.stack([x[0]] * 2), np.stack([y[0]] * 2), [t, 0], [(i + 0.5) / n, 0], [j], [0, 2])
                got[t if acc[0] else nxt[0]] += q[t] / n / 5
    assert np.abs(got - p).max() < 0.05   # five points of the second number


def test_verify_marks_rows_without_a_distribution():
    x = np.full((2, 4), -np.inf)
    acc, nxt, prob = verify_f64(x, None, [1, 0], [0.0, 0], [0.5], [0, 2])
    assert acc[0] == 0 and nxt[0] == -1 and prob.tolist() == [0.0, 0.0]
    acc, nxt, _ = verify_f64(x, None, [], [], [0.5], [0, 0])
    assert acc[0] == 0 and nxt[0] == -1

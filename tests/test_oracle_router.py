"""The oracle of the router (FORMAT F27, F28) against closed forms, a brute force over subsets, and
central differences."""

import itertools
import math

import numpy as np
import pytest

import oracle


def test_scores_closed_forms():
    assert np.allclose(oracle.router_scores([0.0, 0.0, 0.0, 0.0], "softmax"), 0.25)
    assert np.allclose(oracle.router_scores([math.log(1), math.log(3)], "softmax"), [0.25, 0.75])
    assert np.allclose(oracle.router_scores([0.0, math.log(3), -math.inf], "sigmoid"), [0.5, 0.75, 0.0])
    assert np.all(oracle.router_scores([-math.inf] * 3, "softmax") == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_the_choice_has_the_largest_sum_of_all_subsets(score):
    rng = np.random.default_rng(5)
    for _ in range(20):
        x, b = rng.standard_normal(7), 0.3 * rng.standard_normal(7)
        c = oracle.router_scores(x, score) + b
        ids, _ = oracle.route_row(x, 3, score=score, bias=b)
        best = max(itertools.combinations(range(7), 3), key=lambda e: sum(c[list(e)]))
        assert sorted(ids) == list(best) and list(c[ids]) == sorted(c[ids], reverse=True)


def test_groups_by_hand():
    x = [0.1, 0.9, 0.5, 0.55, 0.8, -1.0, 0.2, 0.3]  # four groups of two
    assert list(oracle.route_row(x, 2, groups=4, group_topk=1)[0]) == [1, 0]
    assert list(oracle.route_row(x, 2, groups=4, group_topk=2)[0]) == [1, 4]
    # by sums of two scores the group (2, 3) is ahead of (4, 5)
    assert list(oracle.route_row(x, 4, score="sigmoid", groups=4, group_topk=2, group_top=2)[0]) == [1, 3, 2, 0]


def test_ties_and_missing_experts():
    assert list(oracle.route_row([1.0, 2.0, 2.0, 1.0], 3)[0]) == [1, 2, 0]
    ids, w = oracle.route_row([-math.inf, 0.0, -math.inf, 1.0], 3, renorm=False)
    assert list(ids) == [3, 1, -1] and w[2] == 0 and math.isclose(w[0] + w[1], 1.0)
    ids, w = oracle.route_row([-math.inf] * 4, 2)
    assert list(ids) == [-1, -1] and list(w) == [0, 0]
    ids, w = oracle.route_row([0.0, math.nan, 1.0], 2)
    assert list(ids) == [0, 1] and np.all(np.isnan(w))


def test_renormalised_weights_do_not_underflow():
    ids, w = oracle.route_row([-2000.0, -2000.0 + math.log(3), -math.inf], 2, score="sigmoid", scale=2.0)
    assert list(ids) == [1, 0] and np.allclose(w, [1.5, 0.5])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_central_differences(score, renorm):
    rng = np.random.default_rng(7)
    kw = dict(score=score, renorm=renorm, scale=2.5)
    x, dw = rng.standard_normal((4, 9)), rng.standard_normal((4, 3))
    ids, _ = oracle.expert_route(x, 3, **kw)

    def loss(z):
        total = 0.0
        for t in range(4):
            s = oracle.router_scores(z[t], score)[ids[t]]
            total += 2.5 * np.sum(dw[t] * (s / np.sum(s) if renorm else s))
        return total

    got = oracle.expert_route_backward(x, ids, dw, **kw)
    for t, e in itertools.product(range(4), range(9)):
        h = np.zeros_like(x)
        h[t, e] = 1e-5
        # the error of a central difference: h^2 / 6 of a third derivative of order 10
        assert abs((loss(x + h) - loss(x - h)) / 2e-5 - got[t, e]) < 1e-8


@pytest.mark.parametrize("score,x", [("sigmoid", [40.0, 39.0, 60.0, 59.0]), ("softmax", [0.0, -900.0, -950.0, -901.0, -890.0, -960.0])])
def test_groups_whose_scores_round_together(score, x):
    """1 / (1 + e^-40) and 1 / (1 + e^-60) are 1 in 64 bits, e^-890 is 0: without a bias and by one score the
    groups go by their logits, as the experts do; sums of two scores tie, and go by the lowest index."""
    n = len(x) // 2
    order = sorted(range(n), key=lambda g: -max(x[2 * g:2 * g + 2]))
    for keep in range(1, n):
        ids, _ = oracle.route_row(x, 2 * keep, score=score, groups=n, group_topk=keep)
        assert {e // 2 for e in ids} == set(order[:keep])
        ids, _ = oracle.route_row(x, 2 * keep, score=score, groups=n, group_topk=keep, group_top=2)
        assert {e // 2 for e in ids} == set(range(keep))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_of_undefined_rows(score, renorm):
    """Logits that no slot names count under softmax without renorm alone."""
    x = np.zeros((6, 6))
    x[0, 4], x[1, 4], x[2, 4], x[3, 4], x[5, 1] = math.nan, math.inf, math.nan, -math.inf, math.nan
    ids = np.array([[0, 1], [0, 1], [-1, -1], [0, 1], [0, 1], [0, 1]])
    dw = np.array([[1.0, 3.0]] * 6)
    got = oracle.expert_route_backward(x, ids, dw, score=score, renorm=renorm)
    assert np.all(got[2] == 0) and np.all(np.isfinite(got[3:5]))
    if score == "softmax" and not renorm:
        assert np.all(np.isnan(got[[0, 1, 5]]))
    else:
        assert np.array_equal(got[0], got[4]) and np.array_equal(got[1], got[4])
        assert np.isnan(got[5, 1]) and np.all(got[5, 2:] == 0)
        # softmax and sigmoid of two equal logits, 1/2 each
        want = [-0.5, 0.5] if score == "softmax" else [-0.25, 0.25] if renorm else [0.25, 0.75]
        assert np.allclose(got[4, :2], want) and np.all(got[4, 2:] == 0)

"""The oracle's choice of experts, importances and dense product against
hand-worked values, closed forms and exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import linear as oln
from oracle import select as osel

INF = float("inf")


def test_softmax_scores_by_hand():
    l = np.log(np.array([[1.0, 2.0, 5.0], [3.0, 3.0, 2.0]]))
    assert np.allclose(osel.scores(l, "softmax"), [[1 / 8, 2 / 8, 5 / 8], [3 / 8, 3 / 8, 2 / 8]], rtol=1e-15)
    ids, w = osel.select_experts(l, 2)
    assert ids.tolist() == [[2, 1], [0, 1]]                      # the tie goes to the lower index
    assert np.allclose(w, [[5 / 7, 2 / 7], [1 / 2, 1 / 2]], rtol=1e-15)
    _, w = osel.select_experts(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [[10 / 8, 4 / 8], [6 / 8, 6 / 8]], rtol=1e-15)
    assert np.allclose(osel.expert_importance(l), [1 / 4, 5 / 16, 7 / 16], rtol=1e-15)


def test_sigmoid_scores_by_hand():
    l = np.log(np.array([[1.0, 3.0, 1 / 3]]))
    assert np.allclose(osel.scores(l, "sigmoid"), [[1 / 2, 3 / 4, 1 / 4]], rtol=1e-15)
    ids, w = osel.select_experts(l, 2, bias=np.array([0.0, 0.0, 0.6]), score="sigmoid")
    assert ids.tolist() == [[2, 1]]                              # 0.85, 0.75: chosen with the bias
    assert np.allclose(w, [[1 / 4, 3 / 4]], rtol=1e-15)          # weighted without it


def test_groups_by_hand():
    # keys in groups of 3: (5 0 0) (3 3 0) (4 1 0)
    key = np.array([[5.0, 0, 0, 3, 3, 0, 4, 1, 0]])
    pick = lambda keep, how: osel.select_experts(key, 3, n_groups=3, keep_groups=keep, group_score=how)[0][0].tolist()
    assert pick(1, "max") == [0, 1, 2]
    # softmax scores of the logits: group 0 holds the largest score, and the largest sum of two
    assert pick(2, "max") == [0, 6, 7]
    assert pick(2, "top2") == [0, 6, 7]
    bias = np.array([0.0, 0, 0, 10, 10, 0, 0, 0, 0])
    ids, _ = osel.select_experts(key, 3, bias=bias, score="sigmoid", n_groups=3, keep_groups=1)
    assert ids[0].tolist() == [3, 4, 5]


def test_masked_and_broken_rows():
    l = np.array([[-INF, 0.0, -INF, 0.0], [-INF] * 4, [np.nan, 1.0, 2.0, 3.0], [INF, 0.0, 0.0, 0.0]])
    ids, w = osel.select_experts(l, 3)
    assert ids.tolist() == [[1, 3, 0], [0, 1, 2], [3, 2, 1], [0, 1, 2]]
    assert w[0].tolist() == [0.5, 0.5, 0.0] and w[1].tolist() == [0.0] * 3
    assert np.isnan(w[2]).all() and np.isnan(w[3]).all()
    ids, w = osel.select_experts(l, 2, score="sigmoid", renormalize=False)
    assert w[3].tolist() == [1.0, 0.5] and w[1].tolist() == [0.0, 0.0]
    # a bias of -inf bars an expert
    ids, _ = osel.select_experts(l[:1], 2, bias=np.array([0.0, -INF, 0.0, 0.0]))
    assert ids[0].tolist() == [3, 0]


def test_sigmoids_below_every_float_keep_their_ratios():
    # e^-900 and e^-901 are below float64's smallest: s_1 / s_0 = 1 / e
    _, w = osel.select_experts(np.array([[-900.0, -901.0, -3e38, -INF]]), 4, score="sigmoid")
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1)), 0.0, 0.0]], rtol=1e-14)
    _, w = osel.select_experts(np.full((1, 8), -3e38), 8, score="sigmoid")
    assert (w == 0.125).all()
    # next to 0 both ways of writing it agree
    l = np.array([[-1e-3, -2.0, -30.0]])
    _, w = osel.select_experts(l, 3, score="sigmoid")
    s = osel.scores(l, "sigmoid")
    assert np.allclose(w, s / s.sum(), rtol=1e-14)


def test_every_group_kept_is_the_ungrouped_choice():
    rng = np.random.default_rng(3)
    l = rng.normal(size=(20, 24))
    for score in ("softmax", "sigmoid"):
        a = osel.select_experts(l, 5, score=score)
        b = osel.select_experts(l, 5, score=score, n_groups=6, keep_groups=6)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_linear_against_rationals():
    rng = np.random.default_rng(5)
    x, w = rng.integers(-4, 5, (3, 7)) / 4.0, rng.integers(-4, 5, (6, 7)) / 8.0
    b, r = rng.integers(-8, 9, 6) / 16.0, rng.integers(-8, 9, (3, 6)) / 4.0
    want = [[sum(Fraction(float(x[m, k])) * Fraction(float(w[n, k])) for k in range(7)) + Fraction(float(b[n]))
             + Fraction(float(r[m, n])) for n in range(6)] for m in range(3)]
    assert oln.linear(x, w, b, residual=r).tolist() == [[float(v) for v in row] for row in want]
    g = oln.linear(x, w, b, "relu", gated=True, residual=r[:, :3])
    pre = oln.preactivation(x, w, b)
    assert g.tolist() == (np.maximum(pre[:, :3], 0) * pre[:, 3:] + r[:, :3]).tolist()


@pytest.mark.parametrize("act,at_one,at_minus_one", [
    ("none", 1.0, -1.0), ("relu", 1.0, 0.0),
    ("silu", 0.7310585786300049, -0.2689414213699951),       # 1 / (1 + 1/e)
    ("gelu", 0.8413447460685429, -0.15865525393145707),      # the normal distribution's Phi(1)
    ("gelu_tanh", 0.8411919906082768, -0.15880800939172324)])
def test_activations(act, at_one, at_minus_one):
    got = oln.activate(np.array([1.0, -1.0, 0.0, 40.0, -1000.0]), act)
    assert np.allclose(got[:2], [at_one, at_minus_one], rtol=1e-14)
    assert got[2] == 0.0 and got[3] == 40.0
    assert got[4] == (-1000.0 if act == "none" else 0.0)

"""The routing's and the adapters' oracle against what can be said by hand."""
import numpy as np
import pytest

from oracle import serve_oracle as S


def test_route_by_hand():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w = S.route(l, 2)
    assert ids.tolist() == [[1, 2]]
    np.testing.assert_allclose(w, [[4 / 6, 2 / 6]])
    ids, w = S.route(l, 2, renormalize=False, scale=8.0)
    np.testing.assert_allclose(w, [[4.0, 2.0]])
    # a balance moves the choice and leaves the scores
    ids, w = S.route(l, 2, balance=np.array([0.3, 0.0, 0.0, 0.0]), renormalize=False, scale=8.0)
    assert ids.tolist() == [[1, 0]]
    np.testing.assert_allclose(w, [[4.0, 1.0]])


def test_route_ties_and_masked():
    ids, _ = S.route(np.zeros((1, 5)), 3, scoring="sigmoid")
    assert ids.tolist() == [[0, 1, 2]]
    l = np.array([[np.nan, -np.inf, 0.0, -np.inf, np.inf]])
    ids, w = S.route(l, 5, scoring="sigmoid", renormalize=False)
    assert ids.tolist() == [[4, 2, 1, 3, 0]]
    np.testing.assert_array_equal(w[0, :4], [1.0, 0.5, 0.0, 0.0])
    assert np.isnan(w[0, 4])


def test_route_groups():
    v = np.array([[0.9, 0.0, 0.5, 0.6, 0.1, 0.2, 0.8, 0.0]])
    kw = dict(scoring="sigmoid", balance=np.zeros(8), groups=4)
    l = np.log(np.maximum(v, 1e-9) / (1 - np.maximum(v, 1e-9)))
    assert S.route(l, 2, topk_groups=2, group_score="max", **kw)[0].tolist() == [[0, 6]]
    assert S.route(l, 2, topk_groups=2, group_score="top2", **kw)[0].tolist() == [[0, 3]]
    assert S.route(l, 3, topk_groups=1, group_score="top2", **(kw | dict(groups=2)))[0].tolist() == [[0, 3, 2]]


def test_lora_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 0.0], [0.0, 1.0]], [[1.0, 1.0], [9.0, 9.0]]])
    b = np.array([[[1.0, 10.0]], [[2.0, 7.0]]])
    y, mag, peak = S.lora(x, a, b, [1, 0, -1], base=np.full((3, 1), 100.0), scales=[2.0, 0.5], ranks=[2, 1])
    assert y.tolist() == [[103.0], [186.0], [100.0]]
    assert mag.tolist() == [[3.0], [86.0], [0.0]] and peak.tolist() == [[3.0], [88.0], [0.0]]
    assert S.lora(x, a, b, [2, 5, -7])[0].tolist() == [[0.0], [0.0], [0.0]]


@pytest.mark.parametrize("bias", [False, True])
def test_logits(bias):
    x, w = np.array([[1.0, -2.0]]), np.array([[3.0, 1.0], [0.5, 0.25]])
    c = np.array([1.0, -1.0]) if bias else None
    y, mag = S.logits(x, w, c)
    assert y.tolist() == [[2.0, -1.0]] if bias else [[1.0, 0.0]]
    assert mag.tolist() == [[6.0, 2.0]] if bias else [[5.0, 1.0]]

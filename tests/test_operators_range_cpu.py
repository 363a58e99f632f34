"""The oracle's routing where scores are tiny or huge, without a GPU."""

import numpy as np

from oracle import operators as ops


def test_group_score_is_relative():
    """Sums keep 40 binary places below their larger term: small ones are told
    apart, and sums equal but for binary64's last bits are one number."""
    assert ops.group_score([2.0 ** -60, 2.0 ** -61]) == 1.5 * 2.0 ** -60
    assert ops.group_score([1e-26, 1e-26]) > ops.group_score([1e-26, 0.9e-26]) > 0
    assert ops.group_score([0.5, 0.5]) == ops.group_score([0.5 + 2.0 ** -53, 0.5]) == 1.0
    assert ops.group_score([0.75, 0.25 + 2.0 ** -54]) == 1.0 == ops.group_score([1 - 2.0 ** -53])
    assert ops.group_score([0.0]) == 0.0 and ops.group_score([np.inf, 1.0]) == np.inf
    assert ops.group_score([5e-324]) == 5e-324 and ops.group_score([-3.0, -4.0]) == -7.0


def test_groups_of_small_scores():
    z = np.full((1, 16), -60.0)
    z[0, 8:] = -30.0
    ids, w = ops.route(z, 2, n_group=2, topk_group=1)
    assert ids.tolist() == [[8, 9]] and w.tolist() == [[0.5, 0.5]]
    ids, _ = ops.route(z, 2, n_group=2, topk_group=1, score=ops.SOFTMAX)
    assert ids.tolist() == [[8, 9]]


def test_the_bias_leaves_the_scores_alone():
    z = np.array([[5.0, 1.0, 0.0, -1.0]])
    bias = np.array([-np.inf, 0.0, np.nan, 0.0])
    ids, w = ops.route(z, 2, bias=bias, score=ops.SOFTMAX, renormalize=False)
    assert ids.tolist() == [[1, 3]]
    assert np.allclose(w, np.exp(z[:, [1, 3]]) / np.exp(z).sum(), rtol=1e-14)
    assert np.allclose(w, ops.route_weights(z, ids, ops.SOFTMAX, False, 1.0), rtol=1e-14)

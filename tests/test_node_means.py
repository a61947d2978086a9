"""The bounds of node_means tell right sums from wrong ones: float32 restatements with sums about the
means stay within them at every width; sums that keep a mean, or are differences of larger sums, do
not."""

import numpy as np
import pytest

import node_means as nm
from oracle import node

WIDTHS = [96, 1024, 2048, 4096, 3999, 9001]
BOTH, SMALL, X_ONLY = 0, 4, 3   # rows by kind: means of x and of the gradient large, none, x's alone


def _ratios(S, mode):
    R, kind, x, w, gy = nm.scalar_problem(S, 60)
    h, gx = nm.restated(x, w, gy, mode)
    y_ratio = np.abs(w * h - node.norm_forward(R, x, w, np.zeros(S))) / nm.forward_bound(R, x, w, np.zeros(S))
    gx_ratio = np.abs(gx - node.norm_backward(R, x, w, gy)[0]) / nm.backward_bound(R, x, w, gy)[0]
    return kind, y_ratio, gx_ratio


@pytest.mark.parametrize("S", WIDTHS)
def test_right_sums_are_within_the_bounds(S):
    _, y, gx = _ratios(S, "right")
    assert y.max() <= 1 and gx.max() <= 1


@pytest.mark.parametrize("S", WIDTHS)
def test_sums_with_a_mean_left_are_not(S):
    kind, _, gx = _ratios(S, "uncentred")
    assert gx[kind == BOTH].max() > 4 and (gx[kind == BOTH].max(axis=1) > 1).mean() > 0.5
    assert gx[kind == SMALL].max() <= 1


@pytest.mark.parametrize("S", WIDTHS)
def test_differences_of_large_sums_are_not(S):
    kind, y, gx = _ratios(S, "difference")
    for k in (BOTH, X_ONLY):
        assert y[kind == k].max() > 4 and gx[kind == k].max() > 4
    assert y[kind == SMALL].max() <= 1 and gx[kind == SMALL].max() <= 1


@pytest.mark.parametrize("S", WIDTHS)
def test_bounds_are_below_the_values(S):
    """A bound that a zero or a doubled gradient passes shows nothing."""
    R, kind, x, w, gy = nm.scalar_problem(S, 60)
    ratio = np.abs(node.norm_backward(R, x, w, gy)[0]) / nm.backward_bound(R, x, w, gy)[0]
    assert (ratio > 2).mean() > 0.95 and np.median(ratio) > 20

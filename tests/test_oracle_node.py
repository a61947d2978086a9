"""Pins for the oracle's node-feature operators (oracle/node.py).

* Philox4x32-10 against the known-answer vectors published with the generator;
* norm: closed form on two elements, O(3) equivariance of the forward (rotations and
  reflections), invariance under rescaling as eps -> 0, zero mean and unit mean square;
* backward and double backward against central differences;
* dropout: keep frequency, expectation, equivariance (a channel's components share a mask),
  independence of the layout.
"""

import numpy as np
import pytest
from scipy.spatial.transform import Rotation

from oracle import node
from test_oracle_conv import _act

IRREPS = ["5x0e+3x1o+2x2e", "4x0o+3x0e+2x1e+1x3o"]


def _case(irreps, layout, n=4, seed=3):
    R = node.Rows(irreps, layout)
    g = np.random.default_rng(seed)
    return R, g, g.normal(size=(n, R.dim)) + 0.3, 1 + 0.3 * g.normal(size=R.channels), g.normal(size=R.biases)


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, words):
    assert tuple(node.philox4x32(counter, key)) == words


def test_norm_closed_form():
    R = node.Rows("2x0e+1x1o", eps=1e-3)
    y = node.norm_forward(R, [[3.0, 1.0, 0.0, 4.0, 3.0]], np.array([2.0, 5.0, 3.0]), np.array([0.5, -1.0]))
    s, v = 1 / np.sqrt(1 + 1e-3), 1 / np.sqrt(25 / 3 + 1e-3)
    assert np.allclose(y, [[0.5 + 2 * s, -1 - 5 * s, 0.0, 12 * v, 9 * v]], rtol=1e-14)


@pytest.mark.parametrize("irreps", IRREPS)
@pytest.mark.parametrize("improper", [False, True])
def test_norm_o3_equivariant(irreps, improper, rng):
    R, _, x, w, b = _case(irreps, "ir_mul")
    M = Rotation.random(random_state=1).as_matrix() * (-1 if improper else 1)
    R0, det = M * np.sign(np.linalg.det(M)), np.linalg.det(M)
    a = node.norm_forward(R, _act(R.blocks, x, R0, det, rng), w, b)
    assert np.abs(a - _act(R.blocks, node.norm_forward(R, x, w, b), R0, det, rng)).max() < 1e-10


@pytest.mark.parametrize("irreps", IRREPS)
def test_norm_statistics_and_scale(irreps):
    R, _, x, _, _ = _case(irreps, "mul_ir")
    R.eps = 1e-30
    one, zero = np.ones(R.channels), np.zeros(R.biases)
    y = node.norm_forward(R, x, one, zero)
    assert np.allclose(node.norm_forward(R, 37.0 * x, one, zero), y, rtol=1e-12)
    for b, v in zip(R.blocks, R.parts(y)):
        assert np.allclose((v * v).mean(axis=(1, 2)), 1.0)
        if R.centred(b):
            assert np.abs(v.mean(axis=(1, 2))).max() < 1e-14


@pytest.mark.parametrize("irreps", IRREPS)
@pytest.mark.parametrize("layout", ["ir_mul", "mul_ir"])
def test_gradients_match_differences(irreps, layout):
    R, g, x, w, b = _case(irreps, layout)
    gy, p = g.normal(size=x.shape), g.normal(size=x.shape)
    s, t = g.normal(size=w.shape), g.normal(size=b.shape)
    gx, gw, gb = node.norm_backward(R, x, w, gy)
    f = lambda x, w, b: (gy * node.norm_forward(R, x, w, b)).sum()  # noqa: E731
    d = 1e-6
    assert (f(x + d * p, w, b) - f(x - d * p, w, b)) / (2 * d) == pytest.approx((gx * p).sum(), rel=1e-7)
    assert (f(x, w + d * s, b) - f(x, w - d * s, b)) / (2 * d) == pytest.approx((gw * s).sum(), rel=1e-7)
    assert (f(x, w, b + d * t) - f(x, w, b - d * t)) / (2 * d) == pytest.approx((gb * t).sum(), rel=1e-7)

    def lam(x, w, gy):
        a, c, e = node.norm_backward(R, x, w, gy)
        return (a * p).sum() + (c * s).sum() + (e * t).sum()

    ex, ew, eg = node.norm_double_backward(R, x, w, gy, p, s, t)
    dx, dw, dg = g.normal(size=x.shape), g.normal(size=w.shape), g.normal(size=x.shape)
    assert (lam(x + d * dx, w, gy) - lam(x - d * dx, w, gy)) / (2 * d) == pytest.approx((ex * dx).sum(), rel=1e-6)
    assert (lam(x, w + d * dw, gy) - lam(x, w - d * dw, gy)) / (2 * d) == pytest.approx((ew * dw).sum(), rel=1e-6)
    assert (lam(x, w, gy + d * dg) - lam(x, w, gy - d * dg)) / (2 * d) == pytest.approx((eg * dg).sum(), rel=1e-6)


def test_dropout_frequency_and_expectation():
    R = node.Rows("64x0e+16x1o")
    m = node.dropout_mask(R, 100, 0.3, seed=0x123456789ABCDEF, offset=5)
    kept = (R.parts(m)[0] > 0).mean()
    assert abs(kept - 0.7) < 5 * np.sqrt(0.21 / 6400)     # five standard deviations of 6400 draws
    assert set(np.unique(m)) == {0.0, 1 / 0.7}
    v = R.parts(m)[1]
    assert np.array_equal(v[:, 0], v[:, 1]) and np.array_equal(v[:, 0], v[:, 2])
    assert np.array_equal(node.dropout_mask(R, 3, 0.0, 1), np.ones((3, R.dim)))
    assert np.array_equal(node.dropout_mask(R, 3, 1.0, 1), np.zeros((3, R.dim)))


def test_dropout_layouts_share_the_mask():
    a, b = node.Rows("5x0e+6x1o"), node.Rows("5x0e+6x1o", "mul_ir")
    for u, v in zip(a.parts(node.dropout_mask(a, 7, 0.5, 9)), b.parts(node.dropout_mask(b, 7, 0.5, 9))):
        assert np.array_equal(u, v)

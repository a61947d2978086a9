"""Layer norm on the GPU where means are large (of x, of grad_y, of both): every output of forward and
backward within the bounds of node_means, in groups of lanes, groups of several warps, whole CTAs and
segments read again for each sum; through the passes fused with dropout and the residual sum as well."""

import numpy as np
import pytest

import node_means as nm
from node_helpers import Problem, U, half_step, stored
from oracle import node

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def _problem(irreps, n, dtype="float32"):
    """A Problem with unit spreads and the means of node_means, and its grad_y."""
    p = Problem(irreps, n, dtype, offset=0.0)
    _, mx, mg = nm.offsets(p.R, n)
    if dtype != "float32":           # a spread of one has to survive storage
        mx, mg = mx / 16, mg / 16
    g = np.random.default_rng(11)
    p.x, p.x64 = stored(g.normal(size=mx.shape) + mx, dtype)
    return (p,) + stored(g.normal(size=mx.shape) + mg, dtype)


def _within(got, ref, bound, dtype="float32", what=""):
    got = got.double().cpu().numpy()
    bound = bound + half_step(dtype) * (np.abs(ref) + bound) + (2.0 ** -24 if dtype == "float16" else 1e-37)
    ratio = np.abs(got - ref) / bound
    assert np.all(ratio <= 1), (what, float(np.nanmax(ratio)), int((~(ratio <= 1)).sum()))


def _check_backward(p, x64, gy64, got, dtype="float32"):
    bounds = nm.backward_bound(p.R, x64, p.w64, gy64)
    refs = node.norm_backward(p.R, x64, p.w64, gy64)
    for g, ref, bound, name in zip(got, refs, bounds, ("grad_x", "grad_weight", "grad_bias")):
        _within(g, ref, bound, dtype if name == "grad_x" else "float32", name)


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("irreps,n", nm.SHAPES)
def test_forward_and_backward(irreps, n, dtype):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p, gy, gy64 = _problem(irreps, n, dtype)
    y = B.tpconv_norm_forward(p.plan, p.x, p.w, p.b)
    _within(y, node.norm_forward(p.R, p.x64, p.w64, p.b64), nm.forward_bound(p.R, p.x64, p.w64, p.b64), dtype, "y")
    _check_backward(p, p.x64, gy64, B.tpconv_norm_backward(p.plan, p.x, p.w, gy), dtype)


@pytest.mark.parametrize("irreps,n", nm.SHAPES)
def test_fused_with_dropout_and_residual(irreps, n):
    """The residual's mean is the large one; y is the norm of the sum before it is stored (in float32
    the same), the backward starts from the stored z."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p, gy, gy64 = _problem(irreps, n)
    g = np.random.default_rng(12)
    x, x64 = stored(g.normal(size=p.x64.shape), "float32")
    drop = B.Dropout(0.25, 9, 2)
    mask = node.dropout_mask(p.R, n, 0.25, 9, 2)
    z, y = B.tpconv_dropout_norm_forward(p.plan, x, drop, residual=p.x, weight=p.w, bias=p.b)
    z64 = p.x64 + mask * x64
    e0 = 3 * U * (np.abs(mask * x64) + np.abs(z64))   # the scale, the product, the sum
    _within(z, z64, e0, what="z")
    _within(y, node.norm_forward(p.R, z64, p.w64, p.b64), nm.forward_bound(p.R, z64, p.w64, p.b64, e0), what="y")
    gx, gr, gw, gb = B.tpconv_dropout_norm_backward(p.plan, z, p.w, gy, drop)
    zz = z.double().cpu().numpy()
    _check_backward(p, zz, gy64, (gr, gw, gb))
    assert np.all((gx.cpu().numpy() == 0) >= (mask == 0))
    # grad_x = mask * grad_residual: the scale's and the product's rounding
    _within(gx, mask * gr.double().cpu().numpy(), 3 * U * np.abs(mask * gr.double().cpu().numpy()), what="grad_x")


@pytest.mark.parametrize("S", [96, 1001, 1024, 2048, 4096, 3999, 9001])
@pytest.mark.parametrize("fused", [False, True])
def test_sums_beyond_the_range_about_zero_but_not_about_the_mean(S, fused):
    """Rows whose sum of squares passes float32's range while that about the mean does not, and in the
    backward also the sum of products with the gradient: the same values whatever holds the row."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    n = 24
    p = Problem(f"{S}x0e", n)
    g = np.random.default_rng(3)
    s = np.sqrt(1.2e38 / S)          # S s^2 = 1.2e38, S (s^2 + mean^2) = 5.5e38
    p.x, p.x64 = stored(s * (np.clip(g.normal(size=(n, S)), -3, 3) + 1.9), "float32")
    one, w64 = np.ones(S), np.ones(S)
    for mean in (0.0, 20 * s):       # with the second, S mean(x) mean(grad) = 4.6e39
        gy, gy64 = stored(mean + 0.05 * s * np.clip(g.normal(size=(n, S)), -3, 3), "float32")
        if mean == 0.0:
            gy, gy64 = stored(g.normal(size=(n, S)), "float32")
        if fused:
            got = B.tpconv_dropout_norm_backward(p.plan, p.x, None, gy, B.Dropout(0.0, 1))[1:]
            y = B.tpconv_dropout_norm_forward(p.plan, p.x, B.Dropout(0.0, 1))[1]
        else:
            got = B.tpconv_norm_backward(p.plan, p.x, None, gy)
            y = B.tpconv_norm_forward(p.plan, p.x)
        zero = np.zeros(S)
        _within(y, node.norm_forward(p.R, p.x64, one, zero), nm.forward_bound(p.R, p.x64, one, zero), what="y")
        refs, bounds = node.norm_backward(p.R, p.x64, w64, gy64), nm.backward_bound(p.R, p.x64, w64, gy64)
        for a, ref, bound, name in zip(got, refs, bounds, ("grad_x", "grad_weight", "grad_bias")):
            _within(a, ref, bound, what=name)

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

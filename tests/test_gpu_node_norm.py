"""Irreps layer norm on the GPU: forward, backward, double backward against the float64 oracle
(tolerances derived in node_helpers), over types, layouts, widths from one element to more than a
block holds, one row to many, odd sizes, degenerate rows, and the ways a call can be made
(capture and replay, another stream, no weight, missing outputs, poisoned workspace)."""

import numpy as np
import pytest

from node_helpers import TYPES, Problem, assert_near, stored, tol32
from oracle import node

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


MIXED, ODD = "128x0e+64x1o+32x2e+16x3o", "37x0e+19x1o+6x2e+3x3o"
SHAPES = [("8x0e+8x1o+8x2e", 64), (MIXED, 300), (ODD, 33), ("1x0e", 5), ("1x1o", 5), ("2x0o+3x0e+1x1e", 7),
          ("4096x0e", 9), ("1023x0e", 3), ("12x0e+12x1o", 1), ("600x1o+5x0e", 6), ("5x3o", 4000), ("64x0e", 3001),
          ("128x0e+128x1o+128x2e", 700), ("10000x0e+8x1o", 3), ("20001x0e", 2), ("9000x2e", 2)]


def _all_passes(p):
    """Runs every pass and checks every output."""
    from equivariant_gnn_tensor_dst_b200 import binding
    R, tol = p.R, tol32(p.R)
    y = binding.tpconv_norm_forward(p.plan, p.x, p.w, p.b)
    assert_near(y, node.norm_forward(R, p.x64, p.w64, p.b64), p.forward_scale(p.x64), tol, p.dtype, "y")
    gy, gy64 = p.rows()
    gx, gw, gb = binding.tpconv_norm_backward(p.plan, p.x, p.w, gy)
    ex, ew, eb = node.norm_backward(R, p.x64, p.w64, gy64)
    sx, sw = p.backward_scale(p.x64, gy64)
    assert_near(gx, ex, sx, tol, p.dtype, "grad_x")
    assert_near(gw, ew, sw, p.sum_tol(), what="grad_weight")
    sb = np.concatenate([np.zeros(0)] + [np.abs(v).sum(axis=(0, 1)) for b, v in zip(R.blocks, R.parts(gy64))
                                         if R.centred(b)])
    assert_near(gb, eb, sb, p.sum_tol(), what="grad_bias")
    (t, t64), (s, s64), (q, q64) = p.rows(), p.vector(R.channels), p.vector(R.biases)
    gx, gw, gg = binding.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, t, s, q)
    ex, ew, eg = node.norm_double_backward(R, p.x64, p.w64, gy64, t64, s64, q64)
    sx, sw, sg = p.double_scale(p.x64, gy64, t64, s64, q64)
    assert_near(gx, ex, sx, 2 * tol, p.dtype, "double grad_x")
    assert_near(gw, ew, sw, 2 * p.sum_tol(), what="double grad_weight")
    assert_near(gg, eg, sg, 2 * tol, p.dtype, "grad_grad_y")


@pytest.mark.parametrize("layout", ["ir_mul", "mul_ir"])
@pytest.mark.parametrize("irreps,n", SHAPES)
def test_shapes(irreps, n, layout):
    _all_passes(Problem(irreps, n, layout=layout))


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("irreps,n,layout", [(MIXED, 200, "ir_mul"), (ODD, 65, "mul_ir"), (ODD, 64, "ir_mul"),
                                             ("4096x0e", 40, "ir_mul"), ("64x0e+64x1o+64x2e", 333, "mul_ir"),
                                             ("1x0e+1x1o", 1, "ir_mul"), ("20001x0e", 2, "ir_mul"),
                                             ("8x0e+24x1o", 1000, "ir_mul")])
def test_16_bit(irreps, n, layout, dtype):
    _all_passes(Problem(irreps, n, dtype, layout))


def test_rows_beyond_one_launch_range():
    """More rows than any grid dimension of the launch."""
    _all_passes(Problem("4x0e", 70001))


def test_large_offset():
    """A mean a thousand times the spread: the spread is taken around the mean, not as a
    difference of squares."""
    from equivariant_gnn_tensor_dst_b200 import binding
    p = Problem("96x0e", 50, offset=1000.0)
    y = binding.tpconv_norm_forward(p.plan, p.x, p.w, p.b).double().cpu().numpy()
    ref = node.norm_forward(p.R, p.x64, p.w64, p.b64)
    # an error of 2^-24 of the mean (1000, of rows with spread e^-1.5 .. e^1.5) in every u, and the
    # mean's own sum, 20 additions deep at most
    assert np.abs(y - ref).max() <= 40 * 2.0 ** -24 * 1000 / np.exp(-1.5) * 2


def test_degenerate_rows(torch):
    """Constant, zero, huge, infinite and NaN rows; each touches its own block of its own row."""
    from equivariant_gnn_tensor_dst_b200 import binding
    p = Problem("16x0e+16x1o", 12)
    x = p.x.clone()
    x[1] = 0
    x[2, :16] = 3.0
    x[3] = 1e30                      # squares overflow: q = inf, r = 0
    x[4, 5] = float("nan")
    x[5, 20] = float("inf")
    x[6] = 1e-30
    clean = binding.tpconv_norm_forward(p.plan, p.x, p.w, p.b)
    y = binding.tpconv_norm_forward(p.plan, x, p.w, p.b)
    for i in (0, 7, 8, 9, 10, 11):
        assert torch.equal(y[i], clean[i])
    assert torch.equal(y[1, :16], p.b) and torch.equal(y[1, 16:], torch.zeros_like(y[1, 16:]))
    assert torch.equal(y[2, :16], p.b)
    assert torch.equal(y[3, 16:], torch.zeros_like(y[3, 16:]))
    assert torch.isnan(y[4, :16]).all() and torch.equal(y[4, 16:], clean[4, 16:])
    assert torch.equal(y[5, :16], clean[5, :16]) and torch.isnan(y[5, 20])
    assert torch.isfinite(y[6]).all()
    gy, gy64 = p.rows()
    gx, gw, gb = binding.tpconv_norm_backward(p.plan, x, p.w, gy)
    ref = binding.tpconv_norm_backward(p.plan, p.x, p.w, gy)[0]
    for i in (0, 7, 8, 9, 10, 11):
        assert torch.equal(gx[i], ref[i])
    assert torch.isfinite(gx[1]).all() and torch.isfinite(gx[2, :16]).all()


def test_optional_arguments(torch):
    """No weight and bias are ones and zeros; missing tangents are zeros; outputs are computed one
    by one as together."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, 50)
    one, zero = torch.ones_like(p.w), torch.zeros_like(p.b)
    assert torch.equal(B.tpconv_norm_forward(p.plan, p.x), B.tpconv_norm_forward(p.plan, p.x, one, zero))
    gy, _ = p.rows()
    full = B.tpconv_norm_backward(p.plan, p.x, one, gy)
    assert all(torch.equal(a, b) for a, b in zip(B.tpconv_norm_backward(p.plan, p.x, None, gy), full))
    for k, name in enumerate(("need_x", "need_weight", "need_bias")):
        need = dict(need_x=False, need_weight=False, need_bias=False)
        need[name] = True
        got = B.tpconv_norm_backward(p.plan, p.x, one, gy, **need)
        assert torch.equal(got[k], full[k]) and sum(g is None for g in got) == 2
    t, _ = p.rows()
    zx, zw, zb = torch.zeros_like(p.x), torch.zeros_like(p.w), torch.zeros_like(p.b)
    full = B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, t, zw, zb)
    assert all(torch.equal(a, b) for a, b in zip(B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, t), full))
    s, _ = p.vector(p.R.channels)
    a = B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, zx, s, zb)
    assert all(torch.equal(u, v) for u, v in zip(B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, gg_weight=s), a))
    for k, name in enumerate(("need_x", "need_weight", "need_grad_y")):
        need = dict(need_x=False, need_weight=False, need_grad_y=False)
        need[name] = True
        got = B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, t, **need)
        assert torch.equal(got[k], full[k]) and sum(g is None for g in got) == 2


@pytest.mark.parametrize("n", [1, 40, 2000])
def test_workspace_contents_do_not_matter(torch, n):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, n)
    gy, _ = p.rows()
    size = p.plan.workspace_bytes(n)
    got = []
    for fill in (0, 255):            # 255: every float a NaN
        ws = torch.full((size + 64,), fill, dtype=torch.uint8, device="cuda")
        guard = ws[size:].clone()
        got.append(B.tpconv_norm_backward(p.plan, p.x, p.w, gy, ws=ws[:size]))
        assert torch.equal(ws[size:], guard)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_no_rows(torch):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, 0)
    gw, gb = torch.full_like(p.w, 7.0), torch.full_like(p.b, 7.0)
    B.tpconv_norm_backward(p.plan, p.x, p.w, p.x, outputs=(None, gw, gb))
    assert not gw.any() and not gb.any()
    gw.fill_(7.0)
    B.tpconv_norm_double_backward(p.plan, p.x, p.w, p.x, p.x, outputs=(None, gw, None))
    assert not gw.any()
    assert B.tpconv_norm_forward(p.plan, p.x, p.w, p.b).shape == (0, p.plan.dim)


def test_rows_do_not_depend_on_each_other(torch):
    """A row's outputs are the same alone and among others, and nothing is written past the rows."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(ODD, 50)
    gy, _ = p.rows()
    y = B.tpconv_norm_forward(p.plan, p.x, p.w, p.b)
    gx = B.tpconv_norm_backward(p.plan, p.x, p.w, gy)[0]
    for i in (0, 4, 48):             # 4-row steps keep the rows' 16-byte alignment
        n = min(2, p.n - i)
        out = torch.full((n + 2, p.plan.dim), 5.0, device="cuda")
        B.tpconv_norm_forward(p.plan, p.x[i:i + n], p.w, p.b, out=out[:n])
        assert torch.equal(out[:n], y[i:i + n]) and bool((out[n:] == 5.0).all())
        assert torch.equal(B.tpconv_norm_backward(p.plan, p.x[i:i + n], p.w, gy[i:i + n])[0], gx[i:i + n])


def test_capture_replay_and_streams(torch):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, 500)
    (gy, _), (t, _), (s, _), (q, _) = p.rows(), p.rows(), p.vector(p.R.channels), p.vector(p.R.biases)
    ws = B.workspace(p.plan.workspace_bytes(p.n), p.x.device)
    E = torch.empty_like
    outs = [E(p.x), E(p.x), E(p.w), E(p.b), E(p.x), E(p.w), E(p.x)]

    def step():
        B.tpconv_norm_forward(p.plan, p.x, p.w, p.b, out=outs[0])
        B.tpconv_norm_backward(p.plan, p.x, p.w, gy, ws=ws, outputs=tuple(outs[1:4]))
        B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, t, s, q, ws=ws, outputs=tuple(outs[4:]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    ref = [o.clone() for o in outs]
    for stream in (None, torch.cuda.Stream()):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        y = B.tpconv_norm_forward(p.plan, p.x, p.w, p.b, out=outs[0], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    p.x.mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, outs)) and not torch.equal(got[1], ref[1])
    del graph


def test_64_bit_offsets(torch):
    """Rows beyond 2^31 elements (16 bits: 4.4 GB an array): the last rows equal the same rows alone."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    irreps, dim = "2048x0e", 2048
    n = (1 << 31) // dim + 40
    plan = B.NodePlan(irreps, torch.bfloat16)
    x = torch.randn(64, dim, device="cuda").to(torch.bfloat16).repeat(n // 64 + 1, 1)[:n].contiguous()
    gy = x.flip(1).contiguous()
    y = B.tpconv_norm_forward(plan, x)
    gx = B.tpconv_norm_backward(plan, x, None, gy, need_weight=False, need_bias=False)[0]
    tail = n - 40
    assert torch.equal(y[tail:], B.tpconv_norm_forward(plan, x[tail:].clone()))
    assert torch.equal(gx[tail:], B.tpconv_norm_backward(plan, x[tail:].clone(), None, gy[tail:].clone())[0])
    d = B.Dropout(0.5, 3)
    out = B.tpconv_dropout_forward(plan, x, d, out=y)
    kept = out[tail:] != 0
    assert torch.equal(out[tail:], torch.where(kept, 2 * x[tail:], torch.zeros_like(x[tail:])))
    assert 0.45 < kept.float().mean().item() < 0.55


def test_binding_checks(torch):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, 5000)
    gy, _ = p.rows()
    for bad in (lambda: B.tpconv_norm_forward(p.plan, p.x[:, :100]), lambda: B.tpconv_norm_forward(p.plan, p.x.half()),
                lambda: B.tpconv_norm_forward(p.plan, p.x.t().contiguous().t()),
                lambda: B.tpconv_norm_forward(p.plan, p.x, p.w[:-1]),
                lambda: B.tpconv_norm_forward(p.plan, p.x, p.w, p.w),
                lambda: B.tpconv_norm_forward(p.plan, p.x, p.w.double()),
                lambda: B.tpconv_norm_backward(p.plan, p.x, p.w, gy[:9]),
                lambda: B.tpconv_norm_backward(p.plan, p.x, p.w, gy, ws=torch.empty(9)),
                lambda: B.tpconv_norm_forward(p.plan, p.x[0])):
        with pytest.raises(ValueError):
            bad()
    for code, bad in ((1, lambda: B.tpconv_norm_forward(p.plan, p.x, out=p.x)),
                      (1, lambda: B.tpconv_norm_backward(p.plan, p.x, p.w, None)),
                      (4, lambda: B.tpconv_norm_backward(p.plan, p.x, p.w, gy,
                                                         ws=torch.empty(16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(B.TPConvError) as e:
            bad()
        assert e.value.status == code


def test_stored_rounding_is_to_nearest(torch):
    """The helper's storage rounding is torch's, the reference for half a step."""
    t, v = stored([1.0, 1.00390625, 1.01171875], "bfloat16")
    assert v.tolist() == [1.0, 1.0, 1.015625]

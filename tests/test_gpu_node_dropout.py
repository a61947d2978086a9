"""Equivariant dropout and the fused dropout + residual + norm on the GPU against the float64
oracle, and a layer built from convolution, dropout, residual and norm with all its gradients."""

import numpy as np
import pytest

import helpers
from node_helpers import TYPES, U, Problem, assert_near, tol32
from oracle import conv, node

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


MIXED, ODD = "128x0e+64x1o+32x2e+16x3o", "37x0e+19x1o+6x2e+3x3o"
SEED, OFFSET = 0xFEDCBA9876543210, (1 << 40) + 3
CASES = [("8x0e+8x1o+8x2e", 64, 0.1), (MIXED, 60, 0.5), (ODD, 33, 0.3), ("1x0e", 9, 0.5), ("1x1o", 9, 0.5),
         ("5x0o+2x0e+3x3o", 21, 0.9), ("4096x0e", 3, 0.2), ("12x1o+4x0e", 1, 0.25), ("20001x0e", 1, 0.5),
         (ODD, 17, 0.0), (ODD, 17, 1.0), ("64x0e", 700, 0.1), ("4100x1o", 2, 0.5), ("6x0e+10x1o", 300, 0.4),
         ("1001x0e", 20, 0.2), ("2048x0e+4x1o", 30, 0.6)]


def _drop(p, step=None):
    from equivariant_gnn_tensor_dst_b200 import binding
    return binding.Dropout(p, SEED, OFFSET, step)


@pytest.mark.parametrize("layout", ["ir_mul", "mul_ir"])
@pytest.mark.parametrize("irreps,n,p", CASES)
def test_dropout_float32(torch, irreps, n, p, layout):
    """Masks bit for bit; values to the product's, the scale's and the sum's rounding."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    q = Problem(irreps, n, layout=layout)
    mask = node.dropout_mask(q.R, n, p, SEED, OFFSET)
    out = B.tpconv_dropout_forward(q.plan, q.x, _drop(p))
    assert np.array_equal(out.cpu().numpy() != 0, mask * q.x64 != 0)
    assert_near(out, mask * q.x64, np.abs(mask * q.x64), 3 * U)
    res, res64 = q.rows()
    out = B.tpconv_dropout_forward(q.plan, q.x, _drop(p), residual=res)
    assert_near(out, mask * q.x64 + res64, np.abs(mask * q.x64) + np.abs(res64), 3 * U)
    assert torch.equal(out.cpu()[torch.from_numpy(mask == 0)], res.cpu()[torch.from_numpy(mask == 0)])
    assert_near(B.tpconv_dropout_backward(q.plan, res, _drop(p)), mask * res64, np.abs(mask * res64), 3 * U)


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("irreps,n,p", [(MIXED, 40, 0.1), (ODD, 33, 0.5), ("4096x0e", 2, 0.3), ("1x0e", 3, 0.5),
                                        ("8x0e+16x1o+8x2e+24x3o", 500, 0.3), ("3000x0e", 3, 0.5), ("8x3o", 17, 1.0),
                                        ("40x1o", 19, 0.0), ("12x0e+4x2e", 90, 0.25)])
@pytest.mark.parametrize("layout", ["ir_mul", "mul_ir"])
def test_dropout_16_bit(torch, irreps, n, p, dtype, layout):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    q = Problem(irreps, n, dtype, layout)
    mask = node.dropout_mask(q.R, n, p, SEED, OFFSET)
    res, res64 = q.rows()
    out = B.tpconv_dropout_forward(q.plan, q.x, _drop(p), residual=res)
    assert_near(out, mask * q.x64 + res64, np.abs(mask * q.x64) + np.abs(res64), 3 * U, dtype)
    out = B.tpconv_dropout_forward(q.plan, q.x, _drop(p))
    assert_near(out, mask * q.x64, np.abs(mask * q.x64), 3 * U, dtype)


def test_dropped_values_are_zero_whatever_they_were(torch):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    q = Problem(ODD, 40)
    mask = torch.from_numpy(node.dropout_mask(q.R, 40, 0.5, SEED, OFFSET)).cuda()
    x = torch.where(mask == 0, torch.full_like(q.x, float("nan")), q.x)
    assert torch.equal(B.tpconv_dropout_forward(q.plan, x, _drop(0.5)), B.tpconv_dropout_forward(q.plan, q.x, _drop(0.5)))
    nan = torch.full_like(q.x, float("nan"))
    assert not B.tpconv_dropout_forward(q.plan, nan, _drop(1.0)).any()


def test_in_place(torch):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    for irreps in (MIXED, ODD):
        q = Problem(irreps, 50)
        res, _ = q.rows()
        ref = B.tpconv_dropout_forward(q.plan, q.x, _drop(0.3), residual=res)
        a, b = q.x.clone(), res.clone()
        assert torch.equal(B.tpconv_dropout_forward(q.plan, a, _drop(0.3), residual=res, out=a), ref)
        assert torch.equal(B.tpconv_dropout_forward(q.plan, q.x, _drop(0.3), residual=b, out=b), ref)


@pytest.mark.parametrize("irreps,dtype", [(i, d) for i in (MIXED, ODD, "64x0e+24x1o", "3000x0e", "4100x1o", "20001x0e")
                                          for d in TYPES])
@pytest.mark.parametrize("layout", ["ir_mul", "mul_ir"])
def test_in_place_in_every_kernel(torch, irreps, dtype, layout):
    """out equal to x, to the residual and to both, in each storage type: whole packs, rows off the
    boundary, segments wider than a CTA's registers."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    q = Problem(irreps, 37, dtype, layout)
    res, _ = q.rows()
    plain = B.tpconv_dropout_forward(q.plan, q.x, _drop(0.3))
    ref = B.tpconv_dropout_forward(q.plan, q.x, _drop(0.3), residual=res)
    own = B.tpconv_dropout_forward(q.plan, q.x, _drop(0.3), residual=q.x)
    a, b, c, d, e = q.x.clone(), res.clone(), q.x.clone(), q.x.clone(), q.x.clone()
    assert torch.equal(B.tpconv_dropout_forward(q.plan, a, _drop(0.3), residual=res, out=a), ref)
    assert torch.equal(B.tpconv_dropout_forward(q.plan, q.x, _drop(0.3), residual=b, out=b), ref)
    assert torch.equal(B.tpconv_dropout_forward(q.plan, c, _drop(0.3), residual=c, out=c), own)
    assert torch.equal(B.tpconv_dropout_forward(q.plan, d, _drop(0.3), out=d), plain)
    assert torch.equal(B.tpconv_dropout_backward(q.plan, e, _drop(0.3), out=e), plain)


def test_step_counter_and_replay(torch):
    """A captured graph draws the mask of offset + *step as it is when the graph runs."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    q = Problem(MIXED, 30)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = _drop(0.5, step)
    ones, out, z, y = torch.ones_like(q.x), torch.empty_like(q.x), torch.empty_like(q.x), torch.empty_like(q.x)
    gx, gr = torch.empty_like(q.x), torch.empty_like(q.x)

    def run():
        B.tpconv_dropout_forward(q.plan, ones, d, out=out)
        B.tpconv_dropout_norm_forward(q.plan, ones, d, weight=q.w, bias=q.b, outputs=(z, y))
        B.tpconv_dropout_norm_backward(q.plan, q.x, q.w, ones, d, outputs=(gx, gr, None, None))
        step.add_(1)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for s in (0, 1, 2, -1, 1 << 40):
        step.fill_(s)
        graph.replay()
        torch.cuda.synchronize()
        mask = node.dropout_mask(q.R, 30, 0.5, SEED, (OFFSET + s) % (1 << 64))
        assert np.array_equal(out.cpu().numpy(), mask) and np.array_equal(z.cpu().numpy(), mask)
        assert np.array_equal(gx.cpu().numpy(), mask.astype(np.float32) * gr.cpu().numpy())
    del graph


FUSED = [("8x0e+8x1o+8x2e", 64), (MIXED, 90), (ODD, 33), ("1x0e+1x1o", 5), ("4096x0e", 5), ("20001x0e", 2),
         ("64x0e+64x1o+64x2e", 200), ("600x1o+5x0e", 3)]


@pytest.mark.parametrize("irreps,n,dtype,layout,p,residual", [
    c + (t, lay, p, r) for i, c in enumerate(FUSED)
    for t, lay, p, r in [("float32", "ir_mul", 0.3, True), ("float32", "mul_ir", 0.5, i % 2 == 0),
                         (TYPES[1 + i % 2], "ir_mul", 0.1, True), (TYPES[2 - i % 2], "mul_ir", 0.0, False)]])
def test_dropout_norm(torch, irreps, n, dtype, layout, p, residual):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    q = Problem(irreps, n, dtype, layout)
    mask = node.dropout_mask(q.R, n, p, SEED, OFFSET)
    res, res64 = q.rows() if residual else (None, 0.0)
    z, y = B.tpconv_dropout_norm_forward(q.plan, q.x, _drop(p), residual=res, weight=q.w, bias=q.b)
    z64 = mask * q.x64 + res64
    zs = np.abs(mask * q.x64) + np.abs(res64)
    assert_near(z, z64, zs, 3 * U, dtype, "z")
    # y's error from z: 3 roundings of zs in every element and in the means, through w r
    h = Problem.forward_scale(q, np.where(np.abs(z64) > 0, z64, 0.0))
    spread = q.R.rows([w * r * (v + node._mean(v)) * (1 + node._mean(hh * hh)) for w, (hh, r), v in
                       zip(q.R.split(np.abs(q.w64)), q._stats(z64), q.R.parts(zs))])
    assert_near(y, node.norm_forward(q.R, z64, q.w64, q.b64), h + spread, tol32(q.R), dtype, "y")

    (gy, gy64), (gz, gz64) = q.rows(), q.rows()
    got = B.tpconv_dropout_norm_backward(q.plan, z, q.w, gy, _drop(p), grad_z=gz)
    zz = z.double().cpu().numpy()
    ex, ew, eb = node.norm_backward(q.R, zz, q.w64, gy64)
    sx, sw = q.backward_scale(zz, gy64)
    t, ts = ex + gz64, sx + np.abs(gz64)
    assert_near(got[0], t * mask, ts * mask, tol32(q.R), dtype, "grad_x")
    assert_near(got[1], t, ts, tol32(q.R), dtype, "grad_residual")
    assert_near(got[2], ew, sw, q.sum_tol(), what="grad_weight")
    sb = np.concatenate([np.zeros(0)] + [np.abs(v).sum(axis=(0, 1)) for b, v in zip(q.R.blocks, q.R.parts(gy64))
                                         if q.R.centred(b)])
    assert_near(got[3], eb, sb, q.sum_tol(), what="grad_bias")
    none = B.tpconv_dropout_norm_backward(q.plan, z, q.w, gy, _drop(p))
    assert_near(none[1], ex, sx, tol32(q.R), dtype, "grad_residual without grad_z")


def test_fused_equals_parts_in_float32(torch):
    """z of the fused call is dropout's output, y is the norm of it."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    for irreps in (MIXED, ODD):
        q = Problem(irreps, 200)
        res, _ = q.rows()
        z, y = B.tpconv_dropout_norm_forward(q.plan, q.x, _drop(0.2), residual=res, weight=q.w, bias=q.b)
        assert torch.equal(z, B.tpconv_dropout_forward(q.plan, q.x, _drop(0.2), residual=res))
        assert torch.equal(y, B.tpconv_norm_forward(q.plan, z, q.w, q.b))
        gy, _ = q.rows()
        gx, gr, gw, gb = B.tpconv_dropout_norm_backward(q.plan, z, q.w, gy, _drop(0.2))
        ref = B.tpconv_norm_backward(q.plan, z, q.w, gy)
        assert all(torch.equal(a, b) for a, b in zip((gr, gw, gb), ref))
        assert torch.equal(gx, B.tpconv_dropout_backward(q.plan, gr, _drop(0.2)))
        only = B.tpconv_dropout_norm_backward(q.plan, z, q.w, gy, _drop(0.2), need_x=False, need_weight=False,
                                              need_bias=False)
        assert torch.equal(only[1], gr) and only[0] is None


def test_layer_with_convolution(torch):
    """One layer as it is used, z = x + dropout(conv(x)), y = norm(z): forward and every gradient
    against the oracle's chain (relative L2 <= 1e-4, the convolution's tolerance)."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = helpers.Problem(2, n_nodes=80)
    lp, irreps = helpers.lib_plan(p.cfg), p.cfg.irreps_out
    plan, R = B.NodePlan(irreps), node.Rows(irreps)
    g = np.random.default_rng(5)
    w64, b64 = 1 + 0.2 * g.normal(size=R.channels), 0.2 * g.normal(size=R.biases)
    w32, b32 = w64.astype(np.float32), b64.astype(np.float32)
    x, pos, rp, src, W, gy = (helpers.cuda(a) for a in (p.x, p.pos, p.row_ptr, p.src, p.W, p.gout))
    w, b = helpers.cuda(w32), helpers.cuda(b32)
    views = B.tpconv_csr_transpose(rp, src, p.N)
    drop = B.Dropout(0.25, 77, offset=4)

    m = B.tpconv_forward(lp, x, pos, rp, src, W)
    z, y = B.tpconv_dropout_norm_forward(plan, m, drop, residual=x, weight=w, bias=b)
    gm, gres, gw, gb = B.tpconv_dropout_norm_backward(plan, z, w, gy, drop)
    gx, gp, gW = B.tpconv_backward(lp, x, pos, rp, src, *views, W, gm)
    gx = gx + gres

    mask = node.dropout_mask(R, p.N, 0.25, 77, 4)
    m64 = conv.forward(p.plan, p.x, p.pos, p.row_ptr, p.src, p.W)
    z64 = p.x + mask * m64
    assert helpers.rel_l2(y.cpu(), node.norm_forward(R, z64, w32, b32)) <= 1e-4
    t, ew, eb = node.norm_backward(R, z64, w32.astype(np.float64), p.gout)
    ex, ep, eW = conv.backward(p.plan, p.x, p.pos, p.row_ptr, p.src, p.W, t * mask)
    for got, ref in ((gx, ex + t), (gp, ep), (gW, eW), (gw, ew), (gb, eb)):
        assert helpers.rel_l2(got.cpu(), ref) <= 1e-4


def test_force_training_through_the_layer(torch):
    """Double backward of energy = <c, norm(dropout(conv(x)))> along a force tangent: dLambda/dW of
    Lambda = <gg_pos, dE/dpos>, through conv, dropout and norm, against differences of the oracle's
    dE/dpos in W."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = helpers.Problem(1, n_nodes=24)
    lp, irreps = helpers.lib_plan(p.cfg), p.cfg.irreps_out
    plan, R = B.NodePlan(irreps), node.Rows(irreps)
    g = np.random.default_rng(8)
    w32 = (1 + 0.2 * g.normal(size=R.channels)).astype(np.float32)
    ggp = g.normal(size=p.pos.shape).astype(np.float32)
    x, pos, rp, src, W, c = (helpers.cuda(a) for a in (p.x, p.pos, p.row_ptr, p.src, p.W, p.gout))
    w, gg_pos = helpers.cuda(w32), helpers.cuda(ggp)
    views = B.tpconv_csr_transpose(rp, src, p.N)
    drop = B.Dropout(0.25, 5)
    # E = <c, norm(z)>, z = dropout(m), m = conv(pos, W); gm = dE/dm; forces F = dE/dpos
    m = B.tpconv_forward(lp, x, pos, rp, src, W)
    z = B.tpconv_dropout_forward(plan, m, drop)
    gz = B.tpconv_norm_backward(plan, z, w, c, need_weight=False, need_bias=False)[0]
    gm = B.tpconv_dropout_backward(plan, gz, drop)
    F = B.tpconv_backward(lp, x, pos, rp, src, *views, W, gm, need_x=False, need_W=False)[1]
    # Lambda = <gg_pos, F(W, gm)>: conv's double backward gives its derivative at fixed gm and d/dgm
    _, dW, d_gm = B.tpconv_double_backward(lp, x, pos, rp, src, *views, W, gm, gg_pos=gg_pos, need_x=False)
    d_gz = B.tpconv_dropout_backward(plan, d_gm, drop)
    d_z = B.tpconv_norm_double_backward(plan, z, w, c, gg_x=d_gz, need_weight=False, need_grad_y=False)[0]
    d_m = B.tpconv_dropout_backward(plan, d_z, drop)
    dW = dW + B.tpconv_backward(lp, x, pos, rp, src, *views, W, d_m, need_x=False, need_pos=False)[2]

    mask = node.dropout_mask(R, p.N, 0.25, 5)

    def forces(W64):
        z64 = mask * conv.forward(p.plan, p.x, p.pos, p.row_ptr, p.src, W64)
        gz64 = node.norm_backward(R, z64, w32.astype(np.float64), p.gout)[0]
        return conv.backward(p.plan, p.x, p.pos, p.row_ptr, p.src, W64, gz64 * mask)[1]

    assert helpers.rel_l2(F.cpu(), forces(p.W.astype(np.float64))) <= 1e-4
    for _ in range(3):
        d = g.normal(size=p.W.shape)
        h = 1e-5
        want = (ggp * (forces(p.W + h * d) - forces(p.W - h * d))).sum() / (2 * h)
        got = (dW.cpu().numpy().astype(np.float64) * d).sum()
        scale = np.linalg.norm(dW.cpu().numpy()) * np.linalg.norm(d)
        assert abs(got - want) <= 1e-4 * scale

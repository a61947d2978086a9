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
          ("128x0e+128x1o+128x2e", 700), ("10000x0e+8x1o", 3), ("20001x0e", 2), ("9000x2e", 2),
          # groups of 2, 4, 8 and 16 warps, on the boundary and off it, several rows a CTA and many
          ("1024x0e", 650), ("1001x0e", 900), ("2048x0e", 400), ("1999x0o", 350), ("4096x0e", 500), ("3999x0e", 310),
          ("8192x0e", 160), ("8001x0e", 9), ("2700x1o", 5), ("130x2e+65x1o+700x3o", 40), ("16x0e+4096x0e+1x1o", 7)]


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
                                             ("8x0e+24x1o", 1000, "ir_mul"), ("1024x0e+128x1o", 300, "ir_mul"),
                                             ("8192x0e", 150, "ir_mul"), ("7001x0e", 20, "ir_mul"),
                                             ("2049x0e+3x2e", 170, "mul_ir"), ("128x0e+128x1o+128x2e", 900, "mul_ir")])
def test_16_bit(irreps, n, layout, dtype):
    _all_passes(Problem(irreps, n, dtype, layout))


def test_rows_beyond_one_launch_range():
    """More rows than any grid dimension of the launch."""
    _all_passes(Problem("4x0e", 70001))


@pytest.mark.parametrize("irreps", ["96x0e", "1024x0e", "4096x0e", "1999x0e"])
def test_large_offset(irreps):
    """A mean a thousand times the spread in some rows: the spread is taken around the mean, not as a
    difference of squares; in groups of lanes and of several warps."""
    from equivariant_gnn_tensor_dst_b200 import binding
    p = Problem(irreps, 400)
    p.x[some_rows(400)] += 1000.0
    x64 = p.x.double().cpu().numpy()
    y = binding.tpconv_norm_forward(p.plan, p.x, p.w, p.b).double().cpu().numpy()
    ref = node.norm_forward(p.R, x64, p.w64, p.b64)
    # an error of the mean, 2^-24 (S / 32 + 16) of |x|, in every u, through r; rows scaled by their spread
    spread = np.std(x64, axis=1, keepdims=True)
    err = 2.0 ** -24 * (p.R.dim / 32 + 24) * np.abs(x64).mean(axis=1, keepdims=True) / spread
    h = np.abs(x64 - x64.mean(axis=1, keepdims=True)) / spread
    assert np.all(np.abs(y - ref) <= 2 * (1 + h) * (err + tol32(p.R)) * np.abs(p.w64).max() + tol32(p.R))


def some_rows(n):
    """About a third of the rows, in no regular order."""
    return np.flatnonzero(np.random.default_rng(1).random(n) < 0.33)


@pytest.mark.parametrize("irreps,n", [("96x0e", 40), ("1024x0e", 3000), ("2048x0e", 2000), ("4096x0e", 400),
                                      ("3999x0e", 400)])
def test_large_offset_backward(irreps, n):
    """The same for the backward, in groups of lanes and of several warps, rows of either kind (mean
    large and not) side by side, so that the groups of a CTA are at different sums."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(irreps, n)
    p.x[some_rows(n)] += 1000.0
    x64 = p.x.double().cpu().numpy()
    gy, gy64 = p.rows()
    gx, gw, gb = B.tpconv_norm_backward(p.plan, p.x, p.w, gy)
    ex, ew, _ = node.norm_backward(p.R, x64, p.w64, gy64)
    # an error of the mean, 2^-24 (S / 32 + 16) of |x|, moves every u by as much: relative to the
    # spread (e^-1.5 at least, r <= e^1.5) that is the error of h, of r and of the mean of a h
    S = p.R.dim
    err = 2.0 ** -24 * (S / 32 + 24) * np.abs(x64).mean(axis=1, keepdims=True) * np.exp(1.5)
    scale = np.exp(1.5) * (np.abs(gy64) + 1) * 2.0 * (1 + np.abs(x64 - x64.mean(axis=1, keepdims=True)) * np.exp(1.5))
    assert np.all(np.abs(gx.double().cpu().numpy() - ex) <= 6 * (err + tol32(p.R)) * scale)


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


@pytest.mark.parametrize("irreps,n", [(MIXED, 50), (MIXED, 3000), (ODD, 700), ("4096x0e", 300), ("20001x0e", 3)])
def test_optional_arguments(torch, irreps, n):
    """No weight and bias are ones and zeros; missing tangents are zeros; outputs are computed one
    by one as together."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(irreps, n)
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


def test_first_call_captured(torch):
    """A process whose first calls are made while a graph is captured (kernels not loaded, shared
    memory not yet allowed), replayed, against the same calls afterwards."""
    import subprocess
    import sys
    code = """
import torch
from equivariant_gnn_tensor_dst_b200 import binding as B
plan = B.NodePlan("128x0e+64x1o+32x2e+16x3o+4096x0e")
x, gy = (torch.randn(600, plan.dim, device="cuda") for _ in range(2))
w, b = torch.rand(plan.channels, device="cuda"), torch.rand(plan.biases, device="cuda")
d, ws = B.Dropout(0.3, 5), B.workspace(plan.workspace_bytes(600), x.device)
E = torch.empty_like
o = [E(x), E(x), E(w), E(b), E(x), E(w), E(x), E(x), E(x), E(x), E(x), E(w), E(b)]
def step():
    B.tpconv_norm_forward(plan, x, w, b, out=o[0])
    B.tpconv_norm_backward(plan, x, w, gy, ws=ws, outputs=o[1:4])
    B.tpconv_norm_double_backward(plan, x, w, gy, gy, w, b, ws=ws, outputs=o[4:7])
    B.tpconv_dropout_norm_forward(plan, x, d, residual=gy, weight=w, bias=b, outputs=o[7:9])
    B.tpconv_dropout_norm_backward(plan, x, w, gy, d, grad_z=gy, ws=ws, outputs=o[9:13])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in o]
step()
torch.cuda.synchronize()
assert all(torch.equal(s, t) for s, t in zip(got, o))
print("captured ok")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr


def test_two_streams_and_threads(torch):
    """Calls with one plan from two threads on two streams, each with its own workspace, give what
    they give one after the other."""
    import threading
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, 3000)
    grads = [p.rows()[0] for _ in range(2)]
    ref = [B.tpconv_norm_backward(p.plan, p.x, p.w, g) for g in grads]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]

    def work(i):
        with torch.cuda.stream(streams[i]):
            ws = B.workspace(p.plan.workspace_bytes(p.n), p.x.device)
            for _ in range(20):
                got[i].append(B.tpconv_norm_backward(p.plan, p.x, p.w, grads[i], ws=ws))
        streams[i].synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, ref[i]))


def test_two_graphs_share_a_workspace(torch):
    """Graphs captured with the same workspace, replayed one after the other in either order."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p, q = Problem(MIXED, 2000), Problem(ODD, 900)
    (gp, _), (gq, _) = p.rows(), q.rows()
    ws = B.workspace(max(p.plan.workspace_bytes(p.n), q.plan.workspace_bytes(q.n)), p.x.device)
    calls = [(a, g, tuple(torch.empty_like(t) for t in (a.x, a.w, a.b))) for a, g in ((p, gp), (q, gq))]
    ref = [[t.clone() for t in B.tpconv_norm_backward(a.plan, a.x, a.w, g)] for a, g, _ in calls]
    graphs = []
    for a, g, o in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.tpconv_norm_backward(a.plan, a.x, a.w, g, ws=ws, outputs=o)
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for _, _, o in calls:
            for t in o:
                t.fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (_, _, o), r in zip(calls, ref):
            assert all(torch.equal(s, t) for s, t in zip(o, r))
    del graphs


def test_guard_bands(torch):
    """Nothing outside the outputs is written, whatever the alignment of rows and blocks."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    for irreps in (MIXED, ODD, "1x0e", "3x0e+1x1o", "1001x0e", "8001x0e"):
        for dtype in TYPES:
            for n in (1, 2, 7, 33):
                p = Problem(irreps, n, dtype)
                gy, _ = p.rows()
                size, pad = n * p.plan.dim, 64
                whole = [torch.full((size + 2 * pad,), 9.0, dtype=p.x.dtype, device="cuda") for _ in range(3)]
                outs = [t[pad:pad + size].view(n, p.plan.dim) for t in whole]
                B.tpconv_norm_forward(p.plan, p.x, p.w, p.b, out=outs[0])
                B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, gy, need_weight=False,
                                              outputs=(outs[1], None, outs[2]))
                B.tpconv_dropout_norm_forward(p.plan, p.x, B.Dropout(0.5, 1), residual=gy, outputs=(outs[1], outs[2]))
                B.tpconv_dropout_norm_backward(p.plan, p.x, p.w, gy, B.Dropout(0.5, 1),
                                               outputs=(outs[1], outs[2], None, None))
                B.tpconv_dropout_forward(p.plan, p.x, B.Dropout(0.5, 1), out=outs[0])
                for t in whole:
                    assert bool((t[:pad] == 9.0).all()) and bool((t[pad + size:] == 9.0).all())


@pytest.mark.parametrize("irreps,dtype", [("2048x0e", "bfloat16"), ("2047x0e", "float16")])
def test_64_bit_offsets(torch, irreps, dtype):
    """Rows beyond 2^31 elements (16 bits: 4.4 GB an array), on the 16-byte boundary and off it: the
    last rows equal the same rows alone."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    T = getattr(torch, dtype)
    plan = B.NodePlan(irreps, T)
    dim = plan.dim
    n = (1 << 31) // dim + 80
    x = torch.randn(64, dim, device="cuda").to(T).repeat(n // 64 + 1, 1)[:n].contiguous()
    gy = x.flip(1).contiguous()
    y = B.tpconv_norm_forward(plan, x)
    gx = B.tpconv_norm_backward(plan, x, None, gy, need_weight=False, need_bias=False)[0]
    tail = (n - 40) // 8 * 8         # the same number modulo 8
    assert tail * dim > 1 << 31
    assert torch.equal(y[tail:], B.tpconv_norm_forward(plan, x[tail:].clone()))
    assert torch.equal(gx[tail:], B.tpconv_norm_backward(plan, x[tail:].clone(), None, gy[tail:].clone())[0])
    d = B.Dropout(0.5, 3)
    out = B.tpconv_dropout_forward(plan, x, d, out=y)
    kept = out[tail:] != 0
    assert torch.equal(out[tail:], torch.where(kept, 2 * x[tail:], torch.zeros_like(x[tail:])))
    assert 0.45 < kept.float().mean().item() < 0.55


def test_profile_counts_launches(torch):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(MIXED, 5000)
    gy, _ = p.rows()
    B.tpconv_profile_begin(64)
    B.tpconv_norm_forward(p.plan, p.x, p.w, p.b)                    # one launch
    B.tpconv_norm_backward(p.plan, p.x, p.w, gy)                    # rows, reduction
    B.tpconv_norm_backward(p.plan, p.x, p.w, gy, need_weight=False, need_bias=False)
    B.tpconv_dropout_forward(p.plan, p.x, B.Dropout(0.1, 1))
    ms, n = B.tpconv_profile_end()["node_features"]
    assert n == 5 and ms > 0


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

"""Calls on a stream of their own, with outputs and workspaces that the binding makes, while the
current stream allocates and writes: nothing of a call may be given away before its kernels are done."""

import pytest

import helpers
from node_helpers import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def _check_on_a_busy_stream(torch, call, sizes):
    """call(stream) on a stream that has two milliseconds of work before it; the current stream
    meanwhile fills blocks of the given sizes with NaN bit patterns."""
    ref = call(None)
    side, a = torch.cuda.Stream(), torch.zeros(4096, 4096, dtype=torch.bfloat16, device="cuda")
    c = torch.empty_like(a)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.mm(a, a, out=c)
        got = call(side)
        mine = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert all((s is None and t is None) or torch.equal(s, t) for s, t in zip(got, ref))
        assert all(bool((t == 255).all()) for t in mine)


@pytest.mark.parametrize("irreps,n", [("128x0e+64x1o+32x2e+16x3o", 4000), ("37x0e+19x1o+6x2e+3x3o", 900), ("4096x0e", 300)])
def test_node_operators(torch, irreps, n):
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem(irreps, n)
    (gy, _), (t, _), (s, _), (q, _) = p.rows(), p.rows(), p.vector(p.R.channels), p.vector(p.R.biases)
    d = B.Dropout(0.3, 5)
    sizes = [p.plan.workspace_bytes(n), p.x.numel() * 4, max(p.w.numel() * 4, 512)]
    for call in (lambda st: (B.tpconv_norm_forward(p.plan, p.x, p.w, p.b, stream=st),),
                 lambda st: B.tpconv_norm_backward(p.plan, p.x, p.w, gy, stream=st),
                 lambda st: B.tpconv_norm_backward(p.plan, p.x, p.w, gy, need_x=False, stream=st),
                 lambda st: B.tpconv_norm_double_backward(p.plan, p.x, p.w, gy, t, s, q, stream=st),
                 lambda st: (B.tpconv_dropout_forward(p.plan, p.x, d, gy, stream=st),
                             B.tpconv_dropout_backward(p.plan, gy, d, stream=st)),
                 lambda st: B.tpconv_dropout_norm_forward(p.plan, p.x, d, gy, p.w, p.b, stream=st),
                 lambda st: B.tpconv_dropout_norm_backward(p.plan, p.x, p.w, gy, d, t, stream=st)):
        _check_on_a_busy_stream(torch, call, sizes)


@pytest.mark.parametrize("cfg,n", [(1, 300), (3, 200)])
def test_convolution_and_graph(torch, cfg, n):
    """The same for the convolution's passes and the graph calls (uvw and uvu)."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = helpers.Problem(cfg, n_nodes=n)
    lp = helpers.lib_plan(p.cfg)
    x, pos, rp, src, W, g = (helpers.cuda(a) for a in (p.x, p.pos, p.row_ptr, p.src, p.W, p.gout))
    views = B.tpconv_csr_transpose(rp, src, p.N)
    perm = B.tpconv_spatial_order(pos)
    sizes = [lp.workspace_bytes(p.N, p.E), W.numel() * 4, x.numel() * 4, g.numel() * 4, 4 * p.E, 4 * p.N + 4]
    for call in (lambda st: (B.tpconv_forward(lp, x, pos, rp, src, W, stream=st),),
                 lambda st: B.tpconv_backward(lp, x, pos, rp, src, *views, W, g, stream=st),
                 lambda st: B.tpconv_double_backward(lp, x, pos, rp, src, *views, W, g, gg_x=x, gg_pos=pos, stream=st),
                 lambda st: B.tpconv_csr_transpose(rp, src, p.N, stream=st),
                 lambda st: (B.tpconv_validate_graph(rp, src, p.N, stream=st), B.tpconv_spatial_order(pos, stream=st),
                             B.tpconv_gather_rows(x, perm, stream=st)),
                 lambda st: B.tpconv_permute_graph(rp, src, perm, stream=st)):
        _check_on_a_busy_stream(torch, call, sizes)


def test_captured_on_a_side_stream(torch):
    """A call on a stream that joins a capture allocates from the graph's memory there, too."""
    from equivariant_gnn_tensor_dst_b200 import binding as B
    p = Problem("128x0e+64x1o+32x2e+16x3o", 3000)
    gy, _ = p.rows()
    ref = B.tpconv_norm_backward(p.plan, p.x, p.w, gy)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = B.tpconv_norm_backward(p.plan, p.x, p.w, gy, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    del graph

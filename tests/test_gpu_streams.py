"""Calls on a stream of their own, with outputs and workspaces that the binding makes, while the
current stream allocates and writes: nothing of a call may be given away before its kernels are done."""

import pytest

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

"""Where the binding's own tensors (outputs and workspaces that a call makes) come from when a stream
is given: memory of that stream.  The allocator hands out a block again in the order of the stream
that it was allocated on, so a block of another stream could be given away, or still be in use, while
the call's kernels run.  Seen on the host: the library is a recorder, tensors are on the CPU."""

import contextlib

import pytest
import torch

from equivariant_gnn_tensor_dst_b200 import binding as B


class Side:
    """Stands for a torch stream (of the device that the tensors here are on)."""
    cuda_stream, device_index, device = 77, -1, torch.device("cpu")


class Made(list):
    """Allocations of a call, (stream they are made on, elements); the stream that is current."""
    current = None


@pytest.fixture
def made(monkeypatch):
    made = Made()

    @contextlib.contextmanager
    def enter(stream):
        before, made.current = made.current, stream
        yield
        made.current = before

    def recorded(f):
        def call(*a, **k):
            k.pop("device", None)
            t = f(*a, **k)
            made.append((made.current, t.numel()))
            return t
        return call

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Side.device_index)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 5)
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    return made


@pytest.fixture
def node(monkeypatch, made):
    """A node plan and the streams of the library's calls."""
    streams = []
    plan = B.NodePlan("8x0e+8x1o")
    monkeypatch.setattr(B, "_node_x", lambda plan, x, name: x.data_ptr())
    monkeypatch.setattr(B, "_node_call", lambda device, name, *args: streams.append(made.current))
    monkeypatch.setattr(B.Dropout, "spec", lambda self, device: self._ref)
    x, w, b = torch.ones(3000, plan.dim), torch.ones(plan.channels), torch.ones(plan.biases)
    return plan, x, w, b, streams


NODE_CALLS = {
    "norm_forward": lambda p, x, w, b, **k: B.tpconv_norm_forward(p, x, w, b, **k),
    "norm_backward": lambda p, x, w, b, **k: B.tpconv_norm_backward(p, x, w, x, **k),
    "norm_double_backward": lambda p, x, w, b, **k: B.tpconv_norm_double_backward(p, x, w, x, x, w, b, **k),
    "dropout_forward": lambda p, x, w, b, **k: B.tpconv_dropout_forward(p, x, B.Dropout(0.5, 1), **k),
    "dropout_backward": lambda p, x, w, b, **k: B.tpconv_dropout_backward(p, x, B.Dropout(0.5, 1), **k),
    "dropout_norm_forward": lambda p, x, w, b, **k: B.tpconv_dropout_norm_forward(p, x, B.Dropout(0.5, 1), x, w, b, **k),
    "dropout_norm_backward": lambda p, x, w, b, **k: B.tpconv_dropout_norm_backward(p, x, w, x, B.Dropout(0.5, 1), **k),
}


@pytest.mark.parametrize("name", sorted(NODE_CALLS))
def test_node_tensors_belong_to_the_stream(node, made, name):
    plan, x, w, b, streams = node
    for stream in (Side(), None):
        del made[:], streams[:]
        NODE_CALLS[name](plan, x, w, b, stream=stream)
        assert streams == [stream]
        assert made and all(s is stream for s, _ in made), made
    if name.endswith("backward") and name != "dropout_backward":
        assert (None, max(plan.workspace_bytes(3000), 256)) in made


class Library:
    """The library's host functions; compute calls are recorded by the stream that is current."""

    def __init__(self, real, made, streams):
        self.real, self.made, self.streams = real, made, streams

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes") or name.startswith(("tpconv_plan", "tpconv_node_plan")):
            return getattr(self.real, name)
        return lambda *args: self.streams.append(self.made.current) or 0


@pytest.fixture
def graph(monkeypatch, made):
    streams = []
    plan = B.Plan("4x0e+4x1o", 1, "4x0e+4x1o")
    library = Library(B.lib(), made, streams)
    monkeypatch.setattr(B, "lib", lambda: library)
    monkeypatch.setattr(B, "_need", lambda t, dtype, name: None)
    monkeypatch.setattr(B, "_stream", lambda: None)
    n, e = 50, 400
    i32 = lambda *v: torch.ones(*v, dtype=torch.int32)
    a = dict(x=torch.ones(n, plan.dim_in), pos=torch.ones(n, 3), row_ptr=i32(n + 1), src=i32(e), t_ptr=i32(n + 1),
             t_eid=i32(e), t_dst=i32(e), W=torch.ones(plan.num_basis, plan.weight_cols), g=torch.ones(n, plan.dim_out),
             Y=torch.ones(e, 4), phi=torch.ones(e, plan.num_basis), perm=i32(n), n=n)
    return plan, a, streams


GRAPH_CALLS = {
    "csr_transpose": lambda p, a, **k: B.tpconv_csr_transpose(a["row_ptr"], a["src"], a["n"], **k),
    "validate_graph": lambda p, a, **k: B.tpconv_validate_graph(a["row_ptr"], a["src"], a["n"], **k),
    "forward": lambda p, a, **k: B.tpconv_forward(p, a["x"], a["pos"], a["row_ptr"], a["src"], a["W"], **k),
    "backward": lambda p, a, **k: B.tpconv_backward(
        p, a["x"], a["pos"], a["row_ptr"], a["src"], a["t_ptr"], a["t_eid"], a["t_dst"], a["W"], a["g"], **k),
    "forward_embedded": lambda p, a, **k: B.tpconv_forward_embedded(
        p, a["x"], a["Y"], a["phi"], a["row_ptr"], a["src"], a["W"], **k),
    "backward_embedded": lambda p, a, **k: B.tpconv_backward_embedded(
        p, a["x"], a["Y"], a["phi"], a["row_ptr"], a["src"], a["t_ptr"], a["t_eid"], a["t_dst"], a["W"], a["g"], **k),
    "double_backward": lambda p, a, **k: B.tpconv_double_backward(
        p, a["x"], a["pos"], a["row_ptr"], a["src"], a["t_ptr"], a["t_eid"], a["t_dst"], a["W"], a["g"],
        gg_x=a["x"], need_pos=True, **k),
    "spatial_order": lambda p, a, **k: B.tpconv_spatial_order(a["pos"], **k),
    "permute_graph": lambda p, a, **k: B.tpconv_permute_graph(a["row_ptr"], a["src"], a["perm"], **k),
    "gather_rows": lambda p, a, **k: B.tpconv_gather_rows(a["x"], a["perm"], **k),
}


@pytest.mark.parametrize("name", sorted(GRAPH_CALLS))
def test_convolution_and_graph_tensors_belong_to_the_stream(graph, made, name):
    plan, a, streams = graph
    for stream in (Side(), None):
        del made[:], streams[:]
        GRAPH_CALLS[name](plan, a, stream=stream)
        assert streams == [stream]
        assert made and all(s is stream for s, _ in made), made


@pytest.mark.parametrize("rows", [0, 7, 80])
def test_gathered_rows_are_as_many_as_perm(graph, rows):
    """The library reads and writes perm.numel() rows of arrays that have a.shape[0]."""
    _, a, streams = graph
    with pytest.raises(ValueError):
        B.tpconv_gather_rows(a["x"], torch.ones(rows, dtype=torch.int32))
    assert not streams


def test_current_stream_is_not_entered_again(graph, node, made, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: Side.cuda_stream)
    plan, a, _ = graph
    GRAPH_CALLS["forward"](plan, a, stream=Side())
    node_plan, x, w, b, _ = node
    NODE_CALLS["norm_backward"](node_plan, x, w, b, stream=Side())
    assert made and all(s is None for s, _ in made)
    made.clear()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)   # current on a device that is not
    side = Side()
    GRAPH_CALLS["forward"](plan, a, stream=side)
    assert made and all(s is side for s, _ in made)


def test_stream_of_another_device_is_refused(graph, node):
    plan, a, streams = graph
    node_plan, x, w, b, node_streams = node
    other = Side()
    other.device_index, other.device = 1, torch.device("cuda:1")
    with pytest.raises(ValueError, match="stream is on cuda:1, x on cpu"):
        GRAPH_CALLS["forward"](plan, a, stream=other)
    with pytest.raises(ValueError, match="stream is on cuda:1, x on cpu"):
        NODE_CALLS["norm_forward"](node_plan, x, w, b, stream=other)
    assert not streams and not node_streams

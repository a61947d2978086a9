"""Where the binding's own tensors (outputs and workspaces that a call makes) come from when a stream
is given: memory of that stream.  The allocator hands out a block again in the order of the stream
that it was allocated on, so a block of another stream could be given away, or still be in use, while
the call's kernels run.  Seen on the host: the library is a recorder, tensors are on the CPU."""

import contextlib

import pytest
import torch

from equivariant_gnn_tensor_dst_b200 import binding as B


class Side:
    """Stands for a torch stream."""
    cuda_stream = 77


@pytest.fixture
def made(monkeypatch):
    """Allocations of a call: (stream they are made on, elements)."""
    made, on = [], [None]

    @contextlib.contextmanager
    def enter(stream):
        on.append(stream)
        yield
        on.pop()

    def recorded(f):
        def call(*a, **k):
            k.pop("device", None)
            t = f(*a, **k)
            made.append((on[-1], t.numel()))
            return t
        return call

    monkeypatch.setattr(torch.cuda, "stream", enter)
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    return made


@pytest.fixture
def node(monkeypatch, made):
    """A node plan and the streams of the library's calls."""
    streams = []
    plan = B.NodePlan("8x0e+8x1o")
    monkeypatch.setattr(B, "_node_x", lambda plan, x, name: x.data_ptr())
    monkeypatch.setattr(B, "_node_call", lambda device, name, stream, *args: streams.append(stream))
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

"""Host-side checks of the node-feature operators (include/tpconv_node.h; no GPU needed):
plans, argument counts, and every refusal before a launch."""

import ctypes
import os
import re

import pytest

from equivariant_gnn_tensor_dst_b200 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, PARSE, UNSUPPORTED, SMALL, MISALIGNED = 0, 1, 2, 3, 4, 5
MIB = 1 << 20


def ptr(i, off=0):
    """Distinct aligned addresses 16 MiB apart (never dereferenced: the checks fail first)."""
    return ctypes.c_void_p((i + 1) * 16 * MIB + off)


def test_arity_matches_header():
    txt = open(os.path.join(ROOT, "include", "tpconv_node.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    found = re.findall(r"\b(tpconv_\w+)\s*\(([^;{]*?)\)\s*;", txt, flags=re.S)
    assert len(found) == 12
    for name, params in found:
        assert len(binding.SIGNATURES[name][1]) == params.count(",") + 1, name


def test_plan_numbering():
    p = binding.NodePlan("5x0e+3x0o+2x1o+7x0e")
    assert (p.dim, p.channels, p.biases, p.num_blocks) == (21, 17, 12, 4)
    q = binding.NodePlan("128x0e+64x1o+32x2e+16x3o")
    assert (q.dim, q.channels, q.biases, q.num_blocks) == (592, 240, 128, 4)


@pytest.mark.parametrize("irreps,dtype,eps,code", [
    ("4x0q", 0, 1e-5, PARSE), ("", 0, 1e-5, PARSE), ("0x0e", 0, 1e-5, PARSE), ("4x4e", 0, 1e-5, UNSUPPORTED),
    ("+".join(["1x0e"] * 17), 0, 1e-5, UNSUPPORTED), ("4x0e", 3, 1e-5, UNSUPPORTED), ("4x0e", -1, 1e-5, UNSUPPORTED),
    ("4x0e", 0, 0.0, INVALID), ("4x0e", 0, -1.0, INVALID), ("4x0e", 0, float("nan"), INVALID),
    ("4x0e", 0, float("inf"), INVALID), ("4x0e", 0, 1e-40, INVALID),
])
def test_plan_errors(irreps, dtype, eps, code):
    h = ctypes.c_void_p()
    assert binding.lib().tpconv_node_plan_create(ctypes.byref(h), irreps.encode(), dtype, eps) == code
    assert h.value is None


def test_plan_arguments():
    import torch
    L = binding.lib()
    p = binding.NodePlan("8x0e+8x1o", torch.bfloat16, layout="mul_ir")
    assert L.tpconv_node_plan_set_layout(p.handle, 2) == UNSUPPORTED
    assert L.tpconv_node_plan_set_layout(None, 0) == INVALID
    assert L.tpconv_node_plan_destroy(None) == OK
    assert L.tpconv_node_plan_info(None, None, None, None, None) == INVALID
    for bad in (dict(dtype=torch.float64), dict(layout="mul")):
        with pytest.raises(ValueError):
            binding.NodePlan("8x0e", **bad)
    for p_drop in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            binding.Dropout(p_drop, 0)


def test_workspace_is_bounded():
    p = binding.NodePlan("128x0e+64x1o+32x2e+16x3o")
    assert p.workspace_bytes(0) == 0
    sizes = [p.workspace_bytes(n) for n in (1, 64, 4096, 50000, 1 << 30)]
    assert sizes == sorted(sizes) and 0 < sizes[2] and sizes[-1] <= 16 * MIB
    nb = ctypes.c_size_t()
    for n in (-1, 1 << 31):
        assert binding.lib().tpconv_node_workspace_bytes(p.handle, n, ctypes.byref(nb)) == INVALID
    assert binding.lib().tpconv_node_workspace_bytes(p.handle, 1, None) == INVALID


def _calls(p, N, a, drop, ws_bytes=1 << 30):
    """Every compute entry point with the pointers a[0..9] in its array arguments."""
    L, h, d = binding.lib(), p.handle, (None if drop is None else ctypes.byref(drop))
    return {
        "norm_forward": lambda: L.tpconv_norm_forward(h, N, a[0], a[1], a[2], a[3], None),
        "norm_backward": lambda: L.tpconv_norm_backward(h, N, a[0], a[1], a[2], a[3], a[4], a[5], a[9], ws_bytes, None),
        "norm_double_backward": lambda: L.tpconv_norm_double_backward(
            h, N, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], ws_bytes, None),
        "dropout_forward": lambda: L.tpconv_dropout_forward(h, N, a[0], a[1], d, a[2], None),
        "dropout_backward": lambda: L.tpconv_dropout_backward(h, N, a[0], d, a[2], None),
        "dropout_norm_forward": lambda: L.tpconv_dropout_norm_forward(h, N, a[0], a[1], d, a[2], a[3], a[4], a[5],
                                                                      None),
        "dropout_norm_backward": lambda: L.tpconv_dropout_norm_backward(
            h, N, a[0], a[1], a[2], a[3], d, a[4], a[5], a[6], a[7], a[9], ws_bytes, None),
    }


# positions of the array arguments in a[]: (required, optional)
ARRAYS = {"norm_forward": ((0, 3), (1, 2)), "norm_backward": ((0, 2), (1, 3, 4, 5)),
          "norm_double_backward": ((0, 2), (1, 3, 4, 5, 6, 7, 8)), "dropout_forward": ((0, 2), (1,)),
          "dropout_backward": ((0, 2), ()), "dropout_norm_forward": ((0, 4, 5), (1, 2, 3)),
          "dropout_norm_backward": ((0, 2), (1, 3, 4, 5, 6, 7))}
# (output, input) pairs that must not overlap
OVERLAPS = {"norm_forward": [(3, 0), (3, 1)], "norm_backward": [(3, 0), (3, 2), (4, 1), (4, 3), (5, 9), (3, 9)],
            "norm_double_backward": [(6, 0), (6, 2), (6, 3), (8, 2), (7, 4), (6, 8), (7, 9)],
            "dropout_norm_forward": [(4, 0), (4, 1), (5, 0), (5, 4)],
            "dropout_norm_backward": [(4, 0), (4, 5), (5, 3), (6, 1), (4, 9)]}
N = 20000


@pytest.fixture
def plan():
    return binding.NodePlan("8x0e+8x1o")


@pytest.mark.parametrize("name", sorted(ARRAYS))
def test_refusals_before_launch(plan, name):
    drop = binding.DropoutSpec(0.5, 1, 2, None)
    base = [ptr(i) for i in range(10)]
    for rows in (-1, 1 << 31):
        assert _calls(plan, rows, base, drop)[name]() == INVALID
    L = binding.lib()
    null = type("P", (), {"handle": None})
    assert _calls(null, N, base, drop)[name]() == INVALID
    required, optional = ARRAYS[name]
    for i in required:
        a = list(base)
        a[i] = None
        assert _calls(plan, N, a, drop)[name]() == INVALID, i
    for i in required + optional:
        a = list(base)
        a[i] = ptr(i, 4)
        assert _calls(plan, N, a, drop)[name]() == MISALIGNED, i
    for out, other in OVERLAPS.get(name, []):
        a = list(base)
        a[out] = a[other]
        assert _calls(plan, N, a, drop)[name]() == INVALID, (out, other)
    if name.endswith("backward") and name != "dropout_backward":
        need = plan.workspace_bytes(N)
        assert _calls(plan, N, base, drop, need - 1)[name]() == SMALL
        a = list(base)
        a[9] = None
        assert _calls(plan, N, a, drop)[name]() == INVALID
    if name.startswith("dropout"):
        assert _calls(plan, N, base, None)[name]() == INVALID
        for p in (-1e-9, 1.0 + 1e-9, float("nan")):
            assert _calls(plan, N, base, binding.DropoutSpec(p, 1, 2, None))[name]() == INVALID
        assert _calls(plan, N, base, binding.DropoutSpec(0.5, 1, 2, 4))[name]() == MISALIGNED
    assert L.tpconv_status_string(INVALID)


def test_dropout_overlap_must_be_exact(plan):
    """In place is allowed, a shifted overlap is not."""
    drop = binding.DropoutSpec(0.5, 1, 2, None)
    a = [ptr(i) for i in range(10)]
    a[2] = ptr(0, 16)
    assert _calls(plan, N, a, drop)["dropout_forward"]() == INVALID
    assert _calls(plan, N, a, drop)["dropout_backward"]() == INVALID


@pytest.mark.parametrize("name", ["norm_forward", "dropout_forward", "dropout_backward", "dropout_norm_forward"])
def test_empty_input_is_a_no_op(plan, name):
    drop = binding.DropoutSpec(0.5, 1, 2, None)
    assert _calls(plan, 0, [None] * 10, drop)[name]() == OK


def test_nothing_requested_is_a_no_op(plan):
    drop = binding.DropoutSpec(0.5, 1, 2, None)
    a = [ptr(0), None, ptr(2)] + [None] * 7
    for name in ("norm_backward", "norm_double_backward", "dropout_norm_backward"):
        assert _calls(plan, N, a, drop, 0)[name]() == OK


def test_closed_plan_is_refused():
    p = binding.NodePlan("8x0e")
    p.close()
    assert binding.lib().tpconv_norm_forward(p.handle, 1, ptr(0), None, None, ptr(1), None) == INVALID


def test_workspace_of_every_shape_is_bounded():
    """Widths from one element to a million channels, and both 16-bit and 32-bit rows: no more than
    the sums of one wave of CTAs."""
    import torch
    for irreps in ("1x0e", "4096x0e", "8192x0e", "8191x0e", "20000x0e", "999999x0e", "100x0e+5001x1o+7x3o"):
        for dtype in (torch.float32, torch.bfloat16):
            p = binding.NodePlan(irreps, dtype)
            for n in (1, 7, 1000, 1 << 20, (1 << 31) - 1):
                assert p.workspace_bytes(n) <= 48 * MIB, (irreps, dtype, n)


def test_threads_share_a_plan(plan):
    """Plans are read only at enqueue time; the workspace query keeps its cache consistent."""
    import threading
    want = {n: binding.NodePlan("8x0e+8x1o").workspace_bytes(n) for n in (10, 5000, 70000)}
    bad = []

    def work(n):
        for _ in range(300):
            if plan.workspace_bytes(n) != want[n]:
                bad.append(n)

    ts = [threading.Thread(target=work, args=(n,)) for n in want for _ in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_binding_refuses_bad_tensors(plan):
    import torch
    x = torch.zeros(3, plan.dim)
    d = binding.Dropout(0.1, 1)
    for call in (lambda: binding.tpconv_norm_forward(plan, x), lambda: binding.tpconv_dropout_forward(plan, x, d),
                 lambda: binding.tpconv_norm_backward(plan, x, None, x),
                 lambda: binding.tpconv_dropout_norm_forward(plan, x, d)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        binding.Dropout(0.1, 1, step=torch.zeros(1, dtype=torch.int64))

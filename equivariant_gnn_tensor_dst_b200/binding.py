"""ctypes binding of libtpconv.so (include/tpconv.h, tpconv_graph.h, tpconv_node.h).

Argument marshalling only: every computation runs in the library's kernels.  Tensors
are torch tensors (device memory, float32 / int32, contiguous); PyTorch is used to
allocate outputs and workspaces and to name the current CUDA stream.  If the shared
library is missing the import of ``lib()`` fails loudly; there is no fallback.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtpconv.so")

UVW, UVU = 0, 1
BESSEL, GAUSSIAN = 0, 1
PASS_FORWARD, PASS_BACKWARD, PASS_DOUBLE_BACKWARD = 1, 2, 4
MATH_FP32, MATH_TF32, MATH_BF16 = 0, 1, 2
LAYOUT_IR_MUL, LAYOUT_MUL_IR = 0, 1
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p


class RadialSpec(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("num_basis", ctypes.c_int32), ("r_cut", ctypes.c_float),
                ("r_min", ctypes.c_float), ("r_max", ctypes.c_float), ("poly_p", ctypes.c_int32)]


class DropoutSpec(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step", ctypes.c_void_p)]


# symbol -> (restype, argtypes); mirrors include/tpconv.h
SIGNATURES = {
    "tpconv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tpconv_plan_create": (ctypes.c_int, [ctypes.POINTER(_c_p), ctypes.c_char_p, ctypes.c_int32,
                                          ctypes.c_char_p, ctypes.c_int32, ctypes.POINTER(RadialSpec)]),
    "tpconv_plan_destroy": (ctypes.c_int, [_c_p]),
    "tpconv_plan_info": (ctypes.c_int, [_c_p] + [ctypes.POINTER(_c_i64)] * 5),
    "tpconv_plan_path": (ctypes.c_int, [_c_p, _c_i64, ctypes.POINTER(ctypes.c_int32)]),
    "tpconv_plan_path_coupling": (ctypes.c_int, [_c_p, _c_i64, ctypes.POINTER(ctypes.c_int32),
                                                 ctypes.POINTER(ctypes.c_double), _c_i64]),
    "tpconv_set_workspace_budget": (ctypes.c_int, [_c_p, ctypes.c_size_t]),
    "tpconv_plan_set_math": (ctypes.c_int, [_c_p, ctypes.c_int32]),
    "tpconv_plan_set_layout": (ctypes.c_int, [_c_p, ctypes.c_int32]),
    "tpconv_workspace_bytes": (ctypes.c_int, [_c_p, _c_i64, _c_i64, ctypes.c_uint32,
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "tpconv_csr_transpose_workspace_bytes": (ctypes.c_int, [_c_i64, _c_i64, ctypes.POINTER(ctypes.c_size_t)]),
    "tpconv_csr_transpose": (ctypes.c_int, [_c_i64, _c_i64] + [_c_p] * 6 + [ctypes.c_size_t, _c_p]),
    "tpconv_validate_graph": (ctypes.c_int, [_c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    "tpconv_forward": (ctypes.c_int, [_c_p, _c_i64, _c_i64] + [_c_p] * 7 + [ctypes.c_size_t, _c_p]),
    "tpconv_backward": (ctypes.c_int, [_c_p, _c_i64, _c_i64] + [_c_p] * 13 + [ctypes.c_size_t, _c_p]),
    "tpconv_double_backward": (ctypes.c_int, [_c_p, _c_i64, _c_i64] + [_c_p] * 17 + [ctypes.c_size_t, _c_p]),
    "tpconv_forward_embedded": (ctypes.c_int, [_c_p, _c_i64, _c_i64] + [_c_p] * 8 + [ctypes.c_size_t, _c_p]),
    "tpconv_backward_embedded": (ctypes.c_int, [_c_p, _c_i64, _c_i64] + [_c_p] * 15 + [ctypes.c_size_t, _c_p]),
    "tpconv_profile_begin": (ctypes.c_int, [ctypes.c_int32]),
    "tpconv_profile_end": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_c_i64), ctypes.c_int32]),
    "tpconv_profile_category_name": (ctypes.c_char_p, [ctypes.c_int32]),
    "tpconv_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32)]),
    "tpconv_forward_no_alloc": (ctypes.c_int, [_c_p, _c_i64, _c_i64] + [_c_p] * 6 + [_c_p]),
    # include/tpconv_graph.h
    "tpconv_spatial_order_workspace_bytes": (ctypes.c_int, [_c_i64, ctypes.POINTER(ctypes.c_size_t)]),
    "tpconv_spatial_order": (ctypes.c_int, [_c_i64, _c_p, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "tpconv_permute_graph": (ctypes.c_int, [_c_i64, _c_i64] + [_c_p] * 6 + [_c_p]),
    "tpconv_gather_rows": (ctypes.c_int, [_c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    # include/tpconv_node.h
    "tpconv_node_plan_create": (ctypes.c_int, [ctypes.POINTER(_c_p), ctypes.c_char_p, ctypes.c_int32,
                                               ctypes.c_float]),
    "tpconv_node_plan_destroy": (ctypes.c_int, [_c_p]),
    "tpconv_node_plan_info": (ctypes.c_int, [_c_p] + [ctypes.POINTER(_c_i64)] * 4),
    "tpconv_node_plan_set_layout": (ctypes.c_int, [_c_p, ctypes.c_int32]),
    "tpconv_node_workspace_bytes": (ctypes.c_int, [_c_p, _c_i64, ctypes.POINTER(ctypes.c_size_t)]),
    "tpconv_norm_forward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 5),
    "tpconv_norm_backward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 7 + [ctypes.c_size_t, _c_p]),
    "tpconv_norm_double_backward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 10 + [ctypes.c_size_t, _c_p]),
    "tpconv_dropout_forward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 5),
    "tpconv_dropout_backward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 4),
    "tpconv_dropout_norm_forward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 8),
    "tpconv_dropout_norm_backward": (ctypes.c_int, [_c_p, _c_i64] + [_c_p] * 10 + [ctypes.c_size_t, _c_p]),
}
PROF_CATEGORIES = 14

_lib = None


def lib():
    """Load libtpconv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not found: build it with "
                               "`python -m equivariant_gnn_tensor_dst_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class TPConvError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        msg = lib().tpconv_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})" if where else msg)


def check(status, where=""):
    if status != 0:
        raise TPConvError(status, where)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

class Plan:
    """tpconv_plan_create / tpconv_plan_destroy and the introspection calls."""

    def __init__(self, irreps_in, sh_lmax, irreps_out, mode="uvw", radial="bessel", num_basis=8,
                 r_cut=5.0, r_min=0.0, r_max=0.0, poly_p=6):
        spec = RadialSpec(BESSEL if radial == "bessel" else GAUSSIAN, int(num_basis), float(r_cut),
                          float(r_min), float(r_max), int(poly_p))
        h = _c_p()
        m = UVW if mode == "uvw" else UVU
        check(lib().tpconv_plan_create(ctypes.byref(h), irreps_in.encode(), int(sh_lmax),
                                       irreps_out.encode(), m, ctypes.byref(spec)), "tpconv_plan_create")
        self._h = h
        self.mode = mode
        vals = [_c_i64() for _ in range(5)]
        check(lib().tpconv_plan_info(h, *[ctypes.byref(v) for v in vals]), "tpconv_plan_info")
        self.num_paths, self.dim_in, self.dim_out, self.num_basis, self.weight_cols = (v.value for v in vals)

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().tpconv_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def path(self, i):
        out = (ctypes.c_int32 * 10)()
        check(lib().tpconv_plan_path(self._h, i, out), "tpconv_plan_path")
        keys = ("l_in", "l_sh", "l_out", "block_in", "block_out", "c_in", "c_out", "w_offset",
                "w_count", "nnz")
        return dict(zip(keys, list(out)))

    def paths(self):
        return [self.path(i) for i in range(self.num_paths)]

    def coupling(self, i):
        nnz = self.path(i)["nnz"]
        idx = (ctypes.c_int32 * (3 * max(nnz, 1)))()
        val = (ctypes.c_double * max(nnz, 1))()
        check(lib().tpconv_plan_path_coupling(self._h, i, idx, val, nnz), "tpconv_plan_path_coupling")
        return [tuple(idx[3 * k:3 * k + 3]) for k in range(nnz)], [val[k] for k in range(nnz)]

    def set_workspace_budget(self, nbytes):
        check(lib().tpconv_set_workspace_budget(self._h, int(nbytes)), "tpconv_set_workspace_budget")

    def set_layout(self, layout):
        """LAYOUT_IR_MUL (default, blocks [2l+1][C]) or LAYOUT_MUL_IR (blocks [C][2l+1])."""
        check(lib().tpconv_plan_set_layout(self._h, int(layout)), "tpconv_plan_set_layout")

    def set_math(self, math):
        """MATH_FP32 (default, 3xTF32 contractions), MATH_TF32 (one TF32 product) or
        MATH_BF16 (operands rounded to bf16, one bf16 product)."""
        check(lib().tpconv_plan_set_math(self._h, int(math)), "tpconv_plan_set_math")

    def workspace_bytes(self, n_nodes, n_edges, passes=PASS_FORWARD | PASS_BACKWARD | PASS_DOUBLE_BACKWARD):
        out = ctypes.c_size_t()
        check(lib().tpconv_workspace_bytes(self._h, int(n_nodes), int(n_edges), int(passes),
                                           ctypes.byref(out)), "tpconv_workspace_bytes")
        return out.value

    def fan_in_per_column(self):
        """Per weight column fan-in K*C_in (uvw) or K (uvu), for N(0, 1/fan_in) init."""
        import numpy as np
        f = np.zeros(self.weight_cols)
        for p in self.paths():
            f[p["w_offset"]:p["w_offset"] + p["w_count"]] = self.num_basis * (p["c_in"] if self.mode == "uvw" else 1)
        return f


# ---------------------------------------------------------------------------
# torch-facing calls
#
# A call with stream= runs as inside torch.cuda.stream(stream): inputs have to be ready there, and
# outputs that are used on another stream follow torch's rule for such tensors (wait for the stream;
# Tensor.record_stream before the tensor is dropped).
# ---------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _on(call, args):
    """A call with its arguments (by name, its stream among them) on that stream: its outputs and its
    workspace are made there, too.  The allocator gives a block away again in the order of the stream
    that it was made on, so a workspace that is dropped when the call returns, its kernels still queued,
    is safe there, and a new block has no work of another stream pending."""
    import torch
    stream = args.pop("stream")
    if (stream.cuda_stream == torch._C._cuda_getCurrentRawStream(stream.device_index)
            and stream.device_index == torch._C._cuda_getDevice()):
        return call(**args)     # entering the current stream all the same takes ten microseconds
    for name, a in args.items():
        if isinstance(a, torch.Tensor) and a.get_device() != stream.device_index:
            raise ValueError(f"the stream is on {stream.device}, {name} on {a.device}")
    with torch.cuda.stream(stream):
        return call(**args)


def _need(t, dtype, name):
    import torch
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def workspace(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def tpconv_csr_transpose(row_ptr, src, n_nodes, stream=None):
    if stream is not None:
        return _on(tpconv_csr_transpose, locals())
    import torch
    _need(row_ptr, torch.int32, "row_ptr")
    _need(src, torch.int32, "src")
    E = src.numel()
    dev = row_ptr.device
    t_ptr = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
    t_eid = torch.empty(max(E, 1), dtype=torch.int32, device=dev)
    t_dst = torch.empty(max(E, 1), dtype=torch.int32, device=dev)
    nb = ctypes.c_size_t()
    check(lib().tpconv_csr_transpose_workspace_bytes(n_nodes, E, ctypes.byref(nb)))
    ws = workspace(nb.value, dev)
    check(lib().tpconv_csr_transpose(n_nodes, E, _ptr(row_ptr), _ptr(src), _ptr(t_ptr), _ptr(t_eid),
                                     _ptr(t_dst), _ptr(ws), ws.numel(), _stream()),
          "tpconv_csr_transpose")
    return t_ptr, t_eid[:E], t_dst[:E]


def tpconv_validate_graph(row_ptr, src, n_nodes, stream=None):
    if stream is not None:
        return _on(tpconv_validate_graph, locals())
    import torch
    err = torch.zeros(4, dtype=torch.int32, device=row_ptr.device)
    check(lib().tpconv_validate_graph(n_nodes, src.numel(), _ptr(row_ptr), _ptr(src), _ptr(err),
                                      _stream()), "tpconv_validate_graph")
    return err[:1]


def tpconv_forward(plan, x, pos, row_ptr, src, W, out=None, ws=None, stream=None):
    if stream is not None:
        return _on(tpconv_forward, locals())
    import torch
    for t, n in ((x, "x"), (pos, "pos"), (W, "W")):
        _need(t, torch.float32, n)
    _need(row_ptr, torch.int32, "row_ptr")
    _need(src, torch.int32, "src")
    N, E = pos.shape[0], src.numel()
    if out is None:
        out = torch.empty(N, plan.dim_out, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(plan.workspace_bytes(N, E, PASS_FORWARD), x.device)
    check(lib().tpconv_forward(plan.handle, N, E, _ptr(x), _ptr(pos), _ptr(row_ptr), _ptr(src), _ptr(W),
                               _ptr(out), _ptr(ws), ws.numel(), _stream()), "tpconv_forward")
    return out


def tpconv_backward(plan, x, pos, row_ptr, src, t_ptr, t_eid, t_dst, W, grad_out, need_x=True,
                    need_pos=True, need_W=True, ws=None, outputs=None, stream=None):
    if stream is not None:
        return _on(tpconv_backward, locals())
    import torch
    N, E = pos.shape[0], src.numel()
    dev = x.device
    if outputs is None:
        gx = torch.empty(N, plan.dim_in, dtype=torch.float32, device=dev) if need_x else None
        gp = torch.empty(N, 3, dtype=torch.float32, device=dev) if need_pos else None
        gw = torch.empty(plan.num_basis, plan.weight_cols, dtype=torch.float32, device=dev) if need_W else None
    else:
        gx, gp, gw = outputs
    if ws is None:
        ws = workspace(plan.workspace_bytes(N, E, PASS_BACKWARD), dev)
    check(lib().tpconv_backward(plan.handle, N, E, _ptr(x), _ptr(pos), _ptr(row_ptr), _ptr(src),
                                _ptr(t_ptr), _ptr(t_eid), _ptr(t_dst), _ptr(W), _ptr(grad_out),
                                _ptr(gx), _ptr(gp), _ptr(gw), _ptr(ws), ws.numel(), _stream()),
          "tpconv_backward")
    return gx, gp, gw


def tpconv_forward_embedded(plan, x, Y, phi, row_ptr, src, W, out=None, ws=None, stream=None):
    """Forward with the edge embedding given per edge: Y [E, (lmax+1)^2], phi [E, K]."""
    if stream is not None:
        return _on(tpconv_forward_embedded, locals())
    import torch
    for t, n in ((x, "x"), (Y, "Y"), (phi, "phi"), (W, "W")):
        _need(t, torch.float32, n)
    _need(row_ptr, torch.int32, "row_ptr")
    _need(src, torch.int32, "src")
    N, E = row_ptr.numel() - 1, src.numel()
    if out is None:
        out = torch.empty(N, plan.dim_out, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(plan.workspace_bytes(N, E, PASS_FORWARD), x.device)
    check(lib().tpconv_forward_embedded(plan.handle, N, E, _ptr(x), _ptr(Y), _ptr(phi), _ptr(row_ptr), _ptr(src),
                                        _ptr(W), _ptr(out), _ptr(ws), ws.numel(), _stream()),
          "tpconv_forward_embedded")
    return out


def tpconv_backward_embedded(plan, x, Y, phi, row_ptr, src, t_ptr, t_eid, t_dst, W, grad_out, need_x=True,
                             need_W=True, need_phi=True, need_Y=True, ws=None, outputs=None, stream=None):
    """Returns (grad_x, grad_W, grad_phi [E, K], grad_Y [E, (lmax+1)^2])."""
    if stream is not None:
        return _on(tpconv_backward_embedded, locals())
    import torch
    N, E = row_ptr.numel() - 1, src.numel()
    dev = x.device
    if outputs is None:
        gx = torch.empty(N, plan.dim_in, dtype=torch.float32, device=dev) if need_x else None
        gw = torch.empty(plan.num_basis, plan.weight_cols, dtype=torch.float32, device=dev) if need_W else None
        gphi = torch.empty(E, plan.num_basis, dtype=torch.float32, device=dev) if need_phi else None
        gY = torch.empty(E, Y.shape[1], dtype=torch.float32, device=dev) if need_Y else None
    else:
        gx, gw, gphi, gY = outputs
    if ws is None:
        ws = workspace(plan.workspace_bytes(N, E, PASS_BACKWARD), dev)
    check(lib().tpconv_backward_embedded(plan.handle, N, E, _ptr(x), _ptr(Y), _ptr(phi), _ptr(row_ptr), _ptr(src),
                                         _ptr(t_ptr), _ptr(t_eid), _ptr(t_dst), _ptr(W), _ptr(grad_out),
                                         _ptr(gx), _ptr(gw), _ptr(gphi), _ptr(gY), _ptr(ws), ws.numel(),
                                         _stream()),
          "tpconv_backward_embedded")
    return gx, gw, gphi, gY


def tpconv_double_backward(plan, x, pos, row_ptr, src, t_ptr, t_eid, t_dst, W, grad_out, gg_x=None,
                           gg_pos=None, gg_W=None, need_x=True, need_W=True, need_grad_out=True,
                           need_pos=False, ws=None, outputs=None, stream=None):
    """Returns (grad_x, grad_W, grad_grad_out), plus grad_pos [N, 3] when need_pos
    (``outputs`` then has four entries)."""
    if stream is not None:
        return _on(tpconv_double_backward, locals())
    import torch
    N, E = pos.shape[0], src.numel()
    dev = x.device
    if outputs is None:
        gx = torch.empty(N, plan.dim_in, dtype=torch.float32, device=dev) if need_x else None
        gw = torch.empty(plan.num_basis, plan.weight_cols, dtype=torch.float32, device=dev) if need_W else None
        gg = torch.empty(N, plan.dim_out, dtype=torch.float32, device=dev) if need_grad_out else None
        gp = torch.empty(N, 3, dtype=torch.float32, device=dev) if need_pos else None
    elif need_pos:
        gx, gw, gg, gp = outputs
    else:
        (gx, gw, gg), gp = outputs, None
    if ws is None:
        ws = workspace(plan.workspace_bytes(N, E, PASS_DOUBLE_BACKWARD), dev)
    check(lib().tpconv_double_backward(plan.handle, N, E, _ptr(x), _ptr(pos), _ptr(row_ptr), _ptr(src),
                                       _ptr(t_ptr), _ptr(t_eid), _ptr(t_dst), _ptr(W), _ptr(grad_out),
                                       _ptr(gg_x), _ptr(gg_pos), _ptr(gg_W), _ptr(gx), _ptr(gw), _ptr(gg),
                                       _ptr(gp), _ptr(ws), ws.numel(), _stream()),
          "tpconv_double_backward")
    return (gx, gw, gg, gp) if need_pos else (gx, gw, gg)


def tpconv_spatial_order(pos, stream=None):
    """perm [N] int32: nodes in Morton order of their positions (perm[k] = old id)."""
    if stream is not None:
        return _on(tpconv_spatial_order, locals())
    import torch
    _need(pos, torch.float32, "pos")
    N = pos.shape[0]
    perm = torch.empty(max(N, 1), dtype=torch.int32, device=pos.device)
    nb = ctypes.c_size_t()
    check(lib().tpconv_spatial_order_workspace_bytes(N, ctypes.byref(nb)), "tpconv_spatial_order_workspace_bytes")
    ws = workspace(nb.value, pos.device)
    check(lib().tpconv_spatial_order(N, _ptr(pos), _ptr(perm), _ptr(ws), ws.numel(), _stream()),
          "tpconv_spatial_order")
    return perm[:N]


def tpconv_permute_graph(row_ptr, src, perm, stream=None):
    """The receiver CSR renumbered by perm: (row_ptr_out, src_out, inv)."""
    if stream is not None:
        return _on(tpconv_permute_graph, locals())
    import torch
    _need(row_ptr, torch.int32, "row_ptr")
    _need(src, torch.int32, "src")
    _need(perm, torch.int32, "perm")
    N, E = row_ptr.numel() - 1, src.numel()
    dev = row_ptr.device
    rp = torch.empty(N + 1, dtype=torch.int32, device=dev)
    so = torch.empty(max(E, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(N, 1), dtype=torch.int32, device=dev)
    check(lib().tpconv_permute_graph(N, E, _ptr(row_ptr), _ptr(src), _ptr(perm), _ptr(rp), _ptr(so), _ptr(inv),
                                     _stream()), "tpconv_permute_graph")
    return rp, so[:E], inv[:N]


def tpconv_gather_rows(a, perm, stream=None):
    """out[k] = a[perm[k]] for a 2-D float32 array (node features, positions)."""
    if stream is not None:
        return _on(tpconv_gather_rows, locals())
    import torch
    _need(a, torch.float32, "a")
    _need(perm, torch.int32, "perm")
    rows, width = a.shape[0], (a.numel() // a.shape[0] if a.shape[0] else 0)
    if perm.numel() != rows:
        raise ValueError(f"perm must have {rows} entries, not {perm.numel()}")
    out = torch.empty_like(a)
    check(lib().tpconv_gather_rows(perm.numel(), width, _ptr(a), _ptr(perm), _ptr(out), _stream()),
          "tpconv_gather_rows")
    return out


# ---------------------------------------------------------------------------
# node-feature operators (include/tpconv_node.h)
# ---------------------------------------------------------------------------

_torch = None   # torch, once a NodePlan exists (an import statement in every call costs)


class NodePlan:
    """tpconv_node_plan_create / _destroy: rows of an irreps string in a storage type
    (torch.float32, bfloat16 or float16), the norm's eps and the layout ("ir_mul" or
    "mul_ir", or the LAYOUT_ constants)."""

    def __init__(self, irreps, dtype=None, eps=1e-5, layout=LAYOUT_IR_MUL):
        global _torch
        import torch
        _torch = torch
        dtype = torch.float32 if dtype is None else dtype
        codes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
        if dtype not in codes:
            raise ValueError(f"dtype must be one of {sorted(map(str, codes))}")
        if isinstance(layout, str):
            if layout not in ("ir_mul", "mul_ir"):
                raise ValueError("layout must be 'ir_mul' or 'mul_ir'")
            layout = LAYOUT_MUL_IR if layout == "mul_ir" else LAYOUT_IR_MUL
        h = _c_p()
        check(lib().tpconv_node_plan_create(ctypes.byref(h), irreps.encode(), codes[dtype], float(eps)),
              "tpconv_node_plan_create")
        self._h = h
        self.dtype, self.eps = dtype, float(eps)
        vals = [_c_i64() for _ in range(4)]
        check(lib().tpconv_node_plan_info(h, *[ctypes.byref(v) for v in vals]), "tpconv_node_plan_info")
        self.dim, self.channels, self.biases, self.num_blocks = (v.value for v in vals)
        self.set_layout(layout)

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().tpconv_node_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_layout(self, layout):
        """LAYOUT_IR_MUL (blocks [2l+1][C]) or LAYOUT_MUL_IR (blocks [C][2l+1])."""
        check(lib().tpconv_node_plan_set_layout(self._h, int(layout)), "tpconv_node_plan_set_layout")

    def workspace_bytes(self, n_rows):
        """Workspace of norm and dropout-norm backward and of the double backward."""
        out = ctypes.c_size_t()
        check(lib().tpconv_node_workspace_bytes(self._h, int(n_rows), ctypes.byref(out)),
              "tpconv_node_workspace_bytes")
        return out.value


class Dropout:
    """tpconv_dropout_spec: probability p of dropping, seed, offset (one per layer and step) and
    an optional device int64 ``step`` that the kernels add to the offset when they run."""

    def __init__(self, p, seed, offset=0, step=None):
        import torch
        if not 0.0 <= float(p) <= 1.0:
            raise ValueError("p must be in [0, 1]")
        if step is not None:
            _need(step, torch.int64, "step")
            if step.numel() != 1:
                raise ValueError("step must hold one value")
        self.step = step            # kept alive with the spec
        self._spec = DropoutSpec(float(p), int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1),
                                 None if step is None else step.data_ptr())
        self._ref = ctypes.byref(self._spec)

    def spec(self, device):
        """The structure for a call on ``device``."""
        if self.step is not None and self.step.device != device:
            raise ValueError(f"step must be on {device}")
        return self._ref

    @property
    def p(self):
        return self._spec.p

    @property
    def seed(self):
        return self._spec.seed

    @property
    def offset(self):
        return self._spec.offset

    @offset.setter
    def offset(self, value):
        self._spec.offset = int(value) & (2 ** 64 - 1)


def _node_bad(t, name, dtype, shape, device):
    """Says what is wrong with an array that failed the one-line check."""
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    raise ValueError(f"{name} must be on {device}")


def _node_x(plan, x, name):
    """Checks the array that sets a call's rows and device; its address."""
    shape = x.shape
    if not (x.is_cuda and x.dtype is plan.dtype and x.is_contiguous() and len(shape) == 2 and shape[1] == plan.dim):
        _need(x, plan.dtype, name)
        raise ValueError(f"{name} must be [rows, {plan.dim}], not {list(shape)}")
    return x.data_ptr()


def _node_row(t, name, x):
    """Address of a node array like x (0: None)."""
    if t is None:
        return 0
    if not (t.dtype is x.dtype and t.shape == x.shape and t.get_device() == x.get_device() and t.is_contiguous()):
        _node_bad(t, name, x.dtype, x.shape, x.device)
    return t.data_ptr()


def _node_vec(t, n, name, x):
    """Address of a float32 channel vector of n values on x's device (0: None)."""
    if t is None:
        return 0
    if not (t.dtype is _torch.float32 and t.numel() == n and t.get_device() == x.get_device() and t.is_contiguous()):
        _node_bad(t, name, _torch.float32, (n,), x.device)
    return t.data_ptr()


def _node_new(like, need):
    """A new array like another and its address."""
    if not need:
        return None, 0
    t = _torch.empty_like(like)
    return t, t.data_ptr()


def _node_sums(like, n, need, device):
    """A new channel vector (like another, where there is one) and its address."""
    if not need:
        return None, 0
    t = _torch.empty_like(like) if like is not None else _torch.empty(n, dtype=_torch.float32, device=device)
    return t, t.data_ptr()


def _node_call(device, name, *args):
    """One library call on the tensors' device and that device's current stream."""
    if device.index != _torch._C._cuda_getDevice():
        with _torch.cuda.device(device):
            return _node_call(device, name, *args)
    # the handle itself: building a torch Stream object costs several microseconds
    raw = _torch._C._cuda_getCurrentRawStream(device.index)
    status = getattr(_lib, name)(*args, raw)
    if status:
        raise TPConvError(status, name)


def _node_ws(plan, N, ws, device):
    """(workspace, address, bytes)"""
    if ws is None:
        ws = workspace(plan.workspace_bytes(N), device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous and on {device}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def tpconv_norm_forward(plan, x, weight=None, bias=None, out=None, stream=None):
    """Irreps layer norm of node rows x [N, dim]; weight [channels], bias [biases] float32."""
    if stream is not None:
        return _on(tpconv_norm_forward, locals())
    px = _node_x(plan, x, "x")
    pw, pb = _node_vec(weight, plan.channels, "weight", x), _node_vec(bias, plan.biases, "bias", x)
    out, po = _node_new(x, True) if out is None else (out, _node_row(out, "out", x))
    _node_call(x.device, "tpconv_norm_forward", plan._h, x.shape[0], px, pw, pb, po)
    return out


def tpconv_norm_backward(plan, x, weight, grad_y, need_x=True, need_weight=True, need_bias=True, ws=None,
                         outputs=None, stream=None):
    """Returns (grad_x [N, dim], grad_weight [channels], grad_bias [biases])."""
    if stream is not None:
        return _on(tpconv_norm_backward, locals())
    dev, N, C, Cb = x.device, x.shape[0], plan.channels, plan.biases
    px, pg, pw = _node_x(plan, x, "x"), _node_row(grad_y, "grad_y", x), _node_vec(weight, C, "weight", x)
    if outputs is None:
        gx, pgx = _node_new(x, need_x)
        gw, pgw = _node_sums(weight, C, need_weight, dev)
        gb, pgb = _node_sums(None, Cb, need_bias, dev)
    else:
        gx, gw, gb = outputs
        pgx = _node_row(gx, "grad_x", x)
        pgw, pgb = _node_vec(gw, C, "grad_weight", x), _node_vec(gb, Cb, "grad_bias", x)
    ws, pws, nws = _node_ws(plan, N, ws, dev)
    _node_call(dev, "tpconv_norm_backward", plan._h, N, px, pw, pg, pgx, pgw, pgb, pws, nws)
    return gx, gw, gb


def tpconv_norm_double_backward(plan, x, weight, grad_y, gg_x=None, gg_weight=None, gg_bias=None, need_x=True,
                                need_weight=True, need_grad_y=True, ws=None, outputs=None, stream=None):
    """Returns (grad_x [N, dim], grad_weight [channels], grad_grad_y [N, dim])."""
    if stream is not None:
        return _on(tpconv_norm_double_backward, locals())
    dev, N, C = x.device, x.shape[0], plan.channels
    px, pg, pp = _node_x(plan, x, "x"), _node_row(grad_y, "grad_y", x), _node_row(gg_x, "gg_x", x)
    pw, pt = _node_vec(weight, C, "weight", x), _node_vec(gg_weight, C, "gg_weight", x)
    ptb = _node_vec(gg_bias, plan.biases, "gg_bias", x)
    if outputs is None:
        gx, pgx = _node_new(x, need_x)
        gw, pgw = _node_sums(weight, C, need_weight, dev)
        gg, pgg = _node_new(x, need_grad_y)
    else:
        gx, gw, gg = outputs
        pgx, pgg = _node_row(gx, "grad_x", x), _node_row(gg, "grad_grad_y", x)
        pgw = _node_vec(gw, C, "grad_weight", x)
    ws, pws, nws = _node_ws(plan, N, ws, dev)
    _node_call(dev, "tpconv_norm_double_backward", plan._h, N, px, pw, pg, pp, pt, ptb, pgx, pgw, pgg, pws,
               nws)
    return gx, gw, gg


def tpconv_dropout_forward(plan, x, dropout, residual=None, out=None, stream=None):
    """residual + dropout(x); ``dropout`` is a Dropout.  out may be x or residual (in place)."""
    if stream is not None:
        return _on(tpconv_dropout_forward, locals())
    px, pr = _node_x(plan, x, "x"), _node_row(residual, "residual", x)
    out, po = _node_new(x, True) if out is None else (out, _node_row(out, "out", x))
    _node_call(x.device, "tpconv_dropout_forward", plan._h, x.shape[0], px, pr, dropout.spec(x.device), po)
    return out


def tpconv_dropout_backward(plan, grad_out, dropout, out=None, stream=None):
    """grad_x of tpconv_dropout_forward (the residual's gradient is grad_out itself)."""
    if stream is not None:
        return _on(tpconv_dropout_backward, locals())
    pg = _node_x(plan, grad_out, "grad_out")
    out, po = _node_new(grad_out, True) if out is None else (out, _node_row(out, "out", grad_out))
    _node_call(grad_out.device, "tpconv_dropout_backward", plan._h, grad_out.shape[0], pg,
               dropout.spec(grad_out.device), po)
    return out


def tpconv_dropout_norm_forward(plan, x, dropout, residual=None, weight=None, bias=None, outputs=None, stream=None):
    """Returns (z, y): z = residual + dropout(x), y = norm(z)."""
    if stream is not None:
        return _on(tpconv_dropout_norm_forward, locals())
    px, pr = _node_x(plan, x, "x"), _node_row(residual, "residual", x)
    pw, pb = _node_vec(weight, plan.channels, "weight", x), _node_vec(bias, plan.biases, "bias", x)
    if outputs is None:
        (z, pz), (y, py) = _node_new(x, True), _node_new(x, True)
    else:
        z, y = outputs
        pz, py = _node_row(z, "z", x), _node_row(y, "y", x)
    _node_call(x.device, "tpconv_dropout_norm_forward", plan._h, x.shape[0], px, pr, dropout.spec(x.device),
               pw, pb, pz, py)
    return z, y


def tpconv_dropout_norm_backward(plan, z, weight, grad_y, dropout, grad_z=None, need_x=True, need_residual=True,
                                 need_weight=True, need_bias=True, ws=None, outputs=None, stream=None):
    """Returns (grad_x, grad_residual, grad_weight, grad_bias) from the stored z."""
    if stream is not None:
        return _on(tpconv_dropout_norm_backward, locals())
    dev, N, C, Cb = z.device, z.shape[0], plan.channels, plan.biases
    pz, pg, pgz = _node_x(plan, z, "z"), _node_row(grad_y, "grad_y", z), _node_row(grad_z, "grad_z", z)
    pw = _node_vec(weight, C, "weight", z)
    if outputs is None:
        gx, pgx = _node_new(z, need_x)
        gr, pgr = _node_new(z, need_residual)
        gw, pgw = _node_sums(weight, C, need_weight, dev)
        gb, pgb = _node_sums(None, Cb, need_bias, dev)
    else:
        gx, gr, gw, gb = outputs
        pgx, pgr = _node_row(gx, "grad_x", z), _node_row(gr, "grad_residual", z)
        pgw, pgb = _node_vec(gw, C, "grad_weight", z), _node_vec(gb, Cb, "grad_bias", z)
    ws, pws, nws = _node_ws(plan, N, ws, dev)
    _node_call(dev, "tpconv_dropout_norm_backward", plan._h, N, pz, pw, pg, pgz, dropout.spec(dev), pgx, pgr,
               pgw, pgb, pws, nws)
    return gx, gr, gw, gb


def tpconv_profile_begin(max_records=8192):
    check(lib().tpconv_profile_begin(int(max_records)), "tpconv_profile_begin")


def tpconv_profile_end():
    """Returns {category: (milliseconds, launches)} for the launches since begin()."""
    n = PROF_CATEGORIES
    ms = (ctypes.c_double * n)()
    cnt = (_c_i64 * n)()
    check(lib().tpconv_profile_end(ms, cnt, n), "tpconv_profile_end")
    return {lib().tpconv_profile_category_name(c).decode(): (ms[c], cnt[c]) for c in range(n)}


def tpconv_device_error():
    """Read and clear the library's device error word (0 = no bounded wait gave up)."""
    v = ctypes.c_int32()
    check(lib().tpconv_device_error(ctypes.byref(v)), "tpconv_device_error")
    return v.value

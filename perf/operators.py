"""Cases and plain forms of the node-feature operators: irreps layer norm, equivariant dropout, and the two fused
with the residual sum.  ``own`` selects the library's kernels; otherwise ``run`` evaluates the operators in elementary
torch operations in float32.

A node row is the concatenation of the irrep blocks of a string such as "128x0e+64x1o": C channels of order l, stored
[2l+1][C] (layout "ir_mul") or [C][2l+1] ("mul_ir").
"""

import math
import re

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = "8x0e+8x1o+8x2e"                       # output of the tiny workload's convolution
EVEN64 = "64x0e+64x1o+64x2e"                  # uvw forward + backward workload
EVEN128 = "128x0e+128x1o+128x2e"              # channelwise workload
MIXED = "128x0e+64x1o+32x2e+16x3o"            # edge-scaling workload
FORCE = "32x0e+32x1o+32x2e"                   # force-training workload


def _case(name, op, step, irreps, rows, dtype="f32", layout="ir_mul", p=0.0, residual=False):
    return {"name": name, "op": op, "pass": step, "irreps": irreps, "rows": rows, "dtype": dtype, "layout": layout,
            "p": p, "residual": residual}


def listed():
    return [
        # a molecule's features between two layers: the latency of one small call
        _case("norm fwd tiny", "norm", "forward", TINY, 64),
        # the largest graph's node features
        _case("norm fwd mixed 50000", "norm", "forward", MIXED, 50000),
        # training step of the channelwise workload
        _case("norm bwd 128x 16384", "norm", "backward", EVEN128, 16384),
        # scalar features of a wide readout network, 16-bit storage
        _case("norm bwd 4096x0e bf16", "norm", "backward", "4096x0e", 8192, "bf16"),
        # odd channel counts, so that no row and no block starts on a 16-byte boundary
        _case("norm bwd odd f16 mul_ir", "norm", "backward", "37x0e+19x1o+6x2e+3x3o", 5001, "f16", "mul_ir"),
        # force training: the second derivative through the norm
        _case("norm dbl 32x 8192", "norm", "double_backward", FORCE, 8192),
        # a small graph's dropout
        _case("dropout fwd tiny", "dropout", "forward", TINY, 64, p=0.1),
        # residual branch of the largest graph
        _case("dropout fwd mixed 50000", "dropout", "forward", MIXED, 50000, p=0.1, residual=True),
        # gradient of the dropout in the channelwise workload, 16-bit storage
        _case("dropout bwd 128x bf16", "dropout", "backward", EVEN128, 16384, "bf16", p=0.25),
        # between two layers of the uvw workload
        _case("drop-norm fwd 64x 4096", "dropout_norm", "forward", EVEN64, 4096, p=0.1, residual=True),
        # between two layers of the edge-scaling workload, backward
        _case("drop-norm bwd mixed 50000", "dropout_norm", "backward", MIXED, 50000, p=0.1, residual=True),
        # odd channel counts in 16 bits, components innermost
        _case("drop-norm fwd odd bf16", "dropout_norm", "forward", "37x0e+19x1o+6x2e+3x3o", 7777, "bf16", "mul_ir",
              p=0.5, residual=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, step = rng.choice([("norm", "forward"), ("norm", "backward"), ("norm", "double_backward"),
                           ("dropout", "forward"), ("dropout", "backward"), ("dropout_norm", "forward"),
                           ("dropout_norm", "backward")])
    if rng.random() < 0.25:                    # scalars only
        irreps = "%dx0e" % _log_int(rng, 4, 8192)
    else:
        orders = sorted(rng.sample(["0e", "0o", "1o", "1e", "2e", "3o"], rng.randint(1, 4)))
        unit = rng.choice([1, 4, 16])          # odd counts, and multiples of a vector
        least = {"0": 4, "1": 2}               # one or two numbers have no spread to normalise by
        irreps = "+".join("%dx%s" % (max(unit, _log_int(rng, least.get(o[0], 1), 256) // unit * unit), o)
                          for o in orders)
    dim = sum(b[4] for b in _blocks(irreps))
    rows = _log_int(rng, 1, max(1, min(131072, 13000000 // dim)))
    return {"op": op, "pass": step, "irreps": irreps, "rows": rows, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
            "layout": rng.choice(["ir_mul", "ir_mul", "mul_ir"]),
            "p": rng.choice([0.0, 0.1, 0.3, 0.5, rng.random()]) if op != "norm" else 0.0,
            "residual": op != "norm" and step == "forward" and rng.random() < 0.7 or op == "dropout_norm"}


def _blocks(irreps):
    """(channels, components, centred, first element, elements, first channel) of each block."""
    out, off, ch = [], 0, 0
    for m, l, parity in re.findall(r"(\d+)x(\d)([eo])", irreps):
        c, d = int(m), 2 * int(l) + 1
        out.append((c, d, l == "0" and parity == "e", off, c * d, ch))
        off += c * d
        ch += c
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    blocks = _blocks(case["irreps"])
    rows, dim = int(case["rows"]), sum(b[4] for b in blocks)
    channels, biases = sum(b[0] for b in blocks), sum(b[0] for b in blocks if b[2])
    T = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": dict(case), "blocks": blocks, "dtype": T}
    # features: rows of different size, scalar channels with a common offset
    x = normal(rows, dim) * torch.exp(0.5 * normal(rows, 1))
    for c, d, centred, off, size, ch in blocks:
        if centred:
            x[:, off:off + size] += 0.5
    s["x"] = x.to(T)
    if case["op"] != "norm":
        s["p"], s["seed"], s["offset"] = float(case["p"]), (int(seed) * 2654435761 + 12345) % (1 << 63), 7 + int(seed) % 5
        s["residual"] = normal(rows, dim).to(T) if case["residual"] else None
    if case["op"] != "dropout":
        s["weight"], s["bias"] = 1.0 + 0.2 * normal(channels), 0.2 * normal(biases)
    if case["pass"] != "forward":
        s["grad"] = normal(rows, dim).to(T)
    if case["op"] == "dropout_norm" and case["pass"] == "backward":
        s["grad_z"] = normal(rows, dim).to(T)
    if case["pass"] == "double_backward":
        s["gg_x"], s["gg_weight"], s["gg_bias"] = normal(rows, dim).to(T), normal(channels), normal(biases)
    if own:
        from equivariant_gnn_tensor_dst_b200 import binding
        s["plan"] = binding.NodePlan(case["irreps"], T, EPS, case["layout"])
        if case["op"] != "norm":
            s["dropout"] = binding.Dropout(s["p"], s["seed"], s["offset"])
        if case["op"] != "dropout" and case["pass"] != "forward":
            s["ws"] = binding.workspace(s["plan"].workspace_bytes(rows), dev)
    return s


# ---- plain forms: float32, rounded once at the end ----

def _components(v, b, layout):
    """A block's columns as [rows, components, channels]."""
    c, d = b[0], b[1]
    return v.view(-1, d, c) if layout == "ir_mul" else v.view(-1, c, d).transpose(1, 2)


def _flat(v, layout):
    return (v if layout == "ir_mul" else v.transpose(1, 2)).reshape(v.shape[0], -1)


def _split(a, s):
    """The blocks of a node array in float32, each [rows, components, channels]."""
    lay = s["case"]["layout"]
    return [_components(a[:, b[3]:b[3] + b[4]].float(), b, lay) for b in s["blocks"]]


def _join(parts, s):
    return torch.cat([_flat(v, s["case"]["layout"]) for v in parts], 1)


def _mean(v):
    return v.mean((1, 2), keepdim=True)


def _centre(v, b):
    return v - _mean(v) if b[2] else v


def _stats(v, b):
    """h = r u and r of one block."""
    u = _centre(v, b)
    r = 1.0 / torch.sqrt(_mean(u * u) + EPS)
    return u * r, r


def _weight(w, b):
    return w[b[5]:b[5] + b[0]]


def _bias_offsets(blocks):
    return [sum(q[0] for q in blocks[:i] if q[2]) for i in range(len(blocks))]


def _norm(parts, s):
    at = _bias_offsets(s["blocks"])
    out = [_stats(v, b)[0] * _weight(s["weight"], b) for v, b in zip(parts, s["blocks"])]
    return [y + s["bias"][o:o + b[0]] if b[2] else y for y, b, o in zip(out, s["blocks"], at)]


def _norm_backward(parts, grads, s):
    gx, gw, gb = [], [], []
    for v, g, b in zip(parts, grads, s["blocks"]):
        h, r = _stats(v, b)
        a = _centre(g * _weight(s["weight"], b), b)
        gx.append(r * (a - h * _mean(a * h)))
        gw.append((g * h).sum((0, 1)))
        gb.append(g.sum((0, 1))[:b[0] if b[2] else 0])
    return gx, torch.cat(gw), torch.cat(gb)


def _norm_double_backward(s):
    gx, gw, gg = [], [], []
    at = _bias_offsets(s["blocks"])
    for v, g, p, b, o in zip(_split(s["x"], s), _split(s["grad"], s), _split(s["gg_x"], s), s["blocks"], at):
        h, r = _stats(v, b)
        w, q = _weight(s["weight"], b), _weight(s["gg_weight"], b)
        p, a, e = _centre(p, b), _centre(g * w, b), _centre(g * q, b)
        mp, ma = _mean(h * p), _mean(h * a)
        k = r * (p - h * mp)                   # the projection of the tangent
        t = s["gg_bias"][o:o + b[0]] if b[2] else 0.0
        gg.append(w * k + q * h + t)
        gw.append((g * k).sum((0, 1)))
        gx.append(r * r * (h * (3.0 * mp * ma - _mean(p * a)) - ma * p - mp * a) + r * (e - h * _mean(h * e)))
    return gx, torch.cat(gw), gg


def _philox(groups, rows, seed, offset, device):
    """Words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011) as
    [rows, groups, 4]: key = seed, counter = (group, row, offset)."""
    low = 0xFFFFFFFF
    c0 = torch.arange(groups, dtype=torch.int64, device=device).expand(rows, groups)
    c1 = torch.arange(rows, dtype=torch.int64, device=device).view(rows, 1).expand(rows, groups)
    c2, c3 = torch.full_like(c0, offset & low), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), -1)


def _dropout(parts, s):
    """Every channel of a node kept with probability 1 - p and scaled, or dropped with all its components.  Groups of
    four channels share a counter; each block starts a new group."""
    blocks, rows = s["blocks"], parts[0].shape[0]
    n = [(b[0] + 3) // 4 for b in blocks]
    words = _philox(sum(n), rows, s["seed"], s["offset"], parts[0].device).view(rows, -1)
    kept = words >= int(math.floor(s["p"] * 2.0 ** 32 + 0.5))
    scale = 1.0 / (1.0 - s["p"]) if s["p"] < 1.0 else 0.0
    masks = [kept[:, 4 * sum(n[:i]):4 * sum(n[:i]) + b[0]].unsqueeze(1) for i, b in enumerate(blocks)]
    return [torch.where(m, v * scale, torch.zeros_like(v)) for v, m in zip(parts, masks)]


def _plain(s):
    op, step, T = s["case"]["op"], s["case"]["pass"], s["dtype"]
    if op == "norm" and step == "forward":
        return {"y": _join(_norm(_split(s["x"], s), s), s).to(T)}
    if op == "norm" and step == "backward":
        gx, gw, gb = _norm_backward(_split(s["x"], s), _split(s["grad"], s), s)
        return {"grad_x": _join(gx, s).to(T), "grad_weight": gw, "grad_bias": gb}
    if op == "norm":
        gx, gw, gg = _norm_double_backward(s)
        return {"grad_x": _join(gx, s).to(T), "grad_weight": gw, "grad_grad_y": _join(gg, s).to(T)}
    if op == "dropout" and step == "forward":
        out = _join(_dropout(_split(s["x"], s), s), s)
        return {"out": (out + s["residual"].float() if s["residual"] is not None else out).to(T)}
    if op == "dropout":
        return {"grad_x": _join(_dropout(_split(s["grad"], s), s), s).to(T)}
    if step == "forward":
        z = _dropout(_split(s["x"], s), s)
        if s["residual"] is not None:
            z = [a + b for a, b in zip(z, _split(s["residual"], s))]
        return {"z": _join(z, s).to(T), "y": _join(_norm(z, s), s).to(T)}
    gx, gw, gb = _norm_backward(_split(s["x"], s), _split(s["grad"], s), s)      # x holds z here
    t = [a + b for a, b in zip(gx, _split(s["grad_z"], s))]
    return {"grad_x": _join(_dropout(t, s), s).to(T), "grad_residual": _join(t, s).to(T), "grad_weight": gw,
            "grad_bias": gb}


def _own(s):
    from equivariant_gnn_tensor_dst_b200 import binding
    op, step, plan = s["case"]["op"], s["case"]["pass"], s["plan"]
    if op == "norm" and step == "forward":
        return {"y": binding.tpconv_norm_forward(plan, s["x"], s["weight"], s["bias"])}
    if op == "norm" and step == "backward":
        gx, gw, gb = binding.tpconv_norm_backward(plan, s["x"], s["weight"], s["grad"], ws=s["ws"])
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if op == "norm":
        gx, gw, gg = binding.tpconv_norm_double_backward(plan, s["x"], s["weight"], s["grad"], s["gg_x"],
                                                         s["gg_weight"], s["gg_bias"], ws=s["ws"])
        return {"grad_x": gx, "grad_weight": gw, "grad_grad_y": gg}
    if op == "dropout" and step == "forward":
        return {"out": binding.tpconv_dropout_forward(plan, s["x"], s["dropout"], residual=s["residual"])}
    if op == "dropout":
        return {"grad_x": binding.tpconv_dropout_backward(plan, s["grad"], s["dropout"])}
    if step == "forward":
        z, y = binding.tpconv_dropout_norm_forward(plan, s["x"], s["dropout"], residual=s["residual"],
                                                   weight=s["weight"], bias=s["bias"])
        return {"z": z, "y": y}
    gx, gr, gw, gb = binding.tpconv_dropout_norm_backward(plan, s["x"], s["weight"], s["grad"], s["dropout"],
                                                          grad_z=s["grad_z"], ws=s["ws"])
    return {"grad_x": gx, "grad_residual": gr, "grad_weight": gw, "grad_bias": gb}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    blocks = _blocks(case["irreps"])
    dim, channels = sum(b[4] for b in blocks), sum(b[0] for b in blocks)
    biases = sum(b[0] for b in blocks if b[2])
    arrays, flops, params = {
        ("norm", "forward"): (2, 8, channels + biases),
        ("norm", "backward"): (3, 16, 2 * channels + biases),
        ("norm", "double_backward"): (5, 40, 3 * channels + biases),
        ("dropout", "forward"): (3 if case["residual"] else 2, 2, 0),
        ("dropout", "backward"): (2, 1, 0),
        ("dropout_norm", "forward"): (4 if case["residual"] else 3, 10, channels + biases),
        ("dropout_norm", "backward"): (5, 18, 2 * channels + biases),
    }[case["op"], case["pass"]]
    n = case["rows"] * dim
    return {"bytes": n * arrays * (4 if case["dtype"] == "f32" else 2) + 4 * params, "flops": n * flops}


# ---- the definition in 64 bits: gradients by automatic differentiation of the forward's definition ----

def _exact_norm(x, weight, bias, blocks, layout):
    out, k = [], 0
    for c, d, centred, off, size, ch in blocks:
        v = x[:, off:off + size]
        w = weight[ch:ch + c]
        w = w.repeat(d) if layout == "ir_mul" else w.repeat_interleave(d)
        if centred:
            v = v - v.sum(1, keepdim=True) / size
        y = v * torch.rsqrt((v ** 2).sum(1, keepdim=True) / size + EPS) * w
        if centred:
            y = y + bias[k:k + c]
            k += c
        out.append(y)
    return torch.cat(out, 1)


def _exact_mask(case, seed, offset, rows, blocks):
    """Scaled mask per element from the generator's definition, in unsigned host integers."""
    groups = sum(-(-b[0] // 4) for b in blocks)
    u, sh, lo = np.uint64, np.uint64(32), np.uint64(0xFFFFFFFF)
    ctr = [np.tile(np.arange(groups, dtype=u), rows), np.repeat(np.arange(rows, dtype=u), groups),
           np.full(rows * groups, offset % 2 ** 32, u), np.full(rows * groups, offset // 2 ** 32, u)]
    for i in range(10):
        k0, k1 = u((seed + i * 0x9E3779B9) % 2 ** 32), u((seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)
        first, second = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
        ctr = [(second >> sh) ^ ctr[1] ^ k0, second & lo, (first >> sh) ^ ctr[3] ^ k1, first & lo]
    words = np.stack(ctr, 1).reshape(rows, 4 * groups)
    p = case["p"]
    keep = torch.from_numpy(words >= u(math.floor(p * 2.0 ** 32 + 0.5))).cuda()
    cols, g = [], 0
    for c, d, _, _, _, _ in blocks:
        ch = torch.arange(c, device="cuda")
        cols.append(4 * g + (ch.repeat(d) if case["layout"] == "ir_mul" else ch.repeat_interleave(d)))
        g += -(-c // 4)
    return keep[:, torch.cat(cols)].double() * (1.0 / (1.0 - p) if p < 1.0 else 0.0)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    blocks, layout, rows = s["blocks"], case["layout"], int(case["rows"])
    f = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    mask = _exact_mask(case, s["seed"], s["offset"], rows, blocks) if case["op"] != "norm" else None
    if case["op"] == "dropout":
        if case["pass"] == "backward":
            return {"grad_x": f["grad"] * mask}
        return {"out": f["x"] * mask + (f["residual"] if f["residual"] is not None else 0.0)}
    w, b = f["weight"], f["bias"]
    if case["pass"] == "forward":
        if mask is None:
            return {"y": _exact_norm(f["x"], w, b, blocks, layout)}
        z = f["x"] * mask + (f["residual"] if f["residual"] is not None else 0.0)
        return {"z": z, "y": _exact_norm(z, w, b, blocks, layout)}
    leaves = [t.requires_grad_(True) for t in (f["x"], w, b)]
    y = _exact_norm(*leaves, blocks, layout)
    if case["pass"] == "backward":
        gx, gw, gb = torch.autograd.grad(y, leaves, f["grad"], allow_unused=True)
        gb = torch.zeros_like(b) if gb is None else gb
        if mask is None:
            return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
        t = gx + f["grad_z"]
        return {"grad_x": t * mask, "grad_residual": t, "grad_weight": gw, "grad_bias": gb}
    g = f["grad"].requires_grad_(True)
    first = torch.autograd.grad(y, leaves, g, create_graph=True, allow_unused=True)
    pairs = [(t, d) for t, d in zip(first, (f["gg_x"], f["gg_weight"], f["gg_bias"])) if t is not None]
    total = sum((t * d).sum() for t, d in pairs)
    gx, gw, gg = torch.autograd.grad(total, (f["x"], w, g))
    return {"grad_x": gx, "grad_weight": gw, "grad_grad_y": gg}

"""Error bounds of the layer norm's outputs where means are large, and float32 restatements of its
sums, right and wrong.

Bounds (first order, U = 2^-24, one block of S elements, all means over the block).  D = S / 256 + 20
additions one after another at most: a lane's pairs, then trees over lanes and warps, or S / 256
elements of a thread where a whole CTA holds a segment.
  mean         dmu  = (D + 2) U mean|x|, the same for all elements; u moves by dmu + U |u|
  mean square  dq   = (D + 5) U q + 2 dmu^2 (a common shift has no first-order part: u has no mean),
                      and 13 (D + 3) U q for a difference of sums, which is taken while mean^2 <= 4 q
                      (sum of squares 5 S q, product of means 4 S q with two more roundings)
  r            er   = dq r^2 / 2 + 6 U, relative (two units in the last place of the root, eps, 1/S)
  h = r u      dh   = r (dmu + U |u|) + (er + U) |h|
  a = w g      U |a|;  mean(a): dma = (D + 3) U mean|a|;  c = a - mean(a)
  mean(u c)    2 U mean|u a| + U mean|u c| + dmu (dma + U mean|a|) + (D + 2) U mean|u c|: neither
               common shift has a first-order part, because u and c have no means.  As a difference of
               sums: (D + 3) U (mean|x a| + 3 |mean x| mean|a|)
  m = mean(h c)  dm = r d(mean(u c)) + (er + 3 U) |m|
  grad_x = r (c - h m):  r (U |a| + dma + U |mean a|) + (er + 2 U) |r c| + r (dh |m| + |h| dm)
                         + (er + 4 U) |r h m| + U |grad_x|
  grad_weight  sum |g| dh + (terms + 2) U sum |g h|;  grad_bias  (terms) U sum |g|
An element error e0 that x already has (a sum that is not stored) adds mean(e0) to dmu, e0 to u,
2 mean(|u| e0) to q and mean(|c| e0) to mean(u c).
"""

import numpy as np

from node_helpers import U
from oracle import node


def _mean(v):
    return v.mean(axis=(1, 2), keepdims=True)


def _stats(R, b, v, e0):
    """u, h, r and the bounds of u's common shift, of r and of h."""
    D = b.size / 256 + 20
    u, dmu = v, 0.0
    if R.centred(b):
        u, dmu = v - _mean(v), (D + 2) * U * _mean(np.abs(v)) + _mean(e0)
    q = _mean(u * u)
    r = (q + R.eps) ** -0.5
    once = R.centred(b) * (_mean(v) ** 2 <= 4.1 * q)
    dq = (D + 5) * U * q + 2 * dmu ** 2 + 2 * _mean(np.abs(u) * e0) + once * 13 * (D + 3) * U * q
    er = 0.5 * dq * r * r + 6 * U
    h = u * r
    return D, u, h, r, dmu, once, er, r * (dmu + U * np.abs(u) + e0) + (er + U) * np.abs(h)


def forward_bound(R, x, w, bias, e0=None):
    out = []
    e0 = np.zeros_like(x) if e0 is None else e0
    for b, v, wb, c, e in zip(R.blocks, R.parts(x), R.split(w), R.split(bias, True), R.parts(e0)):
        _, _, h, _, _, _, _, dh = _stats(R, b, v, e)
        out.append(np.abs(wb) * dh + U * np.abs(wb * h + (0.0 if c is None else c)))
    return R.rows(out)


def backward_bound(R, x, w, gy):
    """(grad_x, grad_weight, grad_bias)"""
    gx, gw, gb = [], [], [np.zeros(0)]
    for b, v, g, wb in zip(R.blocks, R.parts(x), R.parts(gy), R.split(w)):
        D, u, h, r, dmu, once, er, dh = _stats(R, b, v, np.zeros_like(v))
        a = wb * g
        ma, dma = 0.0, 0.0
        if R.centred(b):
            ma, dma = _mean(a), (D + 3) * U * _mean(np.abs(a))
        c, A = a - ma, np.abs(a)
        m = _mean(h * c)
        duc = (2 * U * _mean(np.abs(u) * A) + (D + 3) * U * _mean(np.abs(u * c)) + dmu * (dma + U * _mean(A))
               + once * (D + 3) * U * (_mean(np.abs(v) * A) + 3 * np.abs(_mean(v)) * _mean(A)))
        dm = r * duc + (er + 3 * U) * np.abs(m)
        rhm = np.abs(r * h * m)
        gx.append(r * (U * A + dma + U * np.abs(ma)) + (er + 2 * U) * np.abs(r * c)
                  + r * (dh * np.abs(m) + np.abs(h) * dm) + (er + 4 * U) * rhm + U * np.abs(r * (c - h * m)))
        n = v.shape[0] * b.dim
        gw.append((np.abs(g) * dh).sum(axis=(0, 1)) + (n + 2) * U * np.abs(g * h).sum(axis=(0, 1)))
        if R.centred(b):
            gb.append(n * U * np.abs(g).sum(axis=(0, 1)))
    return R.rows(gx), np.concatenate(gw), np.concatenate(gb)


# ---- float32 restatements of a row of scalars ----

f32 = np.float32


def _fma(a, b, c):
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(f32)


def _tree(v):
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    return v


def _dot(a, b):
    """Sum of products: pairs of a lane one after another, then a tree over the lanes."""
    q = a[:, :, 0] * b[:, :, 0]
    for p in range(1, a.shape[2]):
        q = _fma(a[:, :, p], b[:, :, p], q)
    return _tree(q[..., 0] + q[..., 1])[..., None, None]


def _sum(a):
    s = [a[:, :, p] for p in range(a.shape[2])]
    while len(s) > 1:
        n = len(s)
        s = [s[p] + s[n - 1 - p] if p < n // 2 else s[p] for p in range((n + 1) // 2)]
    return _tree(s[0][..., 0] + s[0][..., 1])[..., None, None]


def restated(x, w, gy, mode, eps=1e-5, elems=8):
    """(h, grad_x) of rows of S scalars in float32, lanes of ``elems`` elements as pairs.  mode:
    "right": sums about the means; "uncentred": mean(a h) from a with its mean; "difference": mean
    square and mean(a h) as differences of sums, whatever the mean."""
    n, S = x.shape
    lanes = 1
    while lanes * elems < S:
        lanes *= 2
    pad = [(0, 0), (0, lanes * elems - S)]
    cut = lambda v: np.pad(v, pad).reshape(n, lanes, elems // 2, 2)
    X, T, inside = cut(x.astype(f32)), cut(w.astype(f32) * gy.astype(f32)), cut(np.ones((n, S), f32))
    inv = f32(1) / f32(S)
    sx, st = _sum(X), _sum(T)
    mu, ma = sx * inv, st * inv
    u = X - mu * inside
    if mode == "difference":
        q, uc = _dot(X, X) - sx * mu, _dot(X, T) - st * mu
    else:
        q = _dot(u, u)
        uc = _dot(u, T - ma * inside if mode == "right" else T)
    r = f32(1) / np.sqrt(np.maximum(q * inv, 0) + f32(eps))
    h = u * r
    gx = _fma(h, -(r * r * uc * inv), _fma(T, r, -(r * ma)))
    back = lambda v: v.reshape(n, -1)[:, :S].astype(np.float64)
    return back(h), back(gx)


# ---- rows whose means are large ----

SHAPES = [("96x0e", 90), ("1024x0e", 400), ("2048x0e", 240), ("4096x0e", 120), ("3999x0e", 120), ("9001x0e", 12),
          ("64x0e+8x1o+40x0e", 60)]
MEANS = [(1000.0, 1000.0), (100.0, 300.0), (0.5, 1000.0), (1000.0, 0.0), (0.5, 0.0), (1.9, 30.0)]


def offsets(R, n, seed=2):
    """Means of x and of grad_y by row (rows of every kind side by side, in no regular order), at the 0e
    blocks' elements."""
    kind = np.random.default_rng(seed).integers(len(MEANS), size=n)
    mx, mg = np.zeros((n, R.dim)), np.zeros((n, R.dim))
    for b in R.blocks:
        if R.centred(b):
            s = slice(b.offset, b.offset + b.size)
            mx[:, s], mg[:, s] = (np.array(MEANS)[kind, i][:, None] for i in (0, 1))
    return kind, mx, mg


def scalar_problem(S, n, seed=4):
    """Rows of S scalars with such means, stored in float32: rows, kinds, x, weight, grad_y."""
    R = node.Rows(f"{S}x0e")
    g = np.random.default_rng(seed)
    kind, mx, mg = offsets(R, n)
    x, gy = ((g.normal(size=(n, S)) + m).astype(f32).astype(np.float64) for m in (mx, mg))
    return R, kind, x, (1 + 0.2 * g.normal(size=S)).astype(f32).astype(np.float64), gy

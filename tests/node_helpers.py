"""Node-feature problems and error scales for the GPU tests.

Tolerances.  Every output is compared element by element with |got - ref| <= tol * scale, where
``scale`` is the formula evaluated with absolute values (so cancellation is accounted for) and

    tol = (24 + 2 depth) 2^-24        float32 arithmetic

24: at most a dozen roundings of an element's own expression, each 2^-24 of one of the terms in
``scale``, and as many through r (a square root, a quotient, eps and the mean's division); depth:
additions one after another in a block's sums, at most S / 32 + 16 for the sums used here (32
lanes or more, then trees), twice for the mean and the mean square.  Storing in 16 bits adds half
a step of the value, eps / 2 = 2^-8 (bf16) or 2^-11 (fp16), plus the smallest subnormal.
Sums over rows of n terms add n 2^-24 of the sum of absolute values (any order of additions).
"""

import numpy as np

from oracle import node

U = 2.0 ** -24
TYPES = ("float32", "bfloat16", "float16")


def half_step(dtype):
    return {"float32": 0.0, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}[dtype]


def tol32(R):
    return (24 + 2 * (max(b.size for b in R.blocks) / 32 + 16)) * U


def stored(a, dtype):
    """A float32 array rounded to the storage type: (CUDA tensor, float64 values)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def assert_near(got, ref, scale, tol, dtype="float32", what=""):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, what
    bound = tol * scale + half_step(dtype) * np.abs(ref) * (1 + tol) + (2.0 ** -24 if dtype == "float16" else 1e-37)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) / np.maximum(bound, 1e-300))))


class Problem:
    def __init__(self, irreps, n, dtype="float32", layout="ir_mul", seed=0, offset=0.5, eps=1e-5):
        import torch
        from equivariant_gnn_tensor_dst_b200 import binding
        self.R = node.Rows(irreps, layout, eps)
        self.dtype, self.n = dtype, n
        self.plan = binding.NodePlan(irreps, getattr(torch, dtype), eps, layout)
        assert (self.plan.dim, self.plan.channels, self.plan.biases) == (self.R.dim, self.R.channels, self.R.biases)
        g = self.rng = np.random.default_rng(seed)
        x = g.normal(size=(n, self.R.dim)) * np.exp(0.5 * g.normal(size=(n, 1)))
        for b in self.R.blocks:
            if self.R.centred(b):
                x[:, b.offset:b.offset + b.size] += offset
        self.x, self.x64 = stored(x, dtype)
        self.w, self.w64 = stored(1 + 0.2 * g.normal(size=self.R.channels), "float32")
        self.b, self.b64 = stored(0.2 * g.normal(size=self.R.biases), "float32")

    def rows(self):
        return stored(self.rng.normal(size=(self.n, self.R.dim)), self.dtype)

    def vector(self, n):
        return stored(self.rng.normal(size=n), "float32")

    # -- scales: the formulas with absolute values --

    def _abs_parts(self, *arrays):
        return [self.R.parts(np.abs(a)) for a in arrays]

    def _stats(self, x):
        """Per block: h-like magnitude (|x| + mean|x|) r, and r."""
        out = []
        for b, v in zip(self.R.blocks, self.R.parts(x)):
            _, r, _ = node._block(self.R, b, v)
            a = np.abs(v) + (node._mean(np.abs(v)) if self.R.centred(b) else 0.0)
            out.append((a * r, r))
        return out

    def _plus_mean(self, b, v):
        return v + node._mean(v) if self.R.centred(b) else v

    def forward_scale(self, x):
        out = []
        for b, (h, r), w, c in zip(self.R.blocks, self._stats(x), self.R.split(np.abs(self.w64)),
                                   self.R.split(np.abs(self.b64), True)):
            # an error in r is relative: |h| (1 + mean of the magnitudes squared, times r^2)
            out.append(w * h * (1 + node._mean(h * h)) + (0.0 if c is None else c))
        return self.R.rows(out)

    def backward_scale(self, x, gy):
        gx, gw = [], []
        for b, (h, r), g, w in zip(self.R.blocks, self._stats(x), self._abs_parts(gy)[0],
                                   self.R.split(np.abs(self.w64))):
            a = self._plus_mean(b, w * g)
            k = 1 + node._mean(h * h)
            gx.append(r * k * (a + h * node._mean(a * h) * k))
            gw.append((g * h * k).sum(axis=(0, 1)))
        return self.R.rows(gx), np.concatenate(gw)

    def double_scale(self, x, gy, p, s, t):
        gx, gw, gg = [], [], []
        for b, (h, r), g, pp, w, q, c in zip(self.R.blocks, self._stats(x), *self._abs_parts(gy, p),
                                             self.R.split(np.abs(self.w64)), self.R.split(np.abs(s)),
                                             self.R.split(np.abs(t), True)):
            a, e, pp = (self._plus_mean(b, v) for v in (w * g, q * g, pp))
            k = 1 + node._mean(h * h)
            P, Q, S = k * node._mean(h * pp), k * node._mean(h * a), node._mean(pp * a)
            proj = r * k * (pp + h * P)
            gg.append(w * proj + q * h * k + (0.0 if c is None else c))
            gw.append((g * proj).sum(axis=(0, 1)))
            gx.append(r * r * k * k * (h * (3 * P * Q + S) + Q * pp + P * a) + r * k * (e + h * k * node._mean(h * e)))
        return self.R.rows(gx), np.concatenate(gw), self.R.rows(gg)

    def sum_tol(self):
        """Relative to the sum of absolute values of a channel's n_rows * (2l+1) terms."""
        return tol32(self.R) + self.n * max(b.dim for b in self.R.blocks) * U

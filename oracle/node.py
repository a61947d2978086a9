"""Node-feature operators in float64: irreps layer norm with its backward and double backward,
and dropout with a counter-based mask.

Layer norm of the S = (2l+1) C elements v of one block of a row (Ba, Kiros, Hinton, arXiv
1607.06450, read per irrep block): u = v - mean(v) for 0e blocks and u = v otherwise,
r = (mean(u^2) + eps)^(-1/2), y = weight_c r u + bias_c (bias for 0e blocks).  The gradients are
the textbook forms, written with the projection K = I - 1 1^T / S (0e) - h h^T / S, h = r u:
grad_x = r K (weight grad_y).  The double backward differentiates
Lambda = <p, grad_x> + <s, grad_weight> + <t, grad_bias>.

Dropout: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011) in Python integers per counter;
key = seed words, counter = (group, row, offset words), four channels of a block per counter.
"""

import numpy as np

from . import irreps as _irreps

MUL_0, MUL_1, WEYL_0, WEYL_1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox4x32(counter, key, rounds=10):
    """Four 32-bit words of one counter (four words) and key (two words)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = MUL_0 * c[0], MUL_1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + WEYL_0) & 0xFFFFFFFF, (k[1] + WEYL_1) & 0xFFFFFFFF]
    return c


class Rows:
    """Rows of an irreps string: blocks, channel, bias and dropout-group numbering."""

    def __init__(self, irreps, layout="ir_mul", eps=1e-5):
        self.blocks = _irreps.parse(irreps)
        self.layout, self.eps = layout, eps
        self.dim = sum(b.size for b in self.blocks)
        self.channels = sum(b.mul for b in self.blocks)
        self.biases = sum(b.mul for b in self.blocks if self.centred(b))

    @staticmethod
    def centred(b):
        return b.l == 0 and b.parity == 1

    def parts(self, a):
        """The blocks of [N, dim] as float64 [N, components, channels]."""
        a = np.asarray(a, np.float64)
        out = []
        for b in self.blocks:
            v = a[:, b.offset:b.offset + b.size]
            out.append(v.reshape(-1, b.dim, b.mul) if self.layout == "ir_mul"
                       else v.reshape(-1, b.mul, b.dim).transpose(0, 2, 1))
        return out

    def rows(self, parts):
        return np.concatenate([(v if self.layout == "ir_mul" else v.transpose(0, 2, 1)).reshape(v.shape[0], -1)
                               for v in parts], axis=1)

    def split(self, vec, biases=False):
        """A channel vector cut by block (None for blocks without a bias)."""
        out, at = [], 0
        for b in self.blocks:
            if biases and not self.centred(b):
                out.append(None)
                continue
            out.append(np.asarray(vec, np.float64)[at:at + b.mul])
            at += b.mul
        return out


def _mean(v):
    return v.mean(axis=(1, 2), keepdims=True)


def _block(R, b, v):
    """h, r and the mean-removing projection of one block."""
    centre = (lambda w: w - _mean(w)) if R.centred(b) else (lambda w: w)
    u = centre(v)
    r = 1.0 / np.sqrt(_mean(u * u) + R.eps)
    return u * r, r, centre


def norm_forward(R, x, weight, bias):
    out = []
    for b, v, w, c in zip(R.blocks, R.parts(x), R.split(weight), R.split(bias, True)):
        h, _, _ = _block(R, b, v)
        out.append(w * h + (0.0 if c is None else c))
    return R.rows(out)


def norm_backward(R, x, weight, grad_y):
    gx, gw, gb = [], [], [np.zeros(0)]
    for b, v, g, w in zip(R.blocks, R.parts(x), R.parts(grad_y), R.split(weight)):
        h, r, centre = _block(R, b, v)
        a = centre(w * g)
        gx.append(r * (a - h * _mean(a * h)))
        gw.append((g * h).sum(axis=(0, 1)))
        if R.centred(b):
            gb.append(g.sum(axis=(0, 1)))
    return R.rows(gx), np.concatenate(gw), np.concatenate(gb)


def norm_double_backward(R, x, weight, grad_y, gg_x, gg_weight, gg_bias):
    gx, gw, gg = [], [], []
    for b, v, g, p, w, s, t in zip(R.blocks, R.parts(x), R.parts(grad_y), R.parts(gg_x), R.split(weight),
                                   R.split(gg_weight), R.split(gg_bias, True)):
        h, r, centre = _block(R, b, v)
        p, a, e = centre(p), centre(w * g), centre(s * g)
        P, Q, S = _mean(h * p), _mean(h * a), _mean(p * a)
        k = r * (p - h * P)
        gg.append(w * k + s * h + (0.0 if t is None else t))
        gw.append((g * k).sum(axis=(0, 1)))
        gx.append(r * r * (h * (3 * P * Q - S) - Q * p - P * a) + r * (e - h * _mean(h * e)))
    return R.rows(gx), np.concatenate(gw), R.rows(gg)


def dropout_mask(R, n_rows, p, seed, offset=0):
    """1 / (1 - p) or 0 per element, [n_rows, dim]."""
    threshold = int(np.floor(p * 2.0 ** 32 + 0.5))
    scale = 1.0 / (1.0 - p) if p < 1.0 else 0.0
    key = (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)
    low, high = offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF
    out, group0 = [], 0
    for b in R.blocks:
        groups = -(-b.mul // 4)
        words = np.array([[philox4x32((group0 + g, n, low, high), key) for g in range(groups)]
                          for n in range(n_rows)], dtype=np.uint64).reshape(n_rows, 4 * groups)[:, :b.mul]
        m = np.where(words >= threshold, scale, 0.0)
        out.append(np.repeat(m[:, None, :], b.dim, axis=1))
        group0 += groups
    return R.rows(out)

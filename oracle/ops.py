"""The operators around the expert layer in 64 bits, on the CPU: products with
an epilogue over ragged groups, their gradients, activations, and dropout with
its counter-based generator. Formulas only; nothing is shared with the CUDA
path."""
from __future__ import annotations

import math

import numpy as np
import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act(u, name):
    u = u.double()
    if name == "relu":
        return u.clamp(min=0)
    if name == "gelu":
        return u * 0.5 * torch.special.erfc(-u / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    if name == "silu":
        return u * torch.sigmoid(u)
    return u


def act_slope(u, name):
    u = u.double()
    if name == "relu":
        return (u > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-u / math.sqrt(2)) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (u + 0.044715 * u ** 3))
        return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * 0.044715 * u * u)
    if name == "silu":
        s = torch.sigmoid(u)
        return s + u * s * (1 - s)
    return torch.ones_like(u)


def groups(offsets):
    return list(enumerate(zip(offsets[:-1], offsets[1:])))


def product(x, offsets, w, bias=None):
    """u [rows, n] and sum_i |x w| (the scale of its rounding errors); NaN outside every group."""
    u = torch.full((x.shape[0], w.shape[1]), math.nan, dtype=torch.float64)
    scale = u.clone()
    for e, (a, b) in groups(offsets):
        u[a:b] = x[a:b].double() @ w[e].double().T
        scale[a:b] = x[a:b].double().abs() @ w[e].double().abs().T
        if bias is not None:
            u[a:b] += bias[e].double()
            scale[a:b] += bias[e].double().abs()
    return u, scale


def input_gradient(dy, offsets, w):
    """dy W per group, and its error scale; NaN outside every group."""
    return product(dy, offsets, w.transpose(1, 2))


def weight_gradient(dy, offsets, x):
    """dw [E, n, k], db [E, n], and their error scales."""
    E = len(offsets) - 1
    dw = torch.zeros((E, dy.shape[1], x.shape[1]), dtype=torch.float64)
    db = torch.zeros((E, dy.shape[1]), dtype=torch.float64)
    sw, sb = torch.zeros_like(dw), torch.zeros_like(db)
    for e, (a, b) in groups(offsets):
        d, v = dy[a:b].double(), x[a:b].double()
        dw[e], db[e] = d.T @ v, d.sum(0)
        sw[e], sb[e] = d.abs().T @ v.abs(), d.abs().sum(0)
    return dw, db, sw, sb


def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., SC 2011). counter: four uint64 arrays of
    32-bit values, key: two ints; returns four uint64 arrays."""
    u = np.uint64
    low = u(0xFFFFFFFF)
    c = [np.asarray(v, dtype=u) for v in counter]
    k = [int(v) for v in key]
    for _ in range(rounds):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> u(32)) ^ c[1] ^ u(k[0]), q & low, (p >> u(32)) ^ c[3] ^ u(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_words(rows, cols, seed, at):
    """word(r, c) of the dropout mask as uint64 [rows, cols]; seed and at (the
    counter offset) are 64-bit integers. rows: a count, or the row indices."""
    r = np.arange(rows) if np.isscalar(rows) else np.asarray(rows)
    at &= (1 << 64) - 1
    seed &= (1 << 64) - 1
    quads = -(-cols // 4)
    shape = (len(r), quads)
    c0 = np.broadcast_to(np.arange(quads, dtype=np.uint64), shape)
    c1 = np.broadcast_to(r.astype(np.uint64)[:, None], shape)
    fill = [np.full(shape, v, dtype=np.uint64) for v in (at & 0xFFFFFFFF, at >> 32)]
    words = philox4x32([c0, c1, *fill], (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack(words, axis=2).reshape(len(r), quads * 4)[:, :cols]


def dropout(x, p, seed, at, rows=None):
    """dropout(x) in 64 bits; rows: the matrix rows that x's rows are (default 0..)."""
    if p == 0:
        return x.double()
    words = dropout_words(x.shape[0] if rows is None else rows, x.shape[1], seed, at)
    keep = torch.from_numpy(words >= np.uint64(math.floor(p * 2 ** 32)))
    return torch.where(keep, x.double() / (1 - p), torch.zeros((), dtype=torch.float64))

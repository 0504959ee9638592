"""Plain 64-bit statements of the expert operators: the norm, the experts' products, the gated
activation, the combination per token, 8-bit rows, and the gradients.

They restate the definitions of ``include/moeroute.h`` in numpy and share no code with the
kernels.  Where a second array is returned it is the sum of the terms' magnitudes, which a
floating-point sum's error is proportional to.
"""
from __future__ import annotations

import numpy as np


def blocks(n):
    return -(-n // 128)


def e4m3_values():
    """The value of each of the 256 codes."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = (-x if s else x) if (c & 127) != 127 else np.nan
    return v


def block_scales(y, least=1e-30):
    """Scales of 8-bit rows: the largest magnitude (NaN passed over) of each block of 128 columns / 448."""
    a = np.abs(y)
    a = np.where(np.isnan(a), 0.0, a)
    return np.stack([np.maximum(a[:, b * 128:(b + 1) * 128].max(1), least) / 448.0 for b in range(blocks(y.shape[1]))], 1)


def widen(scale, cols):
    """A block's scale at each of its columns."""
    return np.repeat(scale, 128, axis=-1)[..., :cols]


def rms_norm(s, g, eps):
    """y and rstd of rows s (the rounded sum)."""
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * g, rstd


def rms_norm_grad(s, g, rstd, dy, dsum=None):
    """(d_x, its magnitude, d_weight, its magnitude)."""
    n = s * rstd[:, None]
    gd = dy * g
    dx = rstd[:, None] * (gd - n * (gd * n).mean(1, keepdims=True))
    mag = rstd[:, None] * (np.abs(gd) + np.abs(n) * np.abs(gd * n).mean(1, keepdims=True))
    if dsum is not None:
        dx, mag = dx + dsum, mag + np.abs(dsum)
    return dx, mag, (dy * n).sum(0), np.abs(dy * n).sum(0)


def silu_gate(h):
    """y of h = [a | b]."""
    a, b = np.split(h, 2, axis=1)
    return a * sigmoid(a) * b


def sigmoid(a):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-a))


def silu_gate_grad(h, dy):
    a, b = np.split(h, 2, axis=1)
    s = sigmoid(a)
    return np.concatenate([dy * b * s * (1 + a * (1 - s)), dy * a * s], 1)


def source(off, order, k, tokens, rows):
    """For each row of the lists: its expert (-1: behind the last segment) and its row of x (-1: padding)."""
    e = np.full(rows, -1)
    for i in range(len(off) - 1):
        e[off[i]:off[i + 1]] = i
    src = np.arange(rows) if order is None else np.where(order < 0, -1, order // k)
    return e, np.where((src >= tokens) | (e < 0), -1, src)


def gemm_rows(x, w, off, order=None, k=1, out=None):
    """Forward products (w [E][N][K], x [.][K]); rows behind the last segment come from `out`.
    With w transposed to [E][K][N] it is the gradient by the rows."""
    rows = len(order) if order is not None else len(x)
    e, src = source(off, order, k, len(x), rows)
    y = np.zeros((rows, w.shape[1])) if out is None else np.array(out, dtype=np.float64)
    mag = np.zeros((rows, w.shape[1]))
    for p in range(rows):
        if e[p] < 0:
            continue
        y[p] = 0.0 if src[p] < 0 else w[e[p]] @ x[src[p]]
        mag[p] = 0.0 if src[p] < 0 else np.abs(w[e[p]]) @ np.abs(x[src[p]])
    return y, mag


def gemm_weight_grad(dy, x, off, order=None, k=1):
    E = len(off) - 1
    e, src = source(off, order, k, len(x), len(dy))
    out = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(out)
    for i in range(E):
        at = np.nonzero((e == i) & (src >= 0))[0]
        out[i] = dy[at].T @ x[src[at]]
        mag[i] = np.abs(dy[at]).T @ np.abs(x[src[at]])
    return out, mag


def combine(z, inv, w=None, add=None):
    T, k = inv.shape
    w = np.ones((T, k)) if w is None else w
    y = np.zeros((T, z.shape[1])) if add is None else add.astype(np.float64)
    mag = np.abs(y)
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                y[t] = y[t] + w[t, j] * z[inv[t, j]]
                mag[t] = mag[t] + np.abs(w[t, j] * z[inv[t, j]])
    return y, mag


def combine_grad(z, inv, w, dout, rows):
    """(d_z, d_weights, its magnitude)."""
    T, k = inv.shape
    w = np.ones((T, k)) if w is None else w
    dz = np.zeros((rows, dout.shape[1]))
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = inv[t, j]
            if r >= 0:
                dz[r] = w[t, j] * dout[t]
                dw[t, j] = dout[t] @ z[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(z[r])
    return dz, dw, mag

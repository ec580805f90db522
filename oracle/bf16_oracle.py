"""FP64 oracle of the bf16 GroupedLinear's gradients and of the adapter linear
(test infrastructure; NumPy, shares no code with the HIP path).

GroupedLinear: y[i] = r[i] W_e x[i] for the rows i of expert e.  Its gradients for dy:
  dX[i] = r[i] W_e^T dy[i],  dr[i] = x[i] . (W_e^T dy[i]),
  dW_e  = sum over the rows i of e of r[i] dy[i] x[i]^T.
Adapter linear: y[m] = W x[m] + s_l B_l (A_l x[m]) with l = ids[m], the second term
only where l is in [0, L).

Each function also returns the sums of magnitudes that error bounds are made of."""
from __future__ import annotations

import numpy as np


def linear_fwd(x, w, off, r=None):
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w[e].T
    return y if r is None else y * r[:, None]


def linear_bwd(dy, x, w, off, r=None):
    """(dX, dW, dr or None)."""
    M, K = x.shape
    g = np.zeros((M, K))
    dw = np.zeros(w.shape)
    for e in range(w.shape[0]):
        rows = slice(off[e], off[e + 1])
        g[rows] = dy[rows] @ w[e]
        scaled = dy[rows] if r is None else dy[rows] * r[rows, None]
        dw[e] = scaled.T @ x[rows]
    if r is None:
        return g, dw, None
    return g * r[:, None], dw, (g * x).sum(1)


def lora_fwd(x, w, a, b, ids, scale=None):
    y = x @ w.T
    for m, l in enumerate(ids):
        if 0 <= l < a.shape[0]:
            s = 1.0 if scale is None else scale[l]
            y[m] += s * (b[l] @ (a[l] @ x[m]))
    return y


def lora_bound(x, w, a, b, ids, scale=None):
    """Bound on |y - exact| of a bf16 result: fp32 sums of exact products (a sum of n
    of them, in any order and with truncation, is off by at most n 2^-23 of their
    magnitudes), s A x held to 2^-16, one rounding to bf16 (2^-8)."""
    K, r = x.shape[1], a.shape[1]
    n23 = 2.0 ** -23
    S = np.abs(x) @ np.abs(w).T
    err = (K + 2) * n23 * S
    for m, l in enumerate(ids):
        if 0 <= l < a.shape[0]:
            s = 1.0 if scale is None else abs(scale[l])
            h = s * (np.abs(a[l]) @ np.abs(x[m]))           # magnitudes; |h| is below
            low = np.abs(b[l]) @ h
            err[m] += ((K + 4) * n23 + 2.0 ** -16) * low
            S[m] += low
    err += (2 * r + 4) * n23 * S
    return 2.0 ** -8 * np.abs(lora_fwd(x, w, a, b, ids, scale)) + (1 + 2.0 ** -8) * err

"""FP64 oracle of the MXFP4 operators.  TEST INFRASTRUCTURE ONLY (like
``oracle/mx_oracle.py``, whose block and scale helpers it uses).

The format (OCP Microscaling formats 1.0, MXFP4): E2M1 elements (1 sign, 2
exponent bits with bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), one
E8M0 scale per 32 values, scale exponent floor(log2 amax) - 2 (2 = exponent of
6) and not below -127, round to nearest even, saturating at 6, the sign kept.

Readings where the format leaves room:

* R4-pack    two codes a byte, the even element in the low half.
* R4-nan     a block that holds an infinity or a NaN gets scale 255 and codes 0.
* R4-layer   the few-token MoE layer quantizes x and z to MXFP8 blocks along
             their contraction axes when the weights are MXFP8 or MXFP4, and
             rounds z to bfloat16 when they are bfloat16; the routing weight
             multiplies z before that; a logit of -inf (or NaN) is never
             routed, a token without routed experts gives a row of zeros.
"""
from __future__ import annotations

import numpy as np

from oracle import mx_oracle as O

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(v):
    """E2M1 codes of float64 values: nearest, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    mid = (E2M1[1:] + E2M1[:-1]) / 2              # exact
    code = np.searchsorted(mid, a, side="left")   # a == mid stays below it
    tie = (code < 7) & (a == mid[np.minimum(code, 6)])
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    return (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def e2m1_decode(c):
    c = np.asarray(c)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def pack(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    b = np.asarray(b)
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def quantize4_lastdim(v):
    """(packed codes [..., C/2], scales [..., C/32]) of v [..., C]."""
    v = np.asarray(v, dtype=np.float64)
    C = v.shape[-1]
    if C % O.BLOCK:
        raise ValueError("last dimension must be a multiple of 32")
    blk = v.reshape(v.shape[:-1] + (C // O.BLOCK, O.BLOCK))
    bad = ~np.isfinite(blk).all(axis=-1)
    blk = np.where(bad[..., None], 0.0, blk)
    amax = np.abs(blk).max(axis=-1)
    X = np.full(amax.shape, -127, dtype=np.int64)
    nz = amax > 0
    X[nz] = np.maximum(O.floor_log2(amax[nz]) - 2, -127)
    codes = e2m1_encode(blk * np.ldexp(1.0, -X)[..., None])
    scales = np.where(bad, 255, X + 127).astype(np.uint8)
    return pack(codes.reshape(v.shape)), scales


def dequantize4_lastdim(codes, scales):
    v = e2m1_decode(unpack(codes))
    blk = v.reshape(v.shape[:-1] + (v.shape[-1] // O.BLOCK, O.BLOCK))
    return (blk * O.e8m0_decode(scales)[..., None]).reshape(v.shape)


def qdq4_lastdim(v):
    return dequantize4_lastdim(*quantize4_lastdim(v))


def route(logits, k):
    """(ids [T, k], weights [T, k]): the k largest logits, lower index among
    equal ones, and their softmax.  NaN counts as -inf; a slot with logit -inf
    has weight 0, and so has every slot of a token with no other logit."""
    lg = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(lg, ids, 1)
    m = v[:, :1]
    with np.errstate(invalid="ignore"):
        p = np.where(np.isneginf(v), 0.0, np.exp(v - m))
    s = p.sum(1, keepdims=True)
    return ids, np.divide(p, s, out=np.zeros_like(p), where=s > 0)


def moe_layer(x, logits, w1, w2, k, mx):
    """out [T, H] of x [T, H] (float64 of bf16 values), logits [T, E] and the
    values w1 [E, 2F, H], w2 [E, H, F] the weights stand for.  mx: MX weights
    (x and z are quantized to MXFP8), else bfloat16 ones (z rounded)."""
    ids, r = route(logits, k)
    F = w2.shape[2]
    xq = O.qdq_lastdim(x) if mx else x
    out = np.zeros((x.shape[0], w2.shape[1]))
    for t in range(x.shape[0]):
        for j in range(k):
            if r[t, j] > 0:
                e = ids[t, j]
                h = w1[e] @ xq[t]
                a, b = h[:F], h[F:]
                z = r[t, j] * a / (1.0 + np.exp(-a)) * b
                z = O.qdq_lastdim(z) if mx else O.round_bf16(z)
                out[t] += w2[e] @ z
    return out

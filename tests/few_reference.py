"""The layer for a few tokens in plain fp64 numpy, with the error bounds that
the tests compare under.

Bounds, by running the sums over absolute values (u = 2^-24, fp32's half
step; a sum of n terms in any order is within n u of the sum of the terms'
absolute values, products and the final additions included in n + 2):
  logits   (d + 2) u (|x| |Wg| + |b|), the noise's share scaled by |noise|
           (Softplus has slope <= 1 and is given 8 u of its own value)
  gates    relative: twice the largest logit error, and (k + 16) u
  hidden   (d + 2) u (|x| |W1| + |b1|), plus half a step of the layer's type
  output   the hidden error through |W2|, (F + 2) u (|h| |W2| + |b2|), the
           gate's error, (k + 2) u of the terms, and half a step of the type
"""
from __future__ import annotations

import math

import numpy as np

from sparsely_gated_mixture_gb300 import workloads as wl

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def f64(a, dtype):
    if a is None:
        return None
    return (wl.bf16_bits_to_f32(a) if dtype == "bf16" else a).astype(np.float64)


def softplus(z):
    return np.logaddexp(0.0, z)


def logits(inp, dtype):
    """H [T, E] and its error bound."""
    x = f64(inp["x"], dtype)
    d = x.shape[1]
    b = 0.0 if inp["bias"] is None else inp["bias"].astype(np.float64)
    Wg = inp["Wg"].astype(np.float64)
    H = x @ Wg + b
    err = (d + 2) * U * (np.abs(x) @ np.abs(Wg) + np.abs(b))
    if inp["Wn"] is not None:
        Wn, n = inp["Wn"].astype(np.float64), inp["noise"].astype(np.float64)
        s = softplus(x @ Wn)
        H = H + n * s
        err = err + np.abs(n) * ((d + 2) * U * (np.abs(x) @ np.abs(Wn)) + 8 * U * s)
        err = err + 2 * U * (np.abs(H) + np.abs(n) * s)
    return H, err


def topk(H, k):
    return np.argsort(-H, axis=1, kind="stable")[:, :k].astype(np.int32)


def softmax(v):
    e = np.exp(v - v.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


def gates(H, idx, mode):
    p = softmax(H) if mode == wl.SWITCH else None
    rows = np.arange(H.shape[0])[:, None]
    return p[rows, idx] if p is not None else softmax(H[rows, idx])


def slots(idx, E, C):
    """Token-order positions (exclusive counts) and keep = pos < C."""
    pos = np.zeros(idx.shape, np.int32)
    seen = np.zeros(E + 1, np.int64)
    for t in range(idx.shape[0]):
        for j in range(idx.shape[1]):
            pos[t, j] = seen[idx[t, j]]
            seen[idx[t, j]] += 1
    return pos, (pos < C).astype(np.uint8)


def output(inp, dtype, idx, gate, keep, gate_rel):
    """y [T, d] for the choices idx with weight gate where keep, its error
    bound, and the sum of the expert terms' absolute values."""
    x = f64(inp["x"], dtype)
    T, d = x.shape
    k = idx.shape[1]
    y = x.copy()
    err = np.zeros_like(x)
    mag = np.abs(x)
    weights = {}
    for t in range(T):
        for j in range(k):
            if not keep[t, j]:
                continue
            e = int(idx[t, j])
            if e not in weights:
                weights[e] = tuple(f64(inp[n][e], dtype) if inp[n] is not None else 0.0
                                   for n in ("W1", "b1", "W2", "b2"))
            W1, b1, W2, b2 = weights[e]
            F = W1.shape[1]
            pre = x[t] @ W1 + b1
            pre_err = (d + 2) * U * (np.abs(x[t]) @ np.abs(W1) + np.abs(b1))
            h = np.maximum(pre, 0.0)
            h_err = pre_err + HALF[dtype] * (h + pre_err)
            z = h @ W2 + b2
            z_err = h_err @ np.abs(W2) + (F + 2) * U * ((h + h_err) @ np.abs(W2) + np.abs(b2))
            g = gate[t, j]
            y[t] += g * z
            err[t] += g * (z_err + gate_rel * np.abs(z))
            mag[t] += g * np.abs(z)
    err += (k + 2) * U * mag
    return y, err + HALF[dtype] * (np.abs(y) + err), mag - np.abs(x)


def capacity(T, E, k, cf):
    return max(1, min(T, math.floor(k * T * cf / E)))

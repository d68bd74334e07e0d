"""The 8-bit format and the backward from it in plain fp64 numpy, with bounds
on what a kernel in the layer's types may be off by."""
from __future__ import annotations

import math

import numpy as np

import few_reference as few
from sparsely_gated_mixture_gb300 import workloads as wl

U = few.U
BLOCK, LOW = 32, -124
VALUES = np.array([m * 2.0 ** -9 for m in range(8)] +
                  [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)])[:127]


def quantise(h):
    """Rows [R, F] -> (bytes, scale bytes, values), by the format's words."""
    h = np.asarray(h, np.float64)
    R, F = h.shape
    q = np.zeros((R, F), np.uint8)
    nb = -(-F // BLOCK)
    s = np.zeros((R, nb), np.uint8)
    v = np.zeros((R, F))
    mid = (VALUES[1:] + VALUES[:-1]) / 2
    for r in range(R):
        for b in range(nb):
            c = slice(b * BLOCK, min(F, (b + 1) * BLOCK))
            x = h[r, c]
            if np.any(np.isnan(x) | (x == np.inf)):
                s[r, b], v[r, c] = 255, np.nan
                continue
            top = max(0.0, x.max())
            e = LOW
            while 448.0 * 2.0 ** e < top:
                e += 1
            z = np.maximum(x, 0.0) / 2.0 ** e
            i = np.searchsorted(mid, z)  # nearest, the lower one on ties
            tie = (i < 126) & (z == mid[np.minimum(i, 125)])
            i = np.where(tie & (i % 2 == 1), i + 1, i)
            i = np.where((x > 0) & (i == 0), 1, i)
            i = np.minimum(i, 119 if e >= 120 else 126)  # 240, 448
            q[r, c], s[r, b], v[r, c] = i, e + 127, VALUES[i] * 2.0 ** e
    return q, s, v


def _cv2_grad(v):
    m, n = v.mean(), v.size
    var = ((v - m) ** 2).mean()
    return 2 * (v - m) / (n * m * m) - 2 * var / (n * m ** 3)


def _phi(u):
    return np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)


def gate_state(inp, dtype):
    x = few.f64(inp["x"], dtype)
    b = 0.0 if inp["bias"] is None else inp["bias"].astype(np.float64)
    c = x @ inp["Wg"].astype(np.float64) + b
    if inp["Wn"] is None:
        return x, c, None, c
    s = few.softplus(x @ inp["Wn"].astype(np.float64))
    return x, c, s, c + inp["noise"].astype(np.float64) * s


def loss(inp, dtype, mode, idx, keep, h, dy, weights, order):
    """L with the discrete choices idx, keep, the thresholds' owners and the
    hidden values' ReLU pattern held fixed and h [T, k, F] as constants (the
    router's side of L; the experts' own gradients have closed forms)."""
    x, c, s, H = gate_state(inp, dtype)
    T, E = H.shape
    k = idx.shape[1]
    G = few.gates(H, idx, mode)
    out = 0.0
    for t in range(T):
        for j in range(k):
            if keep[t, j]:
                e = idx[t, j]
                u = h[t, j] @ few.f64(inp["W2"][e], dtype)
                if inp["b2"] is not None:
                    u = u + few.f64(inp["b2"][e], dtype)
                out += G[t, j] * (u @ dy[t])
    w_imp, w_load, w_aux = weights
    imp = np.zeros(E)
    np.add.at(imp, idx, G)
    out += w_imp * imp.var() / imp.mean() ** 2
    f = np.bincount(idx[:, 0], minlength=E) / T
    out += w_aux * 0.01 * E * (f * few.softmax(H).mean(axis=0)).sum()
    if s is not None and k < E:
        hot = np.zeros((T, E), bool)
        np.put_along_axis(hot, idx.astype(np.int64), True, 1)
        r = np.arange(T)
        thr = np.where(hot, H[r, order[:, k]][:, None], H[r, order[:, k - 1]][:, None])
        load = (0.5 * np.vectorize(math.erfc)(-(c - thr) / s / math.sqrt(2))).sum(axis=0)
        out += w_load * load.var() / load.mean() ** 2
    return out


def backward(inp, dtype, mode, idx, gate, keep, h, dy, weights):
    """Gradients and bounds. h [T, k, F]: the hidden values; gate [T, k]: the
    gates that the experts' rows carry (fp32, as given to the kernel)."""
    x, c, s, H = gate_state(inp, dtype)
    T, E = H.shape
    k, d = idx.shape[1], x.shape[1]
    F = h.shape[2]
    half = few.HALF[dtype]
    row = half if dtype == "bf16" else 2 * U  # what rounding a row operand costs
    rows, cols = np.arange(T)[:, None], np.arange(T)
    g = dict(dW1=np.zeros((E, d, F)), db1=np.zeros((E, F)), dW2=np.zeros((E, F, d)),
             db2=np.zeros((E, d)), dx=dy.copy(), dgate=np.zeros((T, k)))
    err = {n: np.zeros_like(v) for n, v in g.items()}
    mag_dx = np.abs(dy)
    for t in range(T):
        for j in range(k):
            if not keep[t, j]:
                continue
            e = int(idx[t, j])
            W1, W2 = few.f64(inp["W1"][e], dtype), few.f64(inp["W2"][e], dtype)
            hv, w = h[t, j], float(gate[t, j])
            D = W2 @ dy[t]
            D_err = (d + 2) * U * (np.abs(W2) @ np.abs(dy[t]))
            on = hv > 0
            dp = w * D * on
            dp_err = np.abs(w) * D_err * on + row * (np.abs(dp) + np.abs(w) * D_err * on)
            du = w * dy[t]
            du_err = row * np.abs(du)
            b2 = np.zeros(d) if inp["b2"] is None else few.f64(inp["b2"][e], dtype)
            g["dgate"][t, j] = D @ hv + dy[t] @ b2
            err["dgate"][t, j] = (D_err @ hv + (F + d + 4) * U * (np.abs(D) @ hv + np.abs(dy[t]) @ np.abs(b2)))
            for n, a, b, b_err in (("dW1", x[t], dp, dp_err), ("dW2", hv, du, du_err)):
                g[n][e] += np.outer(a, b)
                err[n][e] += np.outer(np.abs(a), b_err + (T + 2) * U * np.abs(b))
            for n, b, b_err in (("db1", dp, dp_err), ("db2", du, 2 * U * np.abs(du))):
                g[n][e] += b
                err[n][e] += b_err + (T + 2) * U * np.abs(b)
            g["dx"][t] += W1 @ dp
            z = np.abs(W1) @ np.abs(dp)
            err["dx"][t] += np.abs(W1) @ dp_err + (F + 2) * U * z
            mag_dx[t] += z
    # The gate. Each factor of a softmax or load term carries the logits'
    # error (at most H_err.max() in an exponent) and a few roundings.
    w_imp, w_load, w_aux = weights
    _, H_err = few.logits(inp, dtype)
    rel = 4 * H_err.max() + (E + 32) * U
    G = gate.astype(np.float64)
    imp = np.zeros(E)
    np.add.at(imp, idx, G)
    coef = w_imp * _cv2_grad(imp)
    g["dgate"] = g["dgate"] + coef[idx]
    # CV^2's gradient: differences of sums over T, each within (T + E) u + rel.
    err["dgate"] += (rel + (T + E + 8) * U) * w_imp * 4 * imp.max() / (E * imp.mean() ** 2)
    p = few.softmax(H)
    first = np.bincount(idx[:, 0], minlength=E) / T
    dp = np.broadcast_to(w_aux * 0.01 * E / T * first, (T, E)).copy()
    dp_err = rel * np.abs(dp)
    dH, dH_err = np.zeros((T, E)), np.zeros((T, E))
    if mode == wl.SWITCH:
        dp[rows, idx] += g["dgate"]
        dp_err[rows, idx] += err["dgate"]
    else:
        m = (G * g["dgate"]).sum(axis=1, keepdims=True)
        m_err = (G * (err["dgate"] + rel * np.abs(g["dgate"]))).sum(axis=1, keepdims=True)
        dH[rows, idx] = G * (g["dgate"] - m)
        dH_err[rows, idx] = G * (err["dgate"] + m_err + rel * (np.abs(g["dgate"]) + np.abs(m)))
    m = (p * dp).sum(axis=1, keepdims=True)
    m_err = (p * (dp_err + rel * np.abs(dp))).sum(axis=1, keepdims=True)
    dH += p * (dp - m)
    dH_err += p * (dp_err + m_err + rel * (np.abs(dp) + np.abs(m)))
    dc, dc_err = np.zeros((T, E)), np.zeros((T, E))
    order = np.argsort(-H, axis=1, kind="stable")
    dz = dz_err = None
    if s is not None:
        ds, ds_err = np.zeros((T, E)), np.zeros((T, E))
        if k < E and w_load:
            hot = np.zeros((T, E), bool)
            np.put_along_axis(hot, idx.astype(np.int64), True, 1)
            thr = np.where(hot, H[cols, order[:, k]][:, None], H[cols, order[:, k - 1]][:, None])
            u = (c - thr) / s
            load = (0.5 * np.vectorize(math.erfc)(-u / math.sqrt(2))).sum(axis=0)
            cl = w_load * _cv2_grad(load)
            gl = cl * _phi(u) / s
            du = 4 * H_err.max() / s * (1 + np.abs(u))  # what u may be off by
            cl_err = 1e-5 * w_load * 4 * load.max() / (E * load.mean() ** 2)
            gl_err = (np.abs(gl) * ((np.abs(u) + 1) * du + 32 * U)
                      + (cl_err + np.abs(cl) * 1e-5) * _phi(u) / s)
            dc, dc_err = gl.copy(), gl_err.copy()
            ds, ds_err = -gl * u, gl_err * np.abs(u) + np.abs(gl) * du
            dH[cols, order[:, k]] -= np.where(hot, gl, 0).sum(axis=1)
            dH_err[cols, order[:, k]] += np.where(hot, gl_err, 0).sum(axis=1)
            dH[cols, idx[:, k - 1]] -= np.where(hot, 0, gl).sum(axis=1)
            dH_err[cols, idx[:, k - 1]] += np.where(hot, 0, gl_err + E * U * np.abs(gl)).sum(axis=1)
        n = inp["noise"].astype(np.float64)
        ds, ds_err = ds + n * dH, ds_err + np.abs(n) * dH_err
        sig = -np.expm1(-s)
        dz = ds * sig
        dz_err = ds_err * sig + np.abs(ds) * (rel + 16 * U)
    dc, dc_err = dc + dH, dc_err + dH_err
    ax = np.abs(x)
    for n, v, e in (("dWg", dc, dc_err), ("dWn", dz, dz_err)):
        if v is None:
            g[n] = None
            continue
        g[n] = x.T @ v
        err[n] = ax.T @ (e + (T + 2) * U * np.abs(v))
        W = inp["Wg" if n == "dWg" else "Wn"].astype(np.float64)
        g["dx"] += v @ W.T
        z = np.abs(v) @ np.abs(W).T
        err["dx"] += e @ np.abs(W).T + (2 * E + 2) * U * z
        mag_dx += z
    g["dbias"] = dc.sum(axis=0)
    err["dbias"] = (dc_err + (T + 2) * U * np.abs(dc)).sum(axis=0)
    err["dx"] += (k + 4) * U * mag_dx
    for n in ("dx", "dW1", "dW2", "db1", "db2"):
        err[n] += half * (np.abs(g[n]) + err[n])
    return g, err, order

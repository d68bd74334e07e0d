"""The gated experts in 64 bits on the CPU (torch.float64), from the formulas,
with a bound of the kernels' rounding errors beside every result.

The bounds add up, element by element:
* half a step for every value rounded to fewer bits (bf16 2^-8 relative, fp32
  2^-24, an e4m3 value: the two neighbours it may go to);
* K * 2^-23 of the sum of magnitudes for an fp32 sum of K products (each partial
  sum is off by at most 2^-23 of it; tensor cores cut instead of rounding);
* the fast exponential's (8 + 2 |v|) * 2^-23 in an activation.
"""
import math

import torch

F64 = torch.float64
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -23
SILU, GELU, RELU = 0, 1, 2
BLOCK = 128


def capacity(T, E, k, cf, min_cap=1):
    return max(min_cap, min(T, math.floor(k * T * cf / E)))


def slots(idx, E, C):
    """pos, keep [T,k], and for each expert its kept (token, choice) pairs."""
    T, k = idx.shape
    pos = torch.full((T, k), -1, dtype=torch.int32)
    keep = torch.zeros((T, k), dtype=torch.uint8)
    rows = [[] for _ in range(E)]
    count = [0] * E
    for t, es in enumerate(idx.tolist()):
        for j, e in enumerate(es):
            if not 0 <= e < E:
                continue
            pos[t, j] = count[e]
            if count[e] < C:
                keep[t, j] = 1
                rows[e].append((t, j))
            count[e] += 1
    return pos, keep, rows


def act(kind, v):
    if kind == SILU:
        return v * torch.sigmoid(v)
    if kind == GELU:
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    return torch.clamp(v, min=0)


def slope(kind, v):
    if kind == SILU:
        t = torch.sigmoid(v)
        return t * (1 + v * (1 - t))
    if kind == GELU:
        return 0.5 * torch.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v * v / 2) / math.sqrt(
            2 * math.pi)
    return (v > 0).to(F64)


def act_error(v):
    return (8 + 2 * v.abs()) * U32


def product(v, ev, W, b):
    """v @ W + b and its bound, v off by at most ev."""
    r, m = v @ W, v.abs() @ W.abs()
    e = v.shape[-1] * U32 * m + ev @ W.abs()
    if b is not None:
        r = r + b
        e = e + 2 * U32 * (m + b.abs())
    return r, e


def of(w, e):
    return None if w is None else w[e].cpu().to(F64)


def forward(kind, x, idx, gate, W1, b1, W3, b3, W2, b2, C, weights8=None):
    """weights8: None, or (s1, s3, s2) with W1, W3, W2 in 8 bits."""
    E = W1.shape[0]
    T, k = idx.shape
    dt = x.dtype
    u = STEP[dt]
    xd = x.cpu().to(F64)
    F = W1.shape[2] if weights8 is None else W1.shape[1]
    pos, keep, rows = slots(idx.cpu(), E, C)
    y, bound = xd.clone(), torch.zeros_like(xd)
    size = xd.abs()
    pre = [torch.zeros((T * k, F), dtype=F64) for _ in range(2)]
    pre_e = [torch.zeros((T * k, F), dtype=F64) for _ in range(2)]
    g_all = gate.cpu().to(F64)
    r0 = 0
    for e in range(E):
        if not rows[e]:
            continue
        t = torch.tensor([r[0] for r in rows[e]])
        j = torch.tensor([r[1] for r in rows[e]])
        v = xd[t]
        if weights8 is None:
            w1, w3, w2 = of(W1, e), of(W3, e), of(W2, e)
        else:
            v = rows8(v)[0]
            w1, w3, w2 = (values8(w[e], s[e], n) for w, s, n in
                          zip((W1, W3, W2), weights8, (x.shape[1], x.shape[1], F)))
        p1, e1 = product(v, torch.zeros_like(v), w1, of(b1, e))
        p3, e3 = product(v, torch.zeros_like(v), w3, of(b3, e))
        a = act(kind, p1)
        h = a * p3
        ea = 1.13 * e1 + a.abs() * act_error(p1)
        eh = ea * (p3.abs() + e3) + (a.abs() + ea) * e3 + 4 * U32 * h.abs()
        if weights8 is None:
            eh = eh + u * (h.abs() + eh)
        else:
            h, eh = hidden8(h, eh)
        z, ez = product(h, eh, w2, of(b2, e))
        g = g_all[t, j][:, None]
        # An expert may stand twice in a token's choices: add row by row. The
        # gate's product, and its rounding to x's type before the combine.
        y.index_add_(0, t, g * z)
        bound.index_add_(0, t, g * ez + (u + 4 * U32) * (g * z.abs() + g * ez))
        size.index_add_(0, t, g * z.abs() + g * ez)
        for q, (p, ep) in enumerate(((p1, e1), (p3, e3))):
            pre[q][r0:r0 + len(t)] = p
            pre_e[q][r0:r0 + len(t)] = ep + u * (p.abs() + ep)
        r0 += len(t)
    bound += (k + 1) * U32 * size
    bound += u * (y.abs() + bound)
    return dict(y=y, y_err=bound, pos=pos, keep=keep, pre=pre, pre_err=pre_e, rows=r0)


def backward(kind, x, idx, gate, p1, p3, W1, W3, W2, b2, dy, C):
    E, d, F = W1.shape
    T, k = idx.shape
    dt = x.dtype
    u = STEP[dt]
    xd, yd, g_all = (v.cpu().to(F64) for v in (x, dy, gate))
    _, _, rows = slots(idx.cpu(), E, C)
    out = dict(dx=yd.clone(), dgate=torch.zeros((T, k), dtype=F64))
    err = {n: torch.zeros_like(v) for n, v in out.items()}
    size = yd.abs()
    for n, shape in dict(dW1=(E, d, F), dW3=(E, d, F), dW2=(E, F, d), db1=(E, F), db3=(E, F),
                         db2=(E, d)).items():
        out[n], err[n] = torch.zeros(shape, dtype=F64), torch.zeros(shape, dtype=F64)
    r0 = 0
    for e in range(E):
        if not rows[e]:
            continue
        n = len(rows[e])
        t = torch.tensor([r[0] for r in rows[e]])
        j = torch.tensor([r[1] for r in rows[e]])
        w1, w3, w2 = of(W1, e), of(W3, e), of(W2, e)
        q1, q3 = (p[r0:r0 + n].cpu().to(F64) for p in (p1, p3))
        r0 += n
        g = g_all[t, j][:, None]
        v, up = xd[t], yd[t]
        a, s = act(kind, q1), slope(kind, q1)
        ea = a.abs() * act_error(q1) + 2.0 ** -24
        es = (2 + q1.abs()) * act_error(q1)
        if kind == RELU:
            ea, es = torch.zeros_like(a), torch.zeros_like(a)
        h = a * q3
        eh = ea * q3.abs() + U32 * h.abs()
        D, eD = product(up, torch.zeros_like(up), w2.t(), None)
        dP1, dP3 = g * D * q3 * s, g * D * a
        e1 = g * q3.abs() * (eD * (s.abs() + es) + D.abs() * es) + 4 * U32 * dP1.abs()
        e3 = g * (eD * (a.abs() + ea) + D.abs() * ea) + 4 * U32 * dP3.abs()
        e1, e3 = (ei + u * (dP.abs() + ei) for ei, dP in ((e1, dP1), (e3, dP3)))
        dU = g * up
        eU = (u + U32) * dU.abs()
        ehr = eh + u * (h.abs() + eh)
        # dgate: D and h stay in 32 bits.
        dg = (D * h).sum(1)
        edg = (eD * (h.abs() + eh) + D.abs() * eh + (F + 64) * U32 * D.abs() * h.abs()).sum(1)
        if b2 is not None:
            b = of(b2, e)
            dg = dg + up @ b
            edg = edg + (d + 64) * U32 * (up.abs() @ b.abs())
        out["dgate"][t, j] = dg
        err["dgate"][t, j] = edg + 4 * U32 * dg.abs()

        def wgrad(name, A, eA, B, eB):
            r = A.t() @ B
            m = A.abs().t() @ B.abs()
            ee = (eA.t() @ (B.abs() + eB)) + A.abs().t() @ eB + n * U32 * m
            out[name][e], err[name][e] = r, ee + u * (r.abs() + ee)
        zero = torch.zeros_like(v)
        wgrad("dW1", v, zero, dP1, e1)
        wgrad("dW3", v, zero, dP3, e3)
        wgrad("dW2", h, ehr, dU, eU)
        for name, B, eB in (("db1", dP1, e1), ("db3", dP3, e3), ("db2", dU, eU)):
            ee = eB.sum(0) + (n + 1) * U32 * B.abs().sum(0)
            out[name][e] = B.sum(0)
            err[name][e] = ee + u * (out[name][e].abs() + ee)
        X1, f1 = product(dP1, e1, w1.t(), None)
        X3, f3 = product(dP3, e3, w3.t(), None)
        ex = f1 + f3 + (d + 2 * F) * U32 * (X1.abs() + X3.abs())
        out["dx"].index_add_(0, t, X1 + X3)
        err["dx"].index_add_(0, t, ex)
        size.index_add_(0, t, X1.abs() + X3.abs())
    err["dx"] += (k + 1) * U32 * size
    err["dx"] += u * (out["dx"].abs() + err["dx"])
    return out, err


# ----------------------------------------------------------------------------- 8 bits
def e4m3_table():
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(v[:127], dtype=F64)


def scale_exponent(top):
    """The smallest e >= -124 with 448 * 2^e >= top, by trying."""
    e = torch.full_like(top, -124.0)
    while True:
        more = 448 * torch.exp2(e) < top
        if not bool(more.any()):
            return e
        e = torch.where(more, e + 1, e)


def nearest(v, e):
    """The e4m3 value nearest to v / 2^e, ties to the even one, times 2^e."""
    table = e4m3_table()
    q = v.abs() / torch.exp2(e)
    i = torch.searchsorted((table[1:] + table[:-1]) / 2, q.contiguous())
    mid = torch.cat([(table[1:] + table[:-1]) / 2, torch.tensor([math.inf], dtype=F64)])
    i = torch.where((q == mid[i]) & (i % 2 == 1), i + 1, i).clamp(max=126)
    return torch.copysign(table[i], v) * torch.exp2(e)


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def by_block(v):
    """Each element's block's largest magnitude, for blocks of 128 columns."""
    n = blocks(v.shape[-1])
    w = torch.nn.functional.pad(v.abs(), (0, n * BLOCK - v.shape[-1]))
    top = w.view(*v.shape[:-1], n, BLOCK).amax(-1)
    return top.repeat_interleave(BLOCK, -1)[..., : v.shape[-1]]


def rows8(v):
    e = scale_exponent(by_block(v))
    return nearest(v, e), e


def hidden8(h, eh):
    """Hidden rows, off by at most eh, through bf16 to 8 bits: the values, and
    how far apart the values are that h - eh and h + eh may go to."""
    b = h.to(torch.float32).to(torch.bfloat16).to(F64)
    q = rows8(b)[0]
    lo, hi = (h - eh), (h + eh)
    lo, hi = (w.to(torch.float32).to(torch.bfloat16).to(F64) for w in (lo, hi))
    mag = torch.maximum(lo.abs(), hi.abs())
    small = torch.where(lo * hi < 0, torch.zeros_like(lo), torch.minimum(lo.abs(), hi.abs()))
    spread = torch.zeros_like(h)
    for top in (by_block(mag), by_block(small)):
        e = scale_exponent(top)
        for w in (lo, hi):
            spread = torch.maximum(spread, (nearest(w.clamp(-448 * torch.exp2(e), 448 *
                                                            torch.exp2(e)), e) - q).abs())
    return q, spread


def weights8(W):
    """W [E,K,N] to (bytes [E,N,Kp], scale bytes), one block after the other."""
    E, K, N = W.shape
    k, n = blocks(K), blocks(N)
    table = e4m3_table()
    q = torch.zeros((E, N, k * BLOCK), dtype=torch.uint8)
    sc = torch.zeros((E, n, k), dtype=torch.uint8)
    Wd = W.cpu().to(F64)
    for e in range(E):
        for a in range(n):
            for b in range(k):
                part = Wd[e, b * BLOCK:(b + 1) * BLOCK, a * BLOCK:(a + 1) * BLOCK]
                ex = scale_exponent(part.abs().amax())
                v = nearest(part, ex) / torch.exp2(ex)
                code = torch.searchsorted(table, v.abs().contiguous()).to(torch.uint8)
                code = code + 128 * torch.signbit(part).to(torch.uint8)
                q[e, a * BLOCK:(a + 1) * BLOCK, b * BLOCK:b * BLOCK + part.shape[0]] = code.t()
                sc[e, a, b] = int(ex) + 127
    return q, sc


def values8(w8, scale, K):
    """One expert's weight [K, N] from its bytes [N, Kp] and scales."""
    table = e4m3_table()
    w8, scale = w8.cpu(), scale.cpu()
    v = table[(w8 & 127).long().clamp(max=126)] * torch.where(w8 > 127, -1.0, 1.0)
    up = torch.exp2(scale.to(F64) - 127)
    up = up.repeat_interleave(BLOCK, 0)[: w8.shape[0]].repeat_interleave(BLOCK, 1)
    return (v * up).t()[:K].contiguous()

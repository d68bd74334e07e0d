"""Cases of the gated experts' operators.

Each expert is a gated feed-forward block, U(x) = (act(x W1 + b1) * (x W3 +
b3)) W2 + b2, applied to tokens whose experts and gate values are given.
Operators and their public calls (sparsely_gated_mixture_gb300.binding):

* ``moe_experts_gated``: capacity, dispatch, the experts and the combine with
  the residual, y = x + sum_j gate_j U_j(x), from one token to long batches;
  a training step also keeps the two pre-activations;
* ``moe_experts_gated_backward``: its gradients from those;
* ``moe_weights_fp8``: expert weights as e4m3 values with one power-of-two
  scale for each block of 128 x 128, laid out for the product below;
* ``moe_experts_gated_fp8``: the same layer for serving, both matrix products
  in e4m3 with such scales (tokens and hidden rows: a scale per 128 columns).

Sizes are those of the repository's workloads (the noisy top-4 layer, the
top-2 large-expert layer) and odd ones around them.
"""
import math

import torch

own = False

SILU, GELU, RELU = "silu", "gelu", "relu"
BLOCK = 128      # values that share a scale
LOW = -124       # the smallest exponent of a scale
FLOPS = 3e12     # most of a drawn case
WEIGHTS = 8 * 4096 * 14336  # most values of one of a drawn case's weights


# ----------------------------------------------------------------------------- cases
def _case(op, T, d, E, d_ff, k, cf=2.0, act=SILU, dtype="bf16", biases=False, keeps=False,
          name=None):
    c = dict(op=op, T=T, d=d, E=E, d_ff=d_ff, k=k, cf=cf, act=act, dtype=dtype, biases=biases,
             keeps=keeps)
    if name:
        c["name"] = name
    return c


def _weights(E, K, N, dtype="bf16", name=None):
    c = dict(op="weights", E=E, K=K, N=N, dtype=dtype)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One token of one stream through small experts: the smallest call,
        # bound by latency.
        _case("gated", 1, 512, 16, 1024, 4, name="gated_t1_top4_e16"),
        # A full decoding batch through the large experts, all of them in use:
        # every weight is read once.
        _case("gated", 64, 4096, 8, 14336, 2, cf=4.0, biases=True, name="gated_t64_top2_large"),
        # An fp32 layer of odd widths and a tight capacity.
        _case("gated", 517, 130, 6, 234, 3, cf=1.1, act=GELU, dtype="f32", biases=True,
              keeps=True, name="gated_odd_f32"),
        # A training batch of the top-4 layer, pre-activations kept.
        _case("gated", 4096, 512, 16, 1024, 4, act=GELU, biases=True, keeps=True,
              name="gated_top4_e16"),
        # A prompt batch of the large-expert layer.
        _case("gated", 8192, 4096, 8, 14336, 2, cf=1.25, name="gated_top2_large"),
        # The backward of the top-4 layer, of the large-expert layer at half
        # its batch, and of the small fp32 layer.
        _case("backward", 4096, 512, 16, 1024, 4, act=GELU, biases=True, name="backward_top4_e16"),
        _case("backward", 4096, 4096, 8, 14336, 2, cf=1.25, name="backward_top2_large"),
        _case("backward", 517, 130, 6, 234, 3, cf=1.1, dtype="f32", biases=True,
              name="backward_odd_f32"),
        # One projection of the large experts to 8 bits, when a checkpoint is
        # loaded for serving; and a ragged fp32 one.
        _weights(8, 4096, 14336, name="weights_fp8_large"),
        _weights(5, 331, 771, dtype="f32", name="weights_fp8_ragged"),
        # One token through the large experts in 8 bits (two experts' weights
        # read), and a prompt batch.
        _case("fp8", 1, 4096, 8, 14336, 2, name="fp8_t1_top2_large"),
        _case("fp8", 8192, 4096, 8, 14336, 2, cf=1.25, name="fp8_top2_large"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "backward", "weights", "fp8", "fp8"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    # Widths in steps of 64 (the usual ones), of 8 or odd.
    step = rng.choice([64, 64, 64, 128, 8, 2, 1])
    E = _log(rng, 2, 256)
    if op == "weights":
        K = max(step, _log(rng, 64, 8192) // step * step)
        N = max(step, min(_log(rng, 64, 16384), WEIGHTS // (E * K) + 1) // step * step)
        return _weights(E, K, N, dtype=dtype)
    if op == "fp8":
        dtype = "bf16"
    k = rng.randint(1, min(8 if op != "backward" else 4, E))
    small = dtype == "f32" or step < 64
    d = max(step, _log(rng, 64, 1024 if small else 4096) // step * step)
    top = min(2048 if small else 14336, WEIGHTS // (E * d))
    d_ff = max(step, _log(rng, 64, max(65, top)) // step * step)
    few = op != "backward" and rng.random() < 0.4
    if few:
        T = _log(rng, 1, 64)
        cf = rng.choice([1.0, 2.0, float(E)])
    else:
        T = _log(rng, 1 if op == "backward" else 65, 8192)
        cf = rng.choice([1.0, 1.25, 2.0])
    most = (0.05 if small else 1.0) * FLOPS / (2 if op == "backward" else 1)
    T = max(1, min(T, int(most / (6 * k * d * d_ff))))
    act = rng.choice([SILU, SILU, GELU, RELU])
    return _case(op, T, d, E, d_ff, k, cf=cf, act=act, dtype=dtype, biases=rng.random() < 0.5,
                 keeps=op == "gated" and not few and rng.random() < 0.5)


def _capacity(c):
    return max(1, min(c["T"], math.floor(c["k"] * c["T"] * c["cf"] / c["E"])))


def _act(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    """The tensors that a program holds before the call: x ~ N(0, 1), weights
    ~ N(0, 1 / fan_in), each token's k experts and their gate values from a
    router that prefers some experts; for the backward the pre-activations
    that the forward kept and dy ~ N(0, 1); for the 8-bit layer the weights'
    values and scales."""
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(seed)
    act = _act(c)

    def normal(*shape, std=1.0, dtype=act):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    if c["op"] == "weights":
        # Columns of different sizes, as trained weights have.
        E, K, N = c["E"], c["K"], c["N"]
        size = torch.exp2(normal(E, 1, N, dtype=torch.float32))
        s = dict(case=c, W=(normal(E, K, N, std=K ** -0.5) * size).to(act))
        if own:
            _plan(s)
        return s
    T, d, E, F, k = c["T"], c["d"], c["E"], c["d_ff"], c["k"]
    H = normal(T, E, dtype=torch.float32) + normal(E, std=0.3, dtype=torch.float32)
    top, idx = torch.sort(H, dim=1, descending=True, stable=True)
    e = torch.exp(top[:, :k] - top[:, :1])
    s = dict(case=c, x=normal(T, d), idx=idx[:, :k].to(torch.int32).contiguous(),
             gate=(e / e.sum(1, keepdim=True)).contiguous(), b1=None, b3=None, b2=None)
    if c["biases"]:
        s.update(b1=normal(E, F, std=0.1), b3=normal(E, F, std=0.1), b2=normal(E, d, std=0.1))
    shapes = dict(W1=(E, d, F), W3=(E, d, F), W2=(E, F, d))
    if c["op"] == "fp8":
        for w, (n, K, N) in shapes.items():
            s[w] = torch.empty((n, N, _blocks(K) * BLOCK), dtype=torch.uint8, device="cuda")
            s["s" + w] = torch.empty((n, _blocks(N), _blocks(K)), dtype=torch.uint8, device="cuda")
            for e in range(n):
                q, ex = _quantise_weights(normal(1, K, N, std=K ** -0.5))
                s[w][e], s["s" + w][e] = q.view(torch.uint8)[0], ex[0]
    else:
        for w, (n, K, N) in shapes.items():
            s[w] = normal(n, K, N, std=K ** -0.5)
    if c["op"] == "backward":
        off, tok = _slots(c, s["idx"])[2:4]
        s.update(dy=normal(T, d), p1=torch.zeros((T * k, F), dtype=act, device="cuda"),
                 p3=torch.zeros((T * k, F), dtype=act, device="cuda"))
        n = off.tolist()
        for e in range(E):
            if n[e + 1] > n[e]:
                rows = s["x"][tok[n[e]:n[e + 1]]]
                for p, w, b in (("p1", "W1", "b1"), ("p3", "W3", "b3")):
                    v = rows @ s[w][e]
                    s[p][n[e]:n[e + 1]] = v if s[b] is None else v + s[b][e]
    if own:
        _plan(s)
    return s


def _plan(s):
    """Workspaces and buffers, sized by the library and kept by the program."""
    from sparsely_gated_mixture_gb300 import binding as B
    c = s["case"]

    def buf(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    if c["op"] == "weights":
        n8, ns = B.moe_weights_fp8_size(c["E"], c["K"], c["N"])
        s.update(w8=buf(n8), ws=buf(256), scale=buf(ns))
        return
    cfg = B.config(c["T"], c["d"], c["E"], c["d_ff"], c["k"], c["cf"],
                   act_dtype=B.MOE_BF16 if c["dtype"] == "bf16" else B.MOE_F32)
    s["cfg"] = cfg
    s["activation"] = dict(silu=B.MOE_ACT_SILU, gelu=B.MOE_ACT_GELU, relu=B.MOE_ACT_RELU)[c["act"]]
    size = dict(gated=B.moe_gated_workspace_size, fp8=B.moe_gated_fp8_workspace_size,
                backward=B.moe_gated_backward_workspace_size)[c["op"]]
    s["ws"] = buf(size(cfg))
    if c["keeps"]:
        s["p1"] = torch.zeros((c["T"] * c["k"], c["d_ff"]), dtype=_act(c), device="cuda")
        s["p3"] = torch.zeros_like(s["p1"])


# ----------------------------------------------------------------------------- plain forms
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _slots(c, idx):
    """Token-order slots under capacity: pos and keep [T, k], the packed rows'
    offsets, and per packed row its token and choice."""
    E = c["E"]
    flat = idx.reshape(-1).long()
    hot = (flat[:, None] == torch.arange(E, device=flat.device)).to(torch.int32)
    pos = (torch.cumsum(hot, 0) - hot).gather(1, flat[:, None]).reshape(idx.shape)
    keep = pos < _capacity(c)
    kept = torch.nonzero(keep.reshape(-1))[:, 0]
    row = kept[torch.sort(flat[kept], stable=True)[1]]
    off = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    off[1:] = torch.cumsum((hot * keep.reshape(-1, 1)).sum(0), 0)
    return pos, keep, off, row // c["k"], row


def _sigmoid(v):
    e = torch.exp(-torch.abs(v))
    return torch.where(v >= 0, 1 / (1 + e), e / (1 + e))


def _activation(c, v):
    if c["act"] == SILU:
        return v * _sigmoid(v)
    if c["act"] == GELU:
        return v * 0.5 * torch.erfc(-v * 0.5 ** 0.5)
    return torch.clamp(v, min=0)


def _slope(c, v):
    if c["act"] == SILU:
        t = _sigmoid(v)
        return t * (1 + v * (1 - t))
    if c["act"] == GELU:
        bell = torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5
        return 0.5 * torch.erfc(-v * 0.5 ** 0.5) + v * bell
    return (v > 0).to(v.dtype)


def _pow2(e):
    """2^e, exactly, for whole e >= -126."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_e4m3(v, top):
    """v in 32 bits and the largest magnitude of its block: e4m3 values and
    the scale's exponent, the smallest whose 448 reaches the largest."""
    m, ex = torch.frexp(top)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    e = torch.where(top > 0, e, LOW).clamp(min=LOW)
    q = v * _pow2(-e)
    step = _pow2((torch.frexp(q)[1] - 1).clamp(min=-6) - 3)
    return torch.round(q / step) * step, e


def _quantise_weights(W):
    """W [E, K, N] to e4m3 [E, N, K rounded up to 128 by zeros] and scale bytes
    (exponent + 127) [E, N / 128, K / 128] (rounded up)."""
    E, K, N = W.shape
    k, n = _blocks(K), _blocks(N)
    b = torch.nn.functional.pad(W, (0, n * BLOCK - N, 0, k * BLOCK - K)).float()
    b = b.view(E, k, BLOCK, n, BLOCK)
    q, e = _to_e4m3(b, b.abs().amax((2, 4), keepdim=True))
    q = q.to(torch.float8_e4m3fn).view(torch.uint8)
    q = q.permute(0, 3, 4, 1, 2).reshape(E, n * BLOCK, k * BLOCK)[:, :N].contiguous()
    e = (e[:, :, 0, :, 0] + 127).to(torch.uint8).transpose(1, 2).contiguous()
    return q.view(torch.float8_e4m3fn), e


def _quantise_rows(v):
    """Rows v [..., K] in 32 bits to the values that e4m3 with a scale per 128
    columns holds."""
    K = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, _blocks(K) * BLOCK - K))
    b = b.view(*v.shape[:-1], -1, BLOCK)
    q, e = _to_e4m3(b, b.abs().amax(-1, keepdim=True))
    return (q * _pow2(e)).reshape(*v.shape[:-1], -1)[..., :K]


def _values(w8, scale, e=None):
    """The weights [.., K, N] of experts e (all: None) that 8 bits hold."""
    if e is not None:
        w8, scale = w8[e], scale[e]
    E, N, K = w8.shape
    q = w8.view(torch.float8_e4m3fn).float().view(E, N, -1, BLOCK)
    up = _pow2(scale.int() - 127).repeat_interleave(BLOCK, 1)[:, :N]
    return (q * up[..., None]).view(E, N, K).transpose(1, 2)


def _experts(s, xs, e=None):
    """The gated blocks of xs [n, m, d] under the weights of experts e [n]
    (all: None): their outputs and both pre-activations."""
    c = s["case"]

    def of(w):
        return w.float() if e is None else w[e].float()

    def product(v, w, b):
        if c["op"] == "fp8":
            m = _values(s[w], s["s" + w], e)
            v = _quantise_rows(v)
            m = m[:, : v.shape[-1]]
        else:
            m = of(s[w])
        r = torch.matmul(v, m)
        return r if s[b] is None else r + of(s[b])[:, None]

    p1, p3 = product(xs, "W1", "b1"), product(xs, "W3", "b3")
    h = _activation(c, p1) * p3
    if c["op"] == "fp8":  # a hidden row is a bf16 row before it is put in 8 bits
        h = h.to(torch.bfloat16).float()
    return product(h, "W2", "b2"), p1, p3


def _plain_gated(s):
    c, x = s["case"], s["x"].float()
    T, E, k, F, act = c["T"], c["E"], c["k"], c["d_ff"], _act(c)
    idx = s["idx"].long()
    pos, keep, _, _, row = _slots(c, idx)
    if T * k < E:  # each choice's own weights
        t = torch.arange(T * k, device=x.device) // k
        o, p1, p3 = (v[:, 0] for v in _experts(s, x[t][:, None], idx.reshape(-1)))
        at = row
    else:          # slots of every expert
        C = _capacity(c)
        slot = torch.where(keep, idx * C + pos, E * C).reshape(-1)
        xs = x.new_zeros((E * C + 1, c["d"]))
        xs[slot] = x.repeat_interleave(k, 0)
        o, p1, p3 = (v.reshape(E * C, -1) for v in _experts(s, xs[: E * C].view(E, C, -1)))
        o = torch.cat([o, o.new_zeros((1, c["d"]))])[slot]
        at = slot[row]
    w = s["gate"] * keep
    y = x + (w[:, :, None] * o.view(T, k, -1)).sum(1)
    r = dict(y=y.to(act), pos=pos.to(torch.int32), keep=keep.to(torch.uint8))
    if c["keeps"]:
        for name, p in (("p1", p1), ("p3", p3)):
            r[name] = torch.zeros((T * k, F), dtype=act, device=x.device)
            r[name][: row.numel()] = p[at].to(act)
    return r


def _plain_backward(s):
    c = s["case"]
    T, d, E, k, C, act = c["T"], c["d"], c["E"], c["k"], _capacity(c), _act(c)
    idx, gate = s["idx"].long(), s["gate"]
    pos, _, _, tok, row = _slots(c, idx)
    n = row.numel()
    slot = (idx * C + pos).reshape(-1)[row]  # rows of each expert in slots of their own
    dy, x = s["dy"].float(), s["x"].float()

    def pad(rows):
        v = rows.new_zeros((E * C, rows.shape[1]))
        v[slot] = rows
        return v.view(E, C, -1)

    def t(w):
        return s[w].float().transpose(1, 2)
    p1, p3 = pad(s["p1"][:n].float()), pad(s["p3"][:n].float())
    a = _activation(c, p1)
    h = a * p3
    g = pad(gate.reshape(-1)[row][:, None])
    dY = pad(dy[tok])
    D = torch.bmm(dY, t("W2"))
    dg = (D * h).sum(2)
    if s["b2"] is not None:
        dg = dg + (dY * s["b2"].float()[:, None]).sum(2)
    D = g * D
    dP1, dP3 = D * p3 * _slope(c, p1), D * a
    dU = g * dY
    dX = torch.bmm(dP1, t("W1")) + torch.bmm(dP3, t("W3"))
    X = pad(x[tok])
    dx = dy.index_add(0, tok, dX.view(E * C, d)[slot])
    dgate = dy.new_zeros(T * k)
    dgate[row] = dg.view(-1)[slot]
    r = dict(dx=dx.to(act), dgate=dgate.view(T, k),
             dW1=torch.bmm(X.transpose(1, 2), dP1).to(act),
             dW3=torch.bmm(X.transpose(1, 2), dP3).to(act),
             dW2=torch.bmm(h.transpose(1, 2), dU).to(act))
    if c["biases"]:
        r.update(db1=dP1.sum(1).to(act), db3=dP3.sum(1).to(act), db2=dU.sum(1).to(act))
    return r


def _plain_weights(s):
    q, e = _quantise_weights(s["W"])
    return dict(w8=q, scale=e)


# ----------------------------------------------------------------------------- the operators
def _own_gated(s):
    from sparsely_gated_mixture_gb300 import binding as B
    c, x = s["case"], s["x"]
    y = torch.empty_like(x)
    pos = torch.empty((c["T"], c["k"]), dtype=torch.int32, device="cuda")
    keep = torch.empty((c["T"], c["k"]), dtype=torch.uint8, device="cuda")
    r = dict(y=y, pos=pos, keep=keep)
    if c["op"] == "fp8":
        B.moe_experts_gated_fp8(s["cfg"], s["activation"], x, s["idx"], s["gate"], s["W1"],
                                s["sW1"], s["b1"], s["W3"], s["sW3"], s["b3"], s["W2"], s["sW2"],
                                s["b2"], y, s["ws"], pos=pos, keep=keep)
        return r
    if c["keeps"]:
        r.update(p1=s["p1"], p3=s["p3"])
    B.moe_experts_gated(s["cfg"], s["activation"], x, s["idx"], s["gate"], s["W1"], s["b1"],
                        s["W3"], s["b3"], s["W2"], s["b2"], y, s["ws"], pre1=r.get("p1"),
                        pre3=r.get("p3"), pos=pos, keep=keep)
    return r


def _own_backward(s):
    from sparsely_gated_mixture_gb300 import binding as B
    c = s["case"]

    def like(v):
        return None if v is None else torch.empty_like(v)
    r = dict(dx=like(s["x"]), dgate=like(s["gate"]), dW1=like(s["W1"]), dW3=like(s["W3"]),
             dW2=like(s["W2"]), db1=like(s["b1"]), db3=like(s["b3"]), db2=like(s["b2"]))
    B.moe_experts_gated_backward(s["cfg"], s["activation"], s["x"], s["idx"], s["gate"], s["p1"],
                                 s["p3"], s["W1"], s["W3"], s["W2"], s["b2"], s["dy"], r["dx"],
                                 r["dgate"], r["dW1"], r["db1"], r["dW3"], r["db3"], r["dW2"],
                                 r["db2"], s["ws"])
    return r


def _own_weights(s):
    from sparsely_gated_mixture_gb300 import binding as B
    c = s["case"]
    B.moe_weights_fp8(c["E"], c["K"], c["N"], B.MOE_BF16 if c["dtype"] == "bf16" else B.MOE_F32,
                      s["W"], s["w8"], s["scale"], s["ws"])
    E, k, n = c["E"], _blocks(c["K"]), _blocks(c["N"])
    return dict(w8=s["w8"].view(torch.float8_e4m3fn).view(E, c["N"], k * BLOCK),
                scale=s["scale"].view(E, n, k))


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(gated=_own_gated, fp8=_own_gated, backward=_own_backward,
                    weights=_own_weights)[op](state)
    return dict(gated=_plain_gated, fp8=_plain_gated, backward=_plain_backward,
                weights=_plain_weights)[op](state)


def work(case):
    """Inputs read once, outputs written once. Experts in use: the distinct
    ones of T tokens' k choices; rows: those under the capacity."""
    c = case
    eb = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "weights":
        n = c["E"] * c["K"] * c["N"]
        return dict(bytes=n * (eb + 1), flops=3 * n)
    T, d, E, F, k = c["T"], c["d"], c["E"], c["d_ff"], c["k"]
    A = min(T * k, E * _capacity(c)) * (1.0 if T <= 64 else 0.97)
    active = E * (1 - (1 - min(1.0, A / T / E)) ** T)
    weights = active * 3 * d * F
    if c["op"] == "backward":
        return dict(bytes=2 * weights * eb + 3 * T * d * eb + 2 * A * F * eb,
                    flops=12 * A * d * F)
    if c["op"] == "fp8":
        return dict(bytes=weights + 2 * T * d * eb, flops=6 * A * d * F)
    return dict(bytes=weights * eb + 2 * T * d * eb + (2 * A * F * eb if c["keeps"] else 0),
                flops=6 * A * d * F)


# ----------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "weights":
        return _exact_weights(s)
    if work(case)["flops"] > 7e12:
        return None
    return _exact_backward(s) if case["op"] == "backward" else _exact_gated(s)


def _rows_of(c, idx, e):
    """Tokens and choices of expert e's accepted rows, in token order."""
    at = torch.nonzero(idx == e)[: _capacity(c)]
    return at[:, 0], at[:, 1]


def _table():
    """e4m3's finite values from zero on, in order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(v, top):
    """The e4m3 value nearest to v / 2^e (the even one on ties) and e, the
    smallest exponent >= LOW with 448 * 2^e >= top, by search."""
    e = torch.full_like(top, LOW)
    lg = torch.floor(torch.log2(top.clamp(min=2.0 ** -130)))
    for step in (-10, -9, -8, -7):
        e = torch.where((448 * torch.exp2(lg + step - 1) < top) & (lg + step >= LOW), lg + step, e)
    table = _table()
    mid = (table[1:] + table[:-1]) / 2
    q = (v.abs() / torch.exp2(e)).contiguous()
    i = torch.searchsorted(mid, q)  # ties: the lower one
    tie = q == mid[i.clamp(max=mid.numel() - 1)]
    i = torch.where(tie & (i % 2 == 1), i + 1, i).clamp(max=126)
    return torch.copysign(table[i], v), e


def _exact_weights(s):
    W = s["W"]
    E, K, N = W.shape
    out = torch.zeros((E, N, _blocks(K) * BLOCK), dtype=torch.float64, device="cuda")
    for e in range(E):
        for lo in range(0, K, BLOCK):
            part = W[e, lo:lo + BLOCK].double()
            col = part.abs().amax(0)
            tops = [col[a:a + BLOCK].amax().expand(min(BLOCK, N - a)) for a in range(0, N, BLOCK)]
            q, _ = _nearest(part, torch.cat(tops).expand_as(part).contiguous())
            out[e, :, lo:lo + part.shape[0]] = q.t()
    return dict(w8=out, scale=None)


def _exact_rows8(v):
    """Rows' values in 8 bits, block by block."""
    out = torch.empty_like(v)
    for lo in range(0, v.shape[1], BLOCK):
        b = v[:, lo:lo + BLOCK]
        top = b.abs().amax(1, keepdim=True).expand_as(b).contiguous()
        q, e = _nearest(b, top)
        out[:, lo:lo + BLOCK] = q * torch.exp2(e)
    return out


def _exact_weight8(s, w, e, K):
    q = s[w][e].view(torch.float8_e4m3fn).double()
    up = torch.exp2(s["s" + w][e].double() - 127)
    up = up.repeat_interleave(BLOCK, 0)[: q.shape[0]].repeat_interleave(BLOCK, 1)
    return (q * up).t()[:K]


def _exact_act(c, v):
    if c["act"] == SILU:
        return v / (1 + torch.exp(-v))
    if c["act"] == GELU:
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2.0)))
    return v * (v > 0)


def _exact_gated(s):
    """Expert by expert."""
    c = s["case"]
    T, d, F, k = c["T"], c["d"], c["d_ff"], c["k"]
    idx = s["idx"].long()
    y = s["x"].double().clone()
    kept = {p: torch.zeros((T * k, F), dtype=torch.float64, device="cuda") for p in ("p1", "p3")}
    r0 = 0
    for e in range(c["E"]):
        t, j = _rows_of(c, idx, e)
        if not t.numel():
            continue
        v = s["x"][t].double()

        def times(v, w, b, K):
            if c["op"] == "fp8":
                r = _exact_rows8(v) @ _exact_weight8(s, w, e, K)
            else:
                r = v @ s[w][e].double()
            return r if s[b] is None else r + s[b][e].double()
        p1, p3 = times(v, "W1", "b1", d), times(v, "W3", "b3", d)
        h = _exact_act(c, p1) * p3
        if c["op"] == "fp8":
            h = h.to(torch.bfloat16).double()
        y[t] += s["gate"][t, j].double()[:, None] * times(h, "W2", "b2", F)
        if c["keeps"]:
            kept["p1"][r0:r0 + t.numel()], kept["p3"][r0:r0 + t.numel()] = p1, p3
        r0 += t.numel()
    r = dict(y=y, pos=None, keep=None)
    return {**r, **kept} if c["keeps"] else r


def _exact_backward(s):
    """Expert by expert, through automatic differentiation of the activation."""
    c = s["case"]
    idx = s["idx"].long()
    f64 = torch.float64
    dy = s["dy"].to(f64)
    dx = dy.clone()
    dgate = torch.zeros(idx.shape, dtype=f64, device="cuda")
    out = {n: torch.zeros(s[n[1:]].shape, dtype=f64, device="cuda")
           for n in ("dW1", "dW3", "dW2") + (("db1", "db3", "db2") if c["biases"] else ())}
    r0 = 0
    for e in range(c["E"]):
        t, j = _rows_of(c, idx, e)
        if not t.numel():
            continue
        rows = slice(r0, r0 + t.numel())
        r0 += t.numel()
        W1, W3, W2 = (s[w][e].to(f64) for w in ("W1", "W3", "W2"))
        gate = s["gate"][t, j].to(f64)[:, None]
        with torch.enable_grad():
            p1 = s["p1"][rows].to(f64).requires_grad_()
            p3 = s["p3"][rows].to(f64).requires_grad_()
            h = _exact_act(c, p1) * p3
        U = h.detach() @ W2
        if s["b2"] is not None:
            U = U + s["b2"][e].to(f64)
        up = gate * dy[t]
        dgate[t, j] = (U * dy[t]).sum(1)
        dP1, dP3 = torch.autograd.grad(h, (p1, p3), up @ W2.t())
        v = s["x"][t].to(f64)
        out["dW1"][e], out["dW3"][e], out["dW2"][e] = v.t() @ dP1, v.t() @ dP3, h.detach().t() @ up
        if c["biases"]:
            out["db1"][e], out["db3"][e], out["db2"][e] = dP1.sum(0), dP3.sum(0), up.sum(0)
        dx.index_add_(0, t, dP1 @ W1.t() + dP3 @ W3.t())
    return dict(dx=dx, dgate=dgate, **out)

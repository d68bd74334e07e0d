"""Cases of the layer's few-token and checkpointed-training operators.

Operators and their public calls (sparsely_gated_mixture_gb300.binding):

* ``moe_forward_few``: the whole flat layer (router, top-k, capacity, experts,
  combine) for the 1 to 64 tokens of a decoding step;
* ``moe_forward_threshold_few``: the same for the threshold mask, the layer's
  inference-time gate;
* ``moe_checkpoint_save`` / ``moe_checkpoint_load``: the hidden activations of
  the experts held in 8 bits (e4m3 values, one power-of-two scale per 32) from
  the forward to the backward, and back;
* ``moe_backward_checkpoint``: the layer's backward from such a checkpoint.

Sizes are those of the repository's workloads (the noisy top-4 layer, the
top-2 large-expert layer, the many-small-experts layer and the balanced /
threshold layer) and odd ones around them.
"""
import math

import torch

own = False

TOPK, SWITCH = "topk", "switch"


# ----------------------------------------------------------------------------- cases
def _case(op, T, d, E, d_ff, k, cf=2.0, mode=TOPK, dtype="bf16", noisy=False, biases=False,
          name=None):
    c = dict(op=op, T=T, d=d, E=E, d_ff=d_ff, k=k, cf=cf, mode=mode, dtype=dtype, noisy=noisy,
             biases=biases)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One token of one stream through the noisy top-4 layer: the smallest
        # call, bound by latency.
        _case("few", 1, 512, 16, 1024, 4, name="few_t1_top4_e16"),
        # One token through the large-expert layer: two experts' weights.
        _case("few", 1, 4096, 8, 14336, 2, name="few_t1_top2_large"),
        # A full decoding batch of it, every expert in use.
        _case("few", 64, 4096, 8, 14336, 2, cf=4.0, noisy=True, biases=True,
              name="few_t64_top2_large"),
        # A batch over many small experts: about one row for each of 150.
        _case("few", 40, 512, 1024, 1024, 4, cf=64.0, name="few_t40_top4_e1024"),
        # An fp32 Switch layer of odd widths, a tight capacity that drops tokens.
        _case("few", 13, 770, 24, 1030, 1, cf=1.5, mode=SWITCH, dtype="f32", biases=True,
              name="few_t13_switch_f32"),
        # The threshold mask where it is meant to be used: one example alone,
        # and a batch of them.
        _case("threshold_few", 1, 1024, 64, 4096, 16, name="threshold_t1_e64"),
        _case("threshold_few", 48, 1024, 64, 4096, 16, biases=True, name="threshold_t48_e64"),
        # The hidden rows of the noisy top-4 layer and of the large-expert
        # layer, saved and loaded.
        _case("checkpoint", 4096, 512, 16, 1024, 4, name="checkpoint_top4_e16"),
        _case("checkpoint", 8192, 4096, 8, 14336, 2, cf=1.25, name="checkpoint_top2_large"),
        # The backward of the noisy top-4 layer, of the large-expert layer at
        # half its batch, and of a small fp32 layer of odd widths.
        _case("backward", 4096, 512, 16, 1024, 4, noisy=True, biases=True,
              name="backward_top4_e16"),
        _case("backward", 4096, 4096, 8, 14336, 2, cf=1.25, noisy=True,
              name="backward_top2_large"),
        _case("backward", 517, 130, 6, 234, 3, cf=1.1, dtype="f32", noisy=True, biases=True,
              name="backward_odd_f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "threshold_few", "checkpoint", "backward"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    # Widths in steps of 8 (the usual ones) or odd.
    step = rng.choice([8, 8, 64, 2, 1])
    biases = rng.random() < 0.5
    if op in ("few", "threshold_few"):
        T = _log(rng, 1, 64)
        E = _log(rng, 2, 1024)
        d = max(step, _log(rng, 64, 4096) // step * step)
        # Weights within the large-expert layer's.
        top = min(14336, (8 * 4096 * 14336 // (1 if dtype == "bf16" else 2)) // (E * d))
        d_ff = max(step, _log(rng, 64, max(64, top)) // step * step)
        if op == "threshold_few":
            return _case(op, T, d, max(E, 17), d_ff * 3 // 4 // step * step or step, 16,
                         dtype=dtype, biases=biases)
        mode = SWITCH if rng.random() < 0.25 else TOPK
        k = 1 if mode == SWITCH else rng.randint(1, min(8, E))
        return _case(op, T, d, E, d_ff, k, cf=rng.choice([1.0, 2.0, float(E)]), mode=mode,
                     dtype=dtype, noisy=rng.random() < 0.3, biases=biases)
    E = _log(rng, 2, 128)
    k = rng.randint(1, min(4, E))
    if op == "checkpoint":
        d_ff = max(step, _log(rng, 64, 14336) // step * step)
        T = min(_log(rng, 1, 16384), 100_000_000 // (k * d_ff) + 1)
        return _case(op, T, 64, E, d_ff, k, cf=rng.choice([1.0, 1.5, 2.0]), dtype=dtype)
    mode = SWITCH if rng.random() < 0.25 else TOPK
    k = 1 if mode == SWITCH else k
    if dtype == "f32" or step < 64:
        d, d_ff = (max(step, _log(rng, 16, 256) // step * step) for _ in range(2))
        T = _log(rng, 1, 2048)
    else:
        d, d_ff = (max(64, _log(rng, 64, 2048) // 64 * 64) for _ in range(2))
        T = _log(rng, 64, 8192)
    return _case(op, T, d, E, d_ff, k, cf=rng.choice([1.0, 1.25, 2.0]), mode=mode, dtype=dtype,
                 noisy=rng.random() < 0.6, biases=biases)


def _capacity(c):
    return max(1, min(c["T"], math.floor(c["k"] * c["T"] * c["cf"] / c["E"])))


def _act(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    """The tensors that a program holds before the call: x ~ N(0, 1), router
    and expert weights ~ N(0, 1 / fan_in) and the supplied noise ~ N(0, 1); for
    the backward also the forward's choices, gates and checkpoint."""
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(seed)
    act = _act(c)
    T, d, E, F, k = c["T"], c["d"], c["E"], c["d_ff"], c["k"]

    def normal(*shape, std=1.0, dtype=act):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    s = dict(case=c)
    if c["op"] == "checkpoint":
        # ReLU rows as the experts make them, each row with a scale of its
        # own; the experts' counts as uneven as a router's, under capacity.
        C, A = _capacity(c), T * k
        share = torch.rand(E, generator=g, device="cuda") + 0.5
        choice = torch.multinomial(share, A, replacement=True, generator=g)
        rows = torch.bincount(choice, minlength=E).to(torch.int32).clamp_(max=C)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.cumsum(rows, 0)
        R = min(A, E * C)
        scale = torch.exp2(torch.randn((R, 1), generator=g, device="cuda"))
        h = torch.empty((R, F), dtype=act, device="cuda")
        for lo in range(0, R, 4096):
            hi = min(R, lo + 4096)
            h[lo:hi] = (normal(hi - lo, F, dtype=torch.float32) * scale[lo:hi]).relu_()
        s.update(h=h, off=off, n=int(off[-1]))
    else:
        # Many experts need a sharper router for two of them to pass 1/16.
        sharp = 1 + 0.6 * math.log2(max(E, 64) / 64) if c["op"] == "threshold_few" else 1.0
        s.update(x=normal(T, d), Wg=normal(d, E, std=sharp * d ** -0.5, dtype=torch.float32),
                 W1=normal(E, d, F, std=d ** -0.5), W2=normal(E, F, d, std=F ** -0.5),
                 Wn=None, noise=None, bias=None, b1=None, b2=None)
        if c["noisy"]:
            s.update(Wn=normal(d, E, std=d ** -0.5, dtype=torch.float32),
                     noise=normal(T, E, dtype=torch.float32))
        if c["biases"]:
            s.update(b1=normal(E, F, std=0.1), b2=normal(E, d, std=0.1))
        if c["op"] == "threshold_few":
            # Stand-ins for learned thresholds: a few experts pass, and never
            # more than k = 16, since a token's probabilities sum to 1.
            s["thr"] = torch.full((E,), 1.0 / 15.9 + (0.0 if E >= 64 else 1.0 / E),
                                  device="cuda")
        if c["op"] == "backward":
            _, _, H = _logits(s)
            idx, gate = _select(c, H)
            _, keep, off, tok, _ = _slots(c, idx)
            R = min(T * k, E * _capacity(c))
            h = torch.zeros((R, F), dtype=act, device="cuda")
            n = off.tolist()
            for e in range(E):
                if n[e + 1] > n[e]:
                    p = s["x"][tok[n[e]:n[e + 1]]] @ s["W1"][e]
                    h[n[e]:n[e + 1]] = (p if s["b1"] is None else p + s["b1"][e]).relu_()
            h8, hs = [], []
            for lo in range(0, R, 4096):
                q, e8, _ = _quantise(h[lo:lo + 4096].float())
                h8.append(q.to(torch.float8_e4m3fn).view(torch.uint8))
                hs.append(e8)
            s.update(idx=idx.to(torch.int32), gate=gate.float(), h8=torch.cat(h8),
                     hs=torch.cat(hs), dy=normal(T, d))
    if own:
        _plan(s)
    return s


def _plan(s):
    """Workspaces, sized by the library and kept by the program."""
    from sparsely_gated_mixture_gb300 import binding as B
    c = s["case"]
    cfg = B.config(c["T"], c["d"], c["E"], c["d_ff"], c["k"], c["cf"],
                   B.MOE_GATE_SWITCH if c["mode"] == SWITCH else B.MOE_GATE_TOPK_SOFTMAX,
                   B.MOE_BF16 if c["dtype"] == "bf16" else B.MOE_F32)
    s["cfg"] = cfg

    def buf(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    if c["op"] in ("few", "threshold_few"):
        s["ws"] = buf(B.moe_few_workspace_size(cfg))
    elif c["op"] == "checkpoint":
        _, n8, ns = B.moe_checkpoint_size(cfg)
        s.update(ws=buf(256), h8=buf(n8), hs=buf(ns), out=torch.zeros_like(s["h"]))
    else:
        s.update(ws=buf(B.moe_workspace_size(cfg)), bws=buf(B.moe_backward_workspace_size(cfg)))


# ----------------------------------------------------------------------------- plain forms
def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-torch.abs(z)))


def _logits(s):
    """Clean logits, noise scales and noisy logits in 64 bits (the choice of
    experts lies next to a border)."""
    x = s["x"].double()
    clean = x @ s["Wg"].double()
    if s.get("bias") is not None:
        clean = clean + s["bias"].double()
    if s.get("Wn") is None:
        return clean, None, clean
    sigma = _softplus(x @ s["Wn"].double())
    return clean, sigma, clean + s["noise"].double() * sigma


def _select(c, H):
    """The k largest (lowest index on ties) and their gates."""
    v, i = torch.sort(H, dim=1, descending=True, stable=True)
    idx = i[:, : c["k"]]
    if c["mode"] == SWITCH:
        e = torch.exp(H - v[:, :1])
        return idx, (1.0 / e.sum(dim=1, keepdim=True))
    e = torch.exp(v[:, : c["k"]] - v[:, :1])
    return idx, e / e.sum(dim=1, keepdim=True)


def _slots(c, idx):
    """Token-order slots under capacity: pos and keep [T, k], the packed rows'
    offsets, and per packed row its token and choice."""
    E = c["E"]
    flat = idx.reshape(-1).long()
    hot = (flat[:, None] == torch.arange(E, device=flat.device)).to(torch.int32)
    pos = (torch.cumsum(hot, 0) - hot).gather(1, flat[:, None]).reshape(idx.shape)
    keep = pos < _capacity(c)
    kept = torch.nonzero(keep.reshape(-1))[:, 0]
    order = torch.sort(flat[kept], stable=True)[1]
    row = kept[order]
    off = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    off[1:] = torch.cumsum((hot * keep.reshape(-1, 1)).sum(0), 0)
    return pos, keep, off, row // c["k"], row


def _experts(s, xs, e=None):
    """ReLU FFN of xs [n, m, d] under the weights of experts e [n] (all: None)."""
    def of(w):
        return w.float() if e is None else w[e].float()
    h = torch.matmul(xs, of(s["W1"]))
    if s["b1"] is not None:
        h = h + of(s["b1"])[:, None]
    o = torch.matmul(torch.clamp(h, min=0), of(s["W2"]))
    return o if s["b2"] is None else o + of(s["b2"])[:, None]


def _plain_few(s):
    c, x = s["case"], s["x"].float()
    T, E, k = c["T"], c["E"], c["k"]
    idx, gate = _select(c, _logits(s)[2])
    pos, keep, _, _, _ = _slots(c, idx)
    if T * k < E:  # each choice's own weights
        t = torch.arange(T * k, device=x.device) // k
        o = _experts(s, x[t][:, None], idx.reshape(-1))[:, 0]
    else:          # slots of every expert
        C = _capacity(c)
        slot = torch.where(keep, idx * C + pos, E * C).reshape(-1)
        xs = x.new_zeros((E * C + 1, c["d"]))
        xs[slot] = x.repeat_interleave(k, 0)
        o = _experts(s, xs[: E * C].view(E, C, -1)).reshape(E * C, -1)
        o = torch.cat([o, o.new_zeros((1, c["d"]))])[slot]
    w = (gate * keep).float()
    y = x + (w[:, :, None] * o.view(T, k, -1)).sum(1)
    return dict(y=y.to(_act(c)), idx=idx.to(torch.int32), gate=gate.float(),
                keep=keep.to(torch.uint8))


def _plain_threshold(s):
    c, x = s["case"], s["x"].float()
    E, k = c["E"], c["k"]
    H = _logits(s)[2]
    p = torch.exp(H - H.max(dim=1, keepdim=True)[0])
    p = p / p.sum(dim=1, keepdim=True)
    take = p > s["thr"].double()
    w = p * take
    w = w / torch.clamp(w.sum(dim=1, keepdim=True), min=1e-300)
    idx = torch.sort(torch.where(take, torch.arange(E, device=x.device), E), dim=1)[0][:, :k]
    gate = torch.cat([w, torch.zeros_like(w[:, :1])], 1).gather(1, idx)
    o = _experts(s, x[None])  # every expert on every token
    y = x + (w.float().t()[:, :, None] * o).sum(0)
    return dict(y=y.to(_act(c)), idx=idx.to(torch.int32), gate=gate.float())


def _pow2(e):
    """2^e, exactly, for whole e >= -126."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


BLOCK = 32       # values that share a scale
LOW = -124       # the smallest exponent of a scale


def _quantise(h):
    """Rows h >= 0 in 32 bits: e4m3 values q and the scale bytes (exponent +
    127) of blocks of 32 columns, and the values q * 2^exponent. The exponent
    is the smallest whose 448 reaches the block's largest; a value over zero
    stays over zero (the ReLU's pattern is what the backward needs)."""
    R, F = h.shape
    n = (F + BLOCK - 1) // BLOCK
    b = torch.nn.functional.pad(h, (0, n * BLOCK - F)).view(R, n, BLOCK)
    top = b.max(dim=2, keepdim=True)[0]
    m, ex = torch.frexp(top)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    e = torch.where(top > 0, e, LOW).clamp(min=LOW)
    q = b * _pow2(-e)
    step = _pow2((torch.frexp(q)[1] - 1).clamp(min=-6) - 3)
    q = torch.round(q / step) * step
    q = torch.where(b > 0, q.clamp(min=2.0 ** -9), 0.0)
    q = torch.minimum(q, torch.where(e >= 120, 240.0, 448.0))
    values = q * _pow2(e)

    def rows(v):
        return v.view(R, n * BLOCK)[:, :F].contiguous()
    return rows(q), (e[:, :, 0] + 127).to(torch.uint8), rows(values)


def _plain_checkpoint(s):
    out = torch.zeros_like(s["h"])
    out[: s["n"]] = _quantise(s["h"][: s["n"]].float())[2].to(out.dtype)
    return out


W_IMP, W_LOAD, W_AUX = 0.1, 0.1, 0.1


def _cv2_grad(v):
    m = v.mean()
    var = ((v - m) ** 2).mean()
    return 2 * (v - m) / (v.numel() * m * m) - 2 * var / (v.numel() * m ** 3)


def _plain_backward(s):
    c = s["case"]
    T, d, E, F, k, C = c["T"], c["d"], c["E"], c["d_ff"], c["k"], _capacity(c)
    act = _act(c)
    idx, gate = s["idx"].long(), s["gate"]
    pos, keep, off, tok, row = _slots(c, idx)
    n = row.numel()
    # Rows of each expert in slots of their own: [E, C].
    slot = (idx * C + pos).reshape(-1)[row]
    dy, x = s["dy"].float(), s["x"].float()

    def pad(rows):
        v = rows.new_zeros((E * C, rows.shape[1]))
        v[slot] = rows
        return v.view(E, C, -1)
    h = torch.zeros((n, (F + BLOCK - 1) // BLOCK * BLOCK), device=x.device)
    h[:, :F] = s["h8"][:n].view(torch.float8_e4m3fn).float()
    h = h.view(n, -1, BLOCK) * _pow2(s["hs"][:n, :, None].int() - 127)
    h = pad(h.view(n, -1)[:, :F])
    g = pad(gate.reshape(-1)[row][:, None])
    dY = pad(dy[tok])
    D = torch.bmm(dY, s["W2"].float().transpose(1, 2))
    dg = (D * h).sum(2)
    if s["b2"] is not None:
        dg = dg + (dY * s["b2"].float()[:, None]).sum(2)
    dP = g * D * (h > 0)
    dU = g * dY
    dX = torch.bmm(dP, s["W1"].float().transpose(1, 2)).view(E * C, d)
    dW2 = torch.bmm(h.transpose(1, 2), dU).to(act)
    dW1 = torch.bmm(pad(x[tok]).transpose(1, 2), dP).to(act)
    db1, db2 = dP.sum(1).to(act), dU.sum(1).to(act)
    # The gate: kept choices' <dy, U>, the balancing losses, the softmax.
    dgate = dy.new_zeros(T * k, dtype=torch.float64)
    dgate[row] = dg.view(-1)[slot].double()
    dgate = dgate.view(T, k)
    clean, sigma, H = _logits(s)
    v, order = torch.sort(H, dim=1, descending=True, stable=True)
    hot = torch.zeros((T, E), dtype=torch.bool, device=x.device).scatter_(1, idx, True)
    gate = gate.double()
    imp = torch.zeros((T, E), dtype=torch.float64, device=x.device).scatter_(1, idx, gate).sum(0)
    dgate = dgate + W_IMP * _cv2_grad(imp)[idx]
    p = torch.exp(H - v[:, :1])
    p = p / p.sum(1, keepdim=True)
    first = torch.bincount(idx[:, 0], minlength=E) / T
    dp = (W_AUX * 0.01 * E / T * first).expand(T, E)
    if c["mode"] == SWITCH:
        dp = dp.scatter_add(1, idx, dgate)
        dH = torch.zeros_like(H)
    else:
        t = gate * (dgate - (gate * dgate).sum(1, keepdim=True))
        dH = torch.zeros_like(H).scatter_(1, idx, t)
    dH = dH + p * (dp - (p * dp).sum(1, keepdim=True))
    dc = dz = None
    if sigma is not None:
        dsig = torch.zeros_like(H)
        dc = torch.zeros_like(H)
        if k < E:
            u = (clean - torch.where(hot, v[:, k:k + 1], v[:, k - 1:k])) / sigma
            load = 0.5 * torch.erfc(-u * 0.5 ** 0.5)
            gl = W_LOAD * _cv2_grad(load.sum(0)) * torch.exp(-0.5 * u * u) * (2 * math.pi) ** -0.5
            gl = gl / sigma
            dc, dsig = gl, -gl * u
            own_out = torch.where(hot, gl, 0.0).sum(1, keepdim=True)
            own_in = torch.where(hot, 0.0, gl).sum(1, keepdim=True)
            dH = dH.scatter_add(1, order[:, k:k + 1], -own_out)
            dH = dH.scatter_add(1, idx[:, k - 1:k], -own_in)
        dsig = dsig + s["noise"].double() * dH
        dz = dsig * (1 - torch.exp(-sigma))
    dc = dH if dc is None else dc + dH
    xd = x.double()
    dxr = dc @ s["Wg"].double().t()
    if dz is not None:
        dxr = dxr + dz @ s["Wn"].double().t()
    dx = dy + dxr.float()
    dx = dx.index_add(0, tok, dX[slot])
    return dict(dx=dx.to(act), dWg=(xd.t() @ dc).float(),
                dWn=None if dz is None else (xd.t() @ dz).float(), dbias=dc.sum(0).float(),
                dW1=dW1, db1=db1, dW2=dW2, db2=db2, dgate=dgate.float())


# ----------------------------------------------------------------------------- the operators
def _own_few(s):
    from sparsely_gated_mixture_gb300 import binding as B
    c, x = s["case"], s["x"]
    y = torch.empty_like(x)
    idx = torch.empty((c["T"], c["k"]), dtype=torch.int32, device="cuda")
    gate = torch.empty((c["T"], c["k"]), dtype=torch.float32, device="cuda")
    keep = torch.empty((c["T"], c["k"]), dtype=torch.uint8, device="cuda")
    B.moe_forward_few(s["cfg"], x, s["Wg"], s["Wn"], s["noise"], s["bias"], s["W1"], s["b1"],
                      s["W2"], s["b2"], y, s["ws"], expert_idx=idx, gate=gate, keep=keep)
    return dict(y=y, idx=idx, gate=gate, keep=keep)


def _own_threshold(s):
    from sparsely_gated_mixture_gb300 import binding as B
    c, x = s["case"], s["x"]
    y = torch.empty_like(x)
    idx = torch.empty((c["T"], c["k"]), dtype=torch.int32, device="cuda")
    gate = torch.empty((c["T"], c["k"]), dtype=torch.float32, device="cuda")
    B.moe_forward_threshold_few(s["cfg"], x, s["Wg"], s["bias"], s["thr"], s["W1"], s["b1"],
                                s["W2"], s["b2"], y, s["ws"], expert_idx=idx, gate=gate)
    return dict(y=y, idx=idx, gate=gate)


def _own_checkpoint(s):
    from sparsely_gated_mixture_gb300 import binding as B
    B.moe_checkpoint_save(s["cfg"], s["h"], s["off"], s["h8"], s["hs"], s["ws"])
    B.moe_checkpoint_load(s["cfg"], s["h8"], s["hs"], s["off"], s["out"], s["ws"])
    return s["out"]


def _own_backward(s):
    from sparsely_gated_mixture_gb300 import binding as B
    c, x = s["case"], s["x"]

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")
    T, d, E, F, act = c["T"], c["d"], c["E"], c["d_ff"], _act(c)
    o = dict(dx=torch.empty_like(x), dWg=empty(d, E),
             dWn=None if s["Wn"] is None else empty(d, E), dbias=empty(E),
             dW1=empty(E, d, F, dtype=act), db1=empty(E, F, dtype=act),
             dW2=empty(E, F, d, dtype=act), db2=empty(E, d, dtype=act), dgate=empty(T, c["k"]))
    B.moe_backward_checkpoint(s["cfg"], x, s["Wg"], s["Wn"], s["noise"], s["bias"], s["W1"],
                              s["W2"], s["b2"], s["idx"], s["gate"], s["h8"], s["hs"], s["dy"],
                              W_IMP, W_LOAD, W_AUX, o["dx"],
                              o["dWg"], o["dWn"], o["dbias"], o["dW1"], o["db1"], o["dW2"],
                              o["db2"], o["dgate"], s["ws"], s["bws"])
    return o


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(few=_own_few, threshold_few=_own_threshold, checkpoint=_own_checkpoint,
                    backward=_own_backward)[op](state)
    return dict(few=_plain_few, threshold_few=_plain_threshold, checkpoint=_plain_checkpoint,
                backward=_plain_backward)[op](state)


def work(case):
    """Inputs read once, outputs written once. Experts in use: the distinct
    ones of T * k random choices (the kept ones')."""
    c = case
    T, d, E, F, k = c["T"], c["d"], c["E"], c["d_ff"], c["k"]
    eb = 2 if c["dtype"] == "bf16" else 4
    A = min(T * k, E * _capacity(c))
    if c["op"] == "checkpoint":
        # Rows, their 8-bit values with scales, and back.
        share = 0.98 * T * k if _capacity(c) * E >= 1.5 * T * k else 0.9 * A
        return dict(bytes=share * F * (2 * eb + 2 * (1 + 1 / BLOCK)), flops=share * F * 4)
    router = d * E * 4 * (2 if c["noisy"] else 1) + (T * E * 4 if c["noisy"] else 0)
    if c["op"] == "backward":
        A = 0.95 * A
        weights = 2 * E * d * F * eb
        return dict(bytes=2 * weights + 2 * router + 3 * T * d * eb + A * F * (1 + 1 / BLOCK),
                    flops=8 * A * d * F)
    if c["op"] == "threshold_few":
        A = min(2.0 * T, T * k)
    active = E * (1 - (1 - min(1.0, A / T / E)) ** T)
    return dict(bytes=router + active * 2 * d * F * eb + 2 * T * d * eb,
                flops=A * 4 * d * F + 2 * T * d * E * (2 if c["noisy"] else 1))


# ----------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _exact_checkpoint(s)
    if case["op"] == "backward":
        return _exact_backward(s) if work(case)["flops"] < 6e12 else None
    return _exact_forward(s)


def _e4m3_values():
    """The 127 finite values from zero on, in order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _exact_checkpoint(s):
    """Nearest of the listed values, the even one on ties, by search."""
    table = _e4m3_values()
    mid = (table[1:] + table[:-1]) / 2
    out = torch.zeros_like(s["h"])
    F = out.shape[1]
    for lo in range(0, s["n"], 512):
        hi = min(s["n"], lo + 512)
        for a in range(0, F, BLOCK * 64):
            z = min(F, a + BLOCK * 64)
            h = s["h"][lo:hi, a:z].double()
            n = -(-(z - a) // BLOCK)
            top = torch.stack([h[:, i * BLOCK:(i + 1) * BLOCK].amax(1) for i in range(n)], 1)
            e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448)).clamp(min=LOW)
            e = torch.where(448 * torch.exp2(e - 1) >= top, (e - 1).clamp(min=LOW), e)
            e = torch.where(448 * torch.exp2(e) < top, e + 1, e)
            e = e.repeat_interleave(BLOCK, 1)[:, : z - a]
            up = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e
            q = (h / up).contiguous()
            i = torch.searchsorted(mid, q)                    # ties: the lower one
            at = mid[i.clamp(max=mid.numel() - 1)]
            i = torch.where((q == at) & (i % 2 == 1), i + 1, i).clamp(max=126)
            i = torch.where((h > 0) & (i == 0), 1, i)
            out[lo:hi, a:z] = (table[i] * up).to(out.dtype)
    return out.double()


def _exact_gate(s):
    """H and the full softmax, token by token's definition."""
    x = s["x"].to(torch.float64)
    H = torch.einsum("td,de->te", x, s["Wg"].to(torch.float64))
    if s.get("Wn") is not None:
        z = torch.einsum("td,de->te", x, s["Wn"].to(torch.float64))
        H = H + s["noise"].to(torch.float64) * torch.logaddexp(z, torch.zeros_like(z))
    return H


def _exact_forward(s):
    """Token by token, choice by choice."""
    c = s["case"]
    T, E, k, C = c["T"], c["E"], c["k"], _capacity(c)
    H = _exact_gate(s)
    P = torch.softmax(H, 1)
    few = c["op"] == "few"
    lists, taken = [], {}
    for t in range(T):
        if few:
            es = sorted(range(E), key=lambda e, h=H[t].tolist(): (-h[e], e))[:k]
            gs = [P[t, es[0]]] if c["mode"] == SWITCH else list(torch.softmax(H[t, es], 0))
            lists.append([(e, gs[j]) for j, e in enumerate(es)])
        else:
            es = torch.nonzero(P[t] > s["thr"].double())[:, 0].tolist()
            tot = P[t, es].sum()
            lists.append([(e, P[t, e] / tot) for e in es][:k])
    y = s["x"].double().clone()
    for t in range(T):
        for e, gt in lists[t]:
            taken[e] = taken.get(e, 0) + 1
            if few and taken[e] > C:
                continue
            taken.setdefault(("rows", e), []).append((t, gt))
    for e in range(E):
        rows = taken.get(("rows", e))
        if not rows:
            continue
        ts = torch.tensor([t for t, _ in rows], device="cuda")
        h = s["x"][ts].double() @ s["W1"][e].double()
        if s["b1"] is not None:
            h += s["b1"][e].double()
        o = h.relu() @ s["W2"][e].double()
        if s["b2"] is not None:
            o += s["b2"][e].double()
        y[ts] += torch.stack([g for _, g in rows])[:, None] * o
    gate = torch.tensor([[float(g) for _, g in r] + [0.0] * (k - len(r)) for r in lists],
                        dtype=torch.float64)
    return dict(y=y, idx=None, gate=gate, keep=None) if few else dict(y=y, idx=None, gate=gate)


def _exact_backward(s):
    """The experts one by one; the gate by automatic differentiation of
    sum <dy, y> and the balancing losses with the choices held fixed."""
    c = s["case"]
    T, d, E, F, k, C = c["T"], c["d"], c["E"], c["d_ff"], c["k"], _capacity(c)
    f64 = torch.float64
    idx = s["idx"].long()
    dy, x = s["dy"].to(f64), s["x"].to(f64)
    dx = dy.clone()
    dU_gate = torch.zeros((T, k), dtype=f64, device="cuda")
    out = dict(dW1=torch.zeros((E, d, F), dtype=f64, device="cuda"),
               db1=torch.zeros((E, F), dtype=f64, device="cuda"),
               dW2=torch.zeros((E, F, d), dtype=f64, device="cuda"),
               db2=torch.zeros((E, d), dtype=f64, device="cuda"))
    r0 = 0
    for e in range(E):
        at = torch.nonzero(idx == e)[:C]
        if not at.shape[0]:
            continue
        t, j = at[:, 0], at[:, 1]
        n = at.shape[0]
        e8 = s["hs"][r0:r0 + n].to(f64).repeat_interleave(BLOCK, 1)[:, :F] - 127
        h = s["h8"][r0:r0 + n].view(torch.float8_e4m3fn).to(f64) * torch.exp2(e8)
        r0 += n
        W1, W2 = s["W1"][e].to(f64), s["W2"][e].to(f64)
        U = h @ W2
        if s["b2"] is not None:
            U = U + s["b2"][e].to(f64)
        dU_gate[t, j] = (U * dy[t]).sum(1)
        up = s["gate"][t, j].to(f64)[:, None] * dy[t]
        dp = (up @ W2.t()) * (h > 0)
        out["dW2"][e], out["db2"][e] = h.t() @ up, up.sum(0)
        out["dW1"][e], out["db1"][e] = x[t].t() @ dp, dp.sum(0)
        dx.index_add_(0, t, dp @ W1.t())
    with torch.enable_grad():
        xg = x.clone().requires_grad_()
        Wg = s["Wg"].to(f64).requires_grad_()
        b = torch.zeros(E, dtype=f64, device="cuda", requires_grad=True)
        clean = xg @ Wg + b
        H, Wn = clean, None
        if s["Wn"] is not None:
            Wn = s["Wn"].to(f64).requires_grad_()
            sigma = torch.logaddexp(xg @ Wn, torch.zeros((), dtype=f64, device="cuda"))
            H = clean + s["noise"].to(f64) * sigma
        P = torch.softmax(H, 1)
        G = P.gather(1, idx) if c["mode"] == SWITCH else torch.softmax(H.gather(1, idx), 1)
        G.retain_grad()

        def cv2(v):
            return v.var(unbiased=False) / v.mean() ** 2
        loss = (G * dU_gate).sum()
        loss = loss + W_IMP * cv2(torch.zeros((T, E), dtype=f64, device="cuda")
                                  .scatter(1, idx, G).sum(0))
        f = torch.bincount(idx[:, 0], minlength=E).to(f64) / T
        loss = loss + W_AUX * 0.01 * E * (f * P.mean(0)).sum()
        if Wn is not None and k < E:
            best = H.detach().sort(dim=1, descending=True, stable=True)[1]
            inside = torch.zeros((T, E), dtype=torch.bool, device="cuda").scatter(1, idx, True)
            thr = torch.where(inside, H.gather(1, best[:, k:k + 1]),
                              H.gather(1, best[:, k - 1:k]))
            loss = loss + W_LOAD * cv2(torch.special.ndtr((clean - thr) / sigma).sum(0))
        loss.backward()
    return dict(dx=dx + xg.grad, dWg=Wg.grad, dWn=None if Wn is None else Wn.grad, dbias=b.grad,
                dgate=G.grad, **out)

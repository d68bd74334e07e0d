"""The gated experts on the GPU against the formulas in 64 bits
(tests/gated_reference.py, which also gives every element's bound)."""
import threading

import pytest
import torch

import gated_reference as R
from sparsely_gated_mixture_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(T, d, E, F, k, dt, seed=0, biases=True, skew=0.5, empty=()):
    """CPU tensors: tokens, choices that prefer some experts (none in `empty`),
    gates, weights of scale 1 / sqrt(fan_in), dy."""
    g = torch.Generator().manual_seed(seed)

    def normal(*s, std=1.0):
        return (torch.randn(s, generator=g) * std).to(dt)
    H = torch.randn((T, E), generator=g) + skew * torch.randn((E,), generator=g)
    for e in empty:
        H[:, e] = -100.0
    top, idx = torch.sort(H, dim=1, descending=True, stable=True)
    s = dict(x=normal(T, d), idx=idx[:, :k].to(torch.int32).contiguous(),
             gate=torch.softmax(top[:, :k], 1).contiguous(), W1=normal(E, d, F, std=d ** -0.5),
             W3=normal(E, d, F, std=d ** -0.5), W2=normal(E, F, d, std=F ** -0.5),
             b1=None, b3=None, b2=None, dy=normal(T, d))
    if biases:
        s.update(b1=normal(E, F, std=0.3), b3=normal(E, F, std=0.3), b2=normal(E, d, std=0.3))
    return s


def config(s, cf=2.0):
    T, d = s["x"].shape
    E, _, F = s["W1"].shape
    return B.config(T, d, E, F, s["idx"].shape[1], cf,
                    act_dtype=B.MOE_BF16 if s["x"].dtype == BF16 else B.MOE_F32)


def cap(cfg):
    return R.capacity(cfg.T, cfg.E, cfg.k, cfg.capacity_factor, cfg.min_capacity)


def dev(s):
    return {n: None if v is None else v.cuda() for n, v in s.items()}


def buf(n, fill=0xAB):
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


def run_forward(cfg, kind, g, keeps=True, y=None, ws=None, stream=None):
    T, k, F, dt = cfg.T, cfg.k, cfg.d_ff, g["x"].dtype
    o = dict(y=torch.empty_like(g["x"]) if y is None else y,
             pos=torch.empty((T, k), dtype=torch.int32, device="cuda"),
             keep=torch.empty((T, k), dtype=torch.uint8, device="cuda"), p1=None, p3=None)
    if keeps:
        o["p1"] = torch.full((T * k, F), 7.0, dtype=dt, device="cuda")
        o["p3"] = torch.full((T * k, F), 7.0, dtype=dt, device="cuda")
    ws = buf(B.moe_gated_workspace_size(cfg)) if ws is None else ws
    B.moe_experts_gated(cfg, kind, g["x"], g["idx"], g["gate"], g["W1"], g["b1"], g["W3"],
                        g["b3"], g["W2"], g["b2"], o["y"], ws, pre1=o["p1"], pre3=o["p3"],
                        pos=o["pos"], keep=o["keep"], stream=stream)
    o["ws"] = ws
    return o


def run_backward(cfg, kind, g, p1, p3, ws=None, stream=None, fill=float("nan")):
    o = {n: torch.full(g[n[1:]].shape, fill, dtype=g["x"].dtype, device="cuda")
         for n in ("dx", "dW1", "dW3", "dW2")}
    o["dgate"] = torch.full(g["gate"].shape, fill, device="cuda")
    for n in ("db1", "db3", "db2"):
        o[n] = None if g[n[1:]] is None else torch.full_like(g[n[1:]], fill)
    ws = buf(B.moe_gated_backward_workspace_size(cfg)) if ws is None else ws
    B.moe_experts_gated_backward(cfg, kind, g["x"], g["idx"], g["gate"], p1, p3, g["W1"], g["W3"],
                                 g["W2"], g["b2"], g["dy"], o["dx"], o["dgate"], o["dW1"],
                                 o["db1"], o["dW3"], o["db3"], o["dW2"], o["db2"], ws,
                                 stream=stream)
    o["ws"] = ws
    return o


def close(name, got, want, err):
    got = got.cpu().double()
    bad = ~((got - want).abs() <= err)
    assert not bool(bad.any()), (name, int(bad.sum()), float((got - want).abs().max()),
                                 float(err.max()))


def check_forward(cfg, kind, s, o, ref):
    st, det = B.moe_last_device_status(o["ws"])
    assert st == 0, (st, det)
    assert torch.equal(o["pos"].cpu(), ref["pos"]) and torch.equal(o["keep"].cpu(), ref["keep"])
    close("y", o["y"], ref["y"], ref["y_err"])
    if o["p1"] is not None:
        for q, n in enumerate(("p1", "p3")):
            r = ref["rows"]
            close(n, o[n][:r], ref["pre"][q][:r], ref["pre_err"][q][:r])
            assert bool((o[n][r:] == 7.0).all()), "rows past the last kept one"


def reference(cfg, kind, s):
    return R.forward(kind, s["x"], s["idx"], s["gate"], s["W1"], s["b1"], s["W3"], s["b3"],
                     s["W2"], s["b2"], cap(cfg))


def check_backward(cfg, kind, s, p1, p3, o):
    st, det = B.moe_last_device_status(o["ws"])
    assert st == 0, (st, det)
    want, err = R.backward(kind, s["x"], s["idx"], s["gate"], p1, p3, s["W1"], s["W3"], s["W2"],
                           s["b2"], s["dy"], cap(cfg))
    for n in ("dx", "dgate", "dW1", "dW3", "dW2", "db1", "db3", "db2"):
        if o[n] is not None:
            close(n, o[n], want[n], err[n])


# T, d, E, F, k, cf, type, biases: one token; a few; odd widths; widths of 8 and
# 64; tight capacities; many experts with few rows; rows around the tiles of
# 32, 128 and 256; one expert.
SHAPES = [
    (1, 64, 4, 128, 2, 2.0, BF16, True), (1, 512, 16, 1024, 4, 2.0, BF16, False),
    (1, 7, 2, 5, 1, 1.0, F32, True), (3, 130, 6, 234, 3, 1.0, F32, True),
    (2, 256, 8, 512, 1, 8.0, BF16, True), (33, 192, 5, 320, 2, 5.0, BF16, True),
    (64, 512, 8, 768, 2, 4.0, BF16, True), (64, 128, 200, 192, 6, 200.0, BF16, False),
    (65, 64, 3, 64, 2, 1.1, BF16, True), (200, 72, 4, 136, 3, 1.25, BF16, True),
    (517, 130, 6, 234, 3, 1.1, F32, True), (517, 130, 6, 234, 3, 1.1, BF16, True),
    (300, 320, 2, 448, 1, 1.3, BF16, False), (600, 256, 4, 512, 2, 2.0, BF16, True),
    (1000, 64, 130, 128, 4, 1.0, BF16, True), (700, 1024, 3, 256, 1, 3.0, BF16, True),
    (520, 64, 1, 192, 1, 1.0, F32, False), (257, 2, 3, 2, 2, 2.0, F32, True),
    (1500, 512, 2, 1280, 2, 1.0, BF16, True), (900, 200, 3, 264, 2, 2.0, F32, True),
]


@pytest.mark.parametrize("kind", [R.SILU, R.GELU, R.RELU])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda v: "-".join(map(str, v[:6])) + str(v[6])[6:])
def test_forward_and_backward(shape, kind):
    T, d, E, F, k, cf, dt, biases = shape
    s = inputs(T, d, E, F, k, dt, seed=T + kind, biases=biases)
    cfg, g = config(s, cf), dev(s)
    ref = reference(cfg, kind, s)
    o = run_forward(cfg, kind, g)
    check_forward(cfg, kind, s, o, ref)
    plain = run_forward(cfg, kind, g, keeps=False)
    assert torch.equal(plain["y"], o["y"])
    check_backward(cfg, kind, s, o["p1"], o["p3"], run_backward(cfg, kind, g, o["p1"], o["p3"]))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_thousand_experts(dt):
    """1024 experts, most of them with a row or two, some with none."""
    s = inputs(900, 64, 1024, 64, 2, dt, skew=1.0)
    cfg, g = config(s, 64.0), dev(s)
    o = run_forward(cfg, R.SILU, g)
    check_forward(cfg, R.SILU, s, o, reference(cfg, R.SILU, s))
    check_backward(cfg, R.SILU, s, o["p1"], o["p3"],
                   run_backward(cfg, R.SILU, g, o["p1"], o["p3"]))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("d,F,skew", [(72, 100, 0.0), (33, 1, 2.0), (181, 300, 1.0)])
def test_weight_gradients_by_slices_of_rows(dt, d, F, skew):
    """Many rows through few small experts on the CUDA cores: the rows' sums in slices,
    some of them empty where the experts' loads differ."""
    s = inputs(2300, d, 4, F, 2, dt, skew=skew)
    cfg, g = config(s, 4.0), dev(s)
    o = run_forward(cfg, R.GELU, g)
    check_forward(cfg, R.GELU, s, o, reference(cfg, R.GELU, s))
    a = run_backward(cfg, R.GELU, g, o["p1"], o["p3"])
    check_backward(cfg, R.GELU, s, o["p1"], o["p3"], a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    ws = a["ws"].clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        b = run_backward(cfg, R.GELU, g, o["p1"], o["p3"], ws=ws)
    for _ in range(2):
        ws.fill_(255)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in ("dx", "dgate", "dW1", "dW3", "dW2"))
    g["x"][0, 0] = float("nan")  # read by dW1 and dW3 alone: pre1 and pre3 are given
    c = run_backward(cfg, R.GELU, g, o["p1"], o["p3"])
    torch.cuda.synchronize()
    assert B.moe_last_device_status(c["ws"])[0] == 4


# Row counts around the tiles of 128 (a CTA) and 256 (a pair of CTAs).
VARIANT_SHAPES = [(300, 128, 3, 320, 1, 3.0), (1100, 192, 4, 256, 1, 4.0),
                  (700, 256, 2, 576, 2, 2.0)]


@pytest.mark.parametrize("variant", ["single", "pair"])
@pytest.mark.parametrize("shape", VARIANT_SHAPES, ids=lambda v: "-".join(map(str, v)))
def test_tensor_core_variants(shape, variant, monkeypatch):
    """The one-CTA and the CTA-pair kernels, each forced; the pairs also with
    every tile's K backwards."""
    T, d, E, F, k, cf = shape
    monkeypatch.setenv("MOE_FFN_TC_VARIANT", variant)
    monkeypatch.setenv("MOE_BWD_TC_VARIANT", variant)
    s = inputs(T, d, E, F, k, BF16, seed=T)
    cfg, g = config(s, cf), dev(s)
    ref = reference(cfg, R.SILU, s)
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    for snake in ("1", "all") if variant == "pair" else ("1",):
        monkeypatch.setenv("MOE_FFN_SNAKE", snake)
        o = run_forward(cfg, R.SILU, g)
        check_forward(cfg, R.SILU, s, o, ref)
        check_backward(cfg, R.SILU, s, o["p1"], o["p3"],
                       run_backward(cfg, R.SILU, g, o["p1"], o["p3"]))
    check_forward(cfg, R.SILU, s, run_fp8(cfg, R.SILU, g, w8), reference8(cfg, R.SILU, s, w8))


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("dt,d,F", [(BF16, 128, 192), (F32, 66, 70)])
def test_empty_experts_repeats_and_bad_indexes(T, dt, d, F):
    """Experts without rows get zero gradients; an expert twice in a token's
    choices counts twice; an index that is no expert is recorded and dropped."""
    s = inputs(T, d, 6, F, 3, dt, empty=(0, 5))
    s["idx"][T // 2] = torch.tensor([2, 2, 3], dtype=torch.int32)
    cfg, g = config(s, 6.0), dev(s)
    o = run_forward(cfg, R.SILU, g)
    check_forward(cfg, R.SILU, s, o, reference(cfg, R.SILU, s))
    b = run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
    check_backward(cfg, R.SILU, s, o["p1"], o["p3"], b)
    for n in ("dW1", "dW3", "dW2", "db1", "db3", "db2"):
        assert not bool(b[n][0].any()) and not bool(b[n][5].any()), n
    s["idx"][0] = torch.tensor([6, -1, 3], dtype=torch.int32)
    g = dev(s)
    o = run_forward(cfg, R.SILU, g)
    assert B.moe_last_device_status(o["ws"])[0] == 6
    check_forward(cfg, R.SILU, s, o, reference(cfg, R.SILU, s))
    b = run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
    assert B.moe_last_device_status(b["ws"])[0] == 6
    check_backward(cfg, R.SILU, s, o["p1"], o["p3"], b)


@pytest.mark.parametrize("T", [1, 30, 500])
def test_nothing_kept_by_choice(T):
    """Every choice is no expert: y is x, dx is dy, the gradients are zero."""
    s = inputs(T, 64, 4, 128, 2, BF16)
    s["idx"].fill_(4)
    cfg, g = config(s), dev(s)
    o = run_forward(cfg, R.GELU, g)
    assert torch.equal(o["y"].cpu(), s["x"]) and not bool(o["keep"].any())
    assert bool((o["p1"] == 7.0).all())
    b = run_backward(cfg, R.GELU, g, o["p1"], o["p3"])
    assert torch.equal(b["dx"].cpu(), s["dy"])
    for n in ("dgate", "dW1", "dW3", "dW2", "db1", "db3", "db2"):
        assert not bool(b[n].any()), n


@pytest.mark.parametrize("T", [1, 20, 400])
@pytest.mark.parametrize("dt,d,F", [(BF16, 128, 256), (F32, 33, 65)])
def test_y_may_be_x(T, dt, d, F):
    s = inputs(T, d, 4, F, 2, dt)
    cfg, g = config(s), dev(s)
    o = run_forward(cfg, R.SILU, g)
    g2 = dev(s)
    assert torch.equal(run_forward(cfg, R.SILU, g2, y=g2["x"])["y"], o["y"])


@pytest.mark.parametrize("T", [1, 24, 400])
@pytest.mark.parametrize("dt,d,F", [(BF16, 128, 256), (BF16, 36, 50), (F32, 48, 64)])
def test_non_finite(T, dt, d, F):
    """A NaN or an Inf in a token reaches that token's y and no other, and is
    recorded; large negative pre-activations stay finite."""
    s = inputs(T, d, 4, F, 2, dt, biases=False)
    cfg, g = config(s, 4.0), dev(s)
    ref = run_forward(cfg, R.SILU, g)
    s["x"][T // 2, 3] = float("nan")
    o = run_forward(cfg, R.SILU, dev(s))
    assert B.moe_last_device_status(o["ws"])[0] == 4
    same = torch.arange(T) != T // 2
    assert torch.equal(o["y"].cpu()[same], ref["y"].cpu()[same])
    assert bool(torch.isnan(o["y"][T // 2]).all())
    s["x"][T // 2, 3] = 0.0
    for big in (-3e4, 3e4):
        s["b1"], s["b3"], s["b2"] = (torch.full(v, big if i == 0 else 1.0, dtype=dt)
                                     for i, v in enumerate(((4, F), (4, F), (4, d))))
        g = dev(s)
        for kind in (R.SILU, R.GELU, R.RELU):
            o = run_forward(cfg, kind, g)
            check_forward(cfg, kind, s, o, reference(cfg, kind, s))
            check_backward(cfg, kind, s, o["p1"], o["p3"],
                           run_backward(cfg, kind, g, o["p1"], o["p3"]))


@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("dt,d,F", [(BF16, 128, 256), (F32, 34, 66)])
def test_streams_graphs_and_repeats(T, dt, d, F):
    """The same bits from run to run, on other streams, from two host threads
    at once with workspaces of their own, and from a replayed graph of a forward and
    a backward that share no workspace with the eager calls between."""
    s = inputs(T, d, 5, F, 2, dt)
    cfg, g = config(s), dev(s)
    o = run_forward(cfg, R.SILU, g)
    b = run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
    names = ("dx", "dgate", "dW1", "dW3", "dW2", "db1", "db3", "db2")

    def same(o2, b2):
        assert torch.equal(o2["y"], o["y"])
        for n in names:
            assert torch.equal(b2[n], b[n]), n
    torch.cuda.synchronize()
    results = {}

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(3):
                o2 = run_forward(cfg, R.SILU, g, stream=st)
                b2 = run_backward(cfg, R.SILU, g, o2["p1"], o2["p3"], stream=st)
            st.synchronize()
        results[i] = (o2, b2)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(results) == 2
    for i in range(2):
        same(*results[i])
    ws, wb = o["ws"].clone(), b["ws"].clone()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        o3 = run_forward(cfg, R.SILU, g, ws=ws)
        b3 = run_backward(cfg, R.SILU, g, o3["p1"], o3["p3"], ws=wb)
    for _ in range(2):
        g2 = dev(inputs(T, d, 5, F, 2, dt, seed=9))
        run_forward(cfg, R.SILU, g2)
        for n in names:
            b3[n].fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        same(o3, b3)


def test_gradients_against_differences():
    """Directional differences of the forward itself, fp32."""
    s = inputs(40, 24, 4, 36, 2, F32, seed=5)
    cfg, g = config(s, 4.0), dev(s)
    for kind in (R.SILU, R.GELU):
        o = run_forward(cfg, kind, g)
        b = run_backward(cfg, kind, g, o["p1"], o["p3"])
        dy = g["dy"].double()
        for n in ("x", "gate", "W1", "W3", "W2", "b1", "b3", "b2"):
            v = torch.randn(g[n].shape, generator=torch.Generator().manual_seed(2)).cuda()
            eps = 2.0 ** -9
            at = {}
            for sign in (1, -1):
                h = dict(g)
                h[n] = g[n] + sign * eps * v
                at[sign] = run_forward(cfg, kind, h)["y"].double()
            diff = float(((at[1] - at[-1]) * dy).sum() / (2 * eps))
            got = float((b["d" + n].double() * v.double()).sum())
            # Rounding: |y| 2^-22 over 2 eps a value, 960 values of random sign; curvature:
            # eps^2 / 6 of a third derivative of the order of the gradient's own size.
            scale = float((b["d" + n].double().abs() * v.double().abs()).sum())
            assert abs(diff - got) < 2e-4 * scale + 0.02, (kind, n, diff, got)


# ----------------------------------------------------------------------------- 8 bits
def quantise(g, name, dt):
    W = g[name]
    E, K, N = W.shape
    n8, ns = B.moe_weights_fp8_size(E, K, N)
    q, sc, ws = buf(n8), buf(ns), buf(256, 0)
    B.moe_weights_fp8(E, K, N, B.MOE_BF16 if dt == BF16 else B.MOE_F32, W, q, sc, ws)
    assert B.moe_last_device_status(ws)[0] == 0
    return q.view(E, N, -1), sc.view(E, R.blocks(N), R.blocks(K))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (2, 128, 128), (3, 130, 70), (1, 127, 257),
                                   (2, 513, 384), (5, 331, 77)])
def test_weights_fp8(E, K, N, dt):
    g = torch.Generator().manual_seed(E * K + N)
    W = torch.randn((E, K, N), generator=g) * torch.exp2(
        torch.randint(-30, 30, (E, 1, N), generator=g).float())
    W[0, 0, 0] = 0.0
    if K > 2:
        W[0, 2] = 0.0
    W = W.to(dt)
    q, sc = quantise(dict(W=W.cuda()), "W", dt)
    qr, sr = R.weights8(W)
    assert torch.equal(sc.cpu(), sr)
    # Zeros of either sign are the same value.
    z = (qr & 127) == 0
    assert torch.equal(torch.where(z, 0, q.cpu()), torch.where(z, 0, qr))
    assert bool(((q.cpu()[z] & 127) == 0).all())


def test_weights_fp8_borders():
    """Ties, the largest of a block at and just over 448 * 2^e, the smallest
    numbers, a block of zeros, an Inf and a NaN."""
    rows = [448.0, 449.0, 447.99997, 3.4e38, 1e-45, 2.0 ** -120, 0.0, 17.0, 19.0, -17.0]
    W = torch.zeros((len(rows), 3, 2))
    for i, v in enumerate(rows):
        W[i, 0, 0] = v
        W[i, 1, 0] = -v / 3
        W[i, 2, 1] = v * 2.0 ** -10
    q, sc = quantise(dict(W=W.cuda()), "W", F32)
    qr, sr = R.weights8(W)
    assert torch.equal(sc.cpu(), sr) and torch.equal(q.cpu() & 127, qr & 127)
    for bad in (float("inf"), float("-inf"), float("nan")):
        W = torch.ones((2, 130, 5), device="cuda")
        W[1, 129, 3] = bad
        n8, ns = B.moe_weights_fp8_size(2, 130, 5)
        q, sc, ws = buf(n8), buf(ns), buf(256, 0)
        B.moe_weights_fp8(2, 130, 5, B.MOE_F32, W, q, sc, ws)
        assert B.moe_last_device_status(ws) == (4, 3)
        assert sc.tolist() == [119, 119, 119, 255]


def run_fp8(cfg, kind, g, w8, ws=None, stream=None, y=None):
    o = dict(y=torch.empty_like(g["x"]) if y is None else y, p1=None,
             pos=torch.empty((cfg.T, cfg.k), dtype=torch.int32, device="cuda"),
             keep=torch.empty((cfg.T, cfg.k), dtype=torch.uint8, device="cuda"))
    ws = buf(B.moe_gated_fp8_workspace_size(cfg)) if ws is None else ws
    (q1, s1), (q3, s3), (q2, s2) = w8
    B.moe_experts_gated_fp8(cfg, kind, g["x"], g["idx"], g["gate"], q1, s1, g["b1"], q3, s3,
                            g["b3"], q2, s2, g["b2"], o["y"], ws, pos=o["pos"], keep=o["keep"],
                            stream=stream)
    o["ws"] = ws
    return o


def reference8(cfg, kind, s, w8):
    q, sc = zip(*w8)
    return R.forward(kind, s["x"], s["idx"], s["gate"], q[0], s["b1"], q[1], s["b3"], q[2],
                     s["b2"], cap(cfg), weights8=sc)


FP8_SHAPES = [
    (1, 128, 4, 256, 2, 2.0, True), (1, 512, 16, 1024, 4, 2.0, False), (2, 7, 3, 5, 1, 1.0, True),
    (33, 200, 5, 330, 2, 5.0, True), (64, 512, 8, 768, 2, 4.0, True),
    (64, 130, 150, 190, 6, 150.0, False), (65, 64, 3, 64, 2, 1.1, True),
    (517, 130, 6, 234, 3, 1.1, True), (600, 256, 4, 512, 2, 2.0, True),
    (1000, 64, 130, 128, 4, 1.0, True), (700, 1024, 3, 256, 1, 3.0, True),
    (300, 384, 1, 640, 1, 1.0, False), (1500, 512, 2, 1280, 2, 1.0, True),
]


@pytest.mark.parametrize("kind", [R.SILU, R.GELU, R.RELU])
@pytest.mark.parametrize("shape", FP8_SHAPES, ids=lambda v: "-".join(map(str, v[:6])))
def test_fp8_layer(shape, kind):
    T, d, E, F, k, cf, biases = shape
    s = inputs(T, d, E, F, k, BF16, seed=T + kind, biases=biases)
    # Rows and blocks of very different sizes.
    s["x"] *= torch.exp2(torch.arange(T) % 7 - 3).to(BF16)[:, None]
    cfg, g = config(s, cf), dev(s)
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    o = run_fp8(cfg, kind, g, w8)
    check_forward(cfg, kind, s, o, reference8(cfg, kind, s, w8))
    y2 = dev(s)
    assert torch.equal(run_fp8(cfg, kind, y2, w8, y=y2["x"])["y"], o["y"])


@pytest.mark.parametrize("T", [1, 24, 400])
def test_fp8_non_finite_and_bad_indexes(T):
    s = inputs(T, 200, 4, 256, 2, BF16)
    cfg, g = config(s, 4.0), dev(s)
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    ref = run_fp8(cfg, R.SILU, g, w8)
    s["x"][T // 2, 3] = float("inf")
    s["idx"][0, 1] = 9
    o = run_fp8(cfg, R.SILU, dev(s), w8)
    assert B.moe_last_device_status(o["ws"])[0] in (4, 6)
    assert bool(torch.isnan(o["y"][T // 2]).all())
    same = torch.arange(T) != T // 2
    same[0] = False
    assert torch.equal(o["y"].cpu()[same], ref["y"].cpu()[same])
    assert int(o["pos"][0, 1]) == -1 and int(o["keep"][0, 1]) == 0


@pytest.mark.parametrize("T", [1, 24, 400])
def test_fp8_non_finite_weight(T):
    """An Inf in a weight makes its expert's outputs NaN, and no other's."""
    s = inputs(T, 200, 4, 256, 1, BF16)
    s["idx"][:, 0] = torch.arange(T) % 4
    cfg, g = config(s, 4.0), dev(s)
    good = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    ref = run_fp8(cfg, R.SILU, g, good)
    for w in range(3):
        W = g[("W1", "W3", "W2")[w]].clone()
        W[0, 130, 7] = float("inf")
        E, K, N = W.shape
        n8, ns = B.moe_weights_fp8_size(E, K, N)
        q, sc, ws = buf(n8), buf(ns), buf(256, 0)
        B.moe_weights_fp8(E, K, N, B.MOE_BF16, W, q, sc, ws)
        assert B.moe_last_device_status(ws)[0] == 4
        w8 = list(good)
        w8[w] = (q.view(E, N, -1), sc.view(E, R.blocks(N), R.blocks(K)))
        o = run_fp8(cfg, R.SILU, g, w8)
        assert B.moe_last_device_status(o["ws"])[0] == 4
        first = s["idx"][:, 0] == 0
        assert torch.equal(o["y"].cpu()[~first], ref["y"].cpu()[~first])
        assert bool(torch.isnan(o["y"].cpu()[first]).any(1).all())


@pytest.mark.parametrize("T", [2, 300])
def test_fp8_streams_and_graphs(T):
    s = inputs(T, 256, 5, 384, 2, BF16)
    cfg, g = config(s), dev(s)
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    o = run_fp8(cfg, R.GELU, g, w8)
    ws = o["ws"].clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2 = run_fp8(cfg, R.GELU, g, w8, stream=st)
    st.synchronize()
    assert torch.equal(o2["y"], o["y"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        o3 = run_fp8(cfg, R.GELU, g, w8, ws=ws)
    for _ in range(2):
        run_fp8(cfg, R.GELU, dev(inputs(T, 256, 5, 384, 2, BF16, seed=4)), w8)
        o3["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o3["y"], o["y"])


# ----------------------------------------------------------------------------- a run of them
def test_a_training_step_and_serving():
    """Router, experts, backward through both, one step of gradient descent, and
    the layer in 8 bits: the loss's gradients against 64 bits, the step's y
    against the formulas, the 8-bit y against its own."""
    T, d, E, F, k = 300, 128, 6, 192, 2
    s = inputs(T, d, E, F, k, BF16, seed=3)
    cfg, g = config(s, 2.0), dev(s)
    Wg = (torch.randn((d, E), generator=torch.Generator().manual_seed(1)) * d ** -0.5).cuda()
    wsl = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    bws = torch.zeros(B.moe_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    thr = torch.empty((T, 2), device="cuda")
    B.moe_gate(cfg, g["x"], Wg, None, None, None, g["idx"], g["gate"], thr, wsl)
    s["idx"], s["gate"] = g["idx"].cpu(), g["gate"].cpu()
    o = run_forward(cfg, R.SILU, g)
    check_forward(cfg, R.SILU, s, o, reference(cfg, R.SILU, s))
    b = run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
    check_backward(cfg, R.SILU, s, o["p1"], o["p3"], b)
    dWg = torch.empty_like(Wg)
    dxg = torch.empty((T, d), device="cuda")
    B.moe_gate_backward(cfg, g["x"], Wg, None, None, g["idx"], g["gate"], b["dgate"], 0.0, 0.0, dWg,
                        None, None, dxg, wsl, bws)
    # dL/dWg through the softmax of the chosen logits.
    gate, dg = s["gate"].double(), b["dgate"].cpu().double()
    dc = gate * (dg - (gate * dg).sum(1, keepdim=True))
    full = torch.zeros((T, E), dtype=torch.float64).scatter_add_(1, s["idx"].long(), dc)
    x = s["x"].double()
    want = x.t() @ full
    tol = 32 * 2.0 ** -23 * (x.abs().t() @ full.abs()) + T * 2.0 ** -23 * (
        x.abs().t() @ (gate * (dg.abs() + (gate * dg.abs()).sum(1, keepdim=True))).new_zeros(
            (T, E)).scatter_add_(1, s["idx"].long(), gate * (dg.abs() + (gate * dg.abs()).sum(
                1, keepdim=True))))
    close("dWg", dWg, want, tol)
    for n in ("W1", "W3", "W2", "b1", "b3", "b2"):
        g[n] -= 0.05 * b["d" + n]
        s[n] = g[n].cpu()
    o = run_forward(cfg, R.SILU, g, keeps=False)
    check_forward(cfg, R.SILU, s, o, reference(cfg, R.SILU, s))
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    o8 = run_fp8(cfg, R.SILU, g, w8)
    check_forward(cfg, R.SILU, s, o8, reference8(cfg, R.SILU, s, w8))


# ----------------------------------------------------------------------------- borders
def sampled(s, at):
    """The same call on some of its tokens (weights shared)."""
    return {n: v if v is None or n not in ("x", "idx", "gate", "dy") else v[at].contiguous()
            for n, v in s.items()}


@pytest.mark.parametrize("T,E,k,cf", [(8192, 16, 4, 0.9), (8193, 16, 4, 0.9), (10000, 1024, 4, 1.0),
                                      (8192, 1024, 4, 0.7), (2048, 3, 2, 0.5)])
def test_routing_of_long_batches(T, E, k, cf):
    """pos and keep on both sides of the one-launch routing (32768 choices), under
    tight capacities; y for some tokens."""
    s = inputs(T, 64, E, 64, k, BF16, seed=T + E, skew=1.0)
    s["idx"][5] = s["idx"][5, 0]  # one expert in all of a token's choices
    s["idx"][7, 0] = E
    cfg, g = config(s, cf), dev(s)
    pos, keep, _ = R.slots(s["idx"], E, cap(cfg))
    o = run_forward(cfg, R.SILU, g, keeps=False)
    assert B.moe_last_device_status(o["ws"])[0] == 6
    assert torch.equal(o["pos"].cpu(), pos) and torch.equal(o["keep"].cpu(), keep)
    at = [t for t in (0, 5, 6, T // 2, T - 1) if bool(keep[t].all())] + [0]
    sub = sampled(s, at)
    sub["gate"] = sub["gate"] * keep[at]
    want = R.forward(R.SILU, sub["x"], sub["idx"], sub["gate"], s["W1"], s["b1"], s["W3"], s["b3"],
                     s["W2"], s["b2"], T * k)
    close("y", o["y"][at], want["y"], want["y_err"])


@pytest.mark.parametrize("T,k,E,min_cap,fp8", [
    (64, 8, 40, 1, False), (64, 8, 40, 1, True),    # 512 choices
    (57, 9, 64, 1, False), (57, 9, 64, 1, True),    # 513
    (64, 2, 2, 1, False), (64, 2, 2, 1, True),      # 64 rows an expert
    (40, 2, 3, 100, False), (40, 2, 3, 100, True),  # more slots than tokens
    (17, 16, 1024, 1, False), (17, 16, 1024, 1, True), (31, 1, 1, 1, False), (48, 3, 7, 1, True)])
def test_few_rows_borders(T, k, E, min_cap, fp8):
    s = inputs(T, 128, E, 192, k, BF16, seed=T * k)
    s["idx"][0] = s["idx"][0, 0]  # one expert in all of a token's choices
    cfg, g = config(s, float(E)), dev(s)
    cfg.min_capacity = min_cap
    if fp8:
        w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
        check_forward(cfg, R.SILU, s, run_fp8(cfg, R.SILU, g, w8), reference8(cfg, R.SILU, s, w8))
    else:
        o = run_forward(cfg, R.SILU, g)
        check_forward(cfg, R.SILU, s, o, reference(cfg, R.SILU, s))


@pytest.mark.parametrize("dt,T,d,F,E,k,min_cap", [
    (F32, 1, 3, 2000, 5, 2, 1), (F32, 1, 2000, 3, 5, 2, 1), (BF16, 3, 770, 1030, 24, 1, 1),
    (F32, 17, 514, 1025, 7, 4, 1), (F32, 64, 36, 40, 2, 2, 1), (BF16, 40, 72, 100, 3, 2, 100),
    (F32, 64, 20, 24, 600, 8, 1), (F32, 57, 20, 24, 64, 9, 1)])
def test_few_rows_on_cuda_cores(dt, T, d, F, E, k, min_cap):
    s = inputs(T, d, E, F, k, dt, seed=T + d)
    s["idx"][0] = s["idx"][0, 0]
    cfg, g = config(s, float(E)), dev(s)
    cfg.min_capacity = min_cap
    for kind in (R.SILU, R.GELU, R.RELU):
        o = run_forward(cfg, kind, g)
        check_forward(cfg, kind, s, o, reference(cfg, kind, s))


@pytest.mark.parametrize("dt,T,d,F", [(BF16, 160000, 64, 14336), (F32, 80000, 9, 30001)])
def test_rows_past_32_bits(dt, T, d, F):
    """Hidden rows of more than 2^31 values: y, pre-activations and gradients of
    tokens on both sides, forward, backward and in 8 bits."""
    s = inputs(T, d, 2, F, 1, dt, biases=False)
    cfg, g = config(s, 2.0), dev(s)
    order = torch.argsort(s["idx"][:, 0], stable=True)  # the packed rows' tokens
    at = torch.cat([order[:5], order[(1 << 31) // F - 2:(1 << 31) // F + 3], order[-20:]])
    sub = sampled(s, at)
    want = R.forward(R.SILU, sub["x"], sub["idx"], sub["gate"], s["W1"], None, s["W3"], None,
                     s["W2"], None, T)
    o = run_forward(cfg, R.SILU, g)
    assert B.moe_last_device_status(o["ws"])[0] == 0
    close("y", o["y"][at.cuda()], want["y"], want["y_err"])
    rows = torch.empty(T, dtype=torch.long)
    rows[order] = torch.arange(T)
    by = torch.argsort(sub["idx"][:, 0], stable=True)  # the sample's packed order
    for q, n in enumerate(("p1", "p3")):
        close(n, o[n][rows[at[by]].cuda()], want["pre"][q], want["pre_err"][q])
    # Only the sample's tokens have a gradient, so the weights' come from them.
    dy = torch.zeros_like(s["dy"])
    dy[at] = s["dy"][at]
    g["dy"] = dy.cuda()
    del o["ws"]
    b = run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
    assert B.moe_last_device_status(b["ws"])[0] == 0
    p = [o[n][rows[at[by]].cuda()].cpu() for n in ("p1", "p3")]
    wb, eb = R.backward(R.SILU, sub["x"], sub["idx"], sub["gate"], p[0], p[1], s["W1"], s["W3"],
                        s["W2"], None, sub["dy"], T)
    for n in ("dx", "dgate"):
        close(n, b[n][at.cuda()], wb[n], eb[n])
    for n in ("dW1", "dW3", "dW2"):
        close(n, b[n], wb[n], eb[n])
    del b, o
    if dt == BF16:
        w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
        o = run_fp8(cfg, R.SILU, g, w8)
        q, sc = zip(*w8)
        want = R.forward(R.SILU, sub["x"], sub["idx"], sub["gate"], q[0], None, q[1], None, q[2],
                         None, T, weights8=sc)
        close("y8", o["y"][at.cuda()], want["y"], want["y_err"])


@pytest.mark.parametrize("T", [3, 600])
def test_weights_past_32_bits(T):
    """Weights of more than 2^31 values: the last experts, in bf16 and 8 bits."""
    E, d, F, k = 1024, 512, 4608, 2
    gen = torch.Generator("cuda").manual_seed(T)

    def normal(*shape, std):
        return torch.randn(shape, generator=gen, device="cuda", dtype=BF16).mul_(std)
    s = inputs(T, d, 8, 64, k, BF16, biases=False)
    s["idx"] = 1016 + s["idx"]
    s["idx"][0, 0] = 0
    g = dict(x=s["x"].cuda(), idx=s["idx"].cuda(), gate=s["gate"].cuda(), b1=None, b3=None,
             b2=None, W1=normal(E, d, F, std=d ** -0.5), W3=normal(E, d, F, std=d ** -0.5),
             W2=normal(E, F, d, std=F ** -0.5))
    cfg = B.config(T, d, E, F, k, float(E))
    at = list(range(0, T, max(1, T // 5)))
    # The experts in use, renumbered, for the reference.
    used = sorted(set(s["idx"].flatten().tolist()))
    idx = torch.tensor([[used.index(e) for e in r] for r in s["idx"].tolist()], dtype=torch.int32)
    few = {n: g[n][used].cpu() for n in ("W1", "W3", "W2")}
    o = run_forward(cfg, R.SILU, g, keeps=False)
    want = R.forward(R.SILU, s["x"][at], idx[at], s["gate"][at], few["W1"], None, few["W3"], None,
                     few["W2"], None, T)
    close("y", o["y"][at], want["y"], want["y_err"])
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    o = run_fp8(cfg, R.SILU, g, w8)
    q = [v[used] for v, _ in w8]
    sc = [v[used] for _, v in w8]
    want = R.forward(R.SILU, s["x"][at], idx[at], s["gate"][at], q[0], None, q[1], None, q[2],
                     None, T, weights8=sc)
    close("y8", o["y"][at], want["y"], want["y_err"])


@pytest.mark.parametrize("T", [3, 700])
def test_waits_that_run_out(T, monkeypatch):
    """With no time to wait, the kernels report MOE_ERR_TIMEOUT and end; the next
    call on the same workspace is right."""
    s = inputs(T, 512, 4, 768, 2, BF16)
    cfg, g = config(s, 4.0), dev(s)
    w8 = [quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    good = run_forward(cfg, R.SILU, g)
    back = run_backward(cfg, R.SILU, g, good["p1"], good["p3"])
    good8 = run_fp8(cfg, R.SILU, g, w8)
    monkeypatch.setenv("MOE_WAIT_LIMIT_NS", "0")
    codes = []
    for call, ws in ((lambda w: run_forward(cfg, R.SILU, g, ws=w), good["ws"]),
                     (lambda w: run_backward(cfg, R.SILU, g, good["p1"], good["p3"], ws=w),
                      back["ws"]),
                     (lambda w: run_fp8(cfg, R.SILU, g, w8, ws=w), good8["ws"])):
        call(ws)
        codes.append(B.moe_last_device_status(ws)[0])
    assert codes[0] == 5 and codes[1] == 5 and codes[2] == 5, codes
    monkeypatch.delenv("MOE_WAIT_LIMIT_NS")
    o = run_forward(cfg, R.SILU, g, ws=good["ws"])
    assert torch.equal(o["y"], good["y"])
    b = run_backward(cfg, R.SILU, g, good["p1"], good["p3"], ws=back["ws"])
    for n in ("dx", "dgate", "dW1", "dW3", "dW2", "db1", "db3", "db2"):
        assert torch.equal(b[n], back[n]), n
    assert torch.equal(run_fp8(cfg, R.SILU, g, w8, ws=good8["ws"])["y"], good8["y"])

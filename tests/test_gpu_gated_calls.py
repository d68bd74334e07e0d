"""Calls of the gated experts that the documentation allows: arguments left out,
first calls of a thread and of a process under capture, the borders of k, of the
capacity and of the widths."""
import os
import subprocess
import sys

import pytest
import torch

import gated_reference as R
import test_gpu_gated as G
from sparsely_gated_mixture_gb300 import binding as B
from test_gpu_threads import on_new_thread

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
GRADS = ("dx", "dgate", "dW1", "dW3", "dW2", "db1", "db3", "db2")

# Few rows and many, on the tensor cores and on the CUDA cores.
FORMS = [(3, BF16, 128, 256), (400, BF16, 128, 256), (3, F32, 34, 66), (400, F32, 34, 66),
         (3, BF16, 36, 50), (400, BF16, 36, 50)]


@pytest.mark.parametrize("T,dt,d,F", FORMS)
def test_arguments_left_out(T, dt, d, F):
    """Without pos and keep the same bits; each bias alone as with zeros in the
    others' places; each bias gradient alone has the bits that it has with the others."""
    s = G.inputs(T, d, 4, F, 2, dt, seed=T)
    cfg, g = G.config(s, 1.25), G.dev(s)
    o = G.run_forward(cfg, R.GELU, g)
    y, ws = torch.empty_like(g["x"]), G.buf(B.moe_gated_workspace_size(cfg))
    B.moe_experts_gated(cfg, R.GELU, g["x"], g["idx"], g["gate"], g["W1"], g["b1"], g["W3"],
                        g["b3"], g["W2"], g["b2"], y, ws)
    assert torch.equal(y, o["y"])
    for name in ("b1", "b3", "b2"):
        zeros = {n: torch.zeros_like(g[n]) for n in ("b1", "b3", "b2") if n != name}
        a = G.run_forward(cfg, R.GELU, dict(g, **zeros))
        b = G.run_forward(cfg, R.GELU, dict(g, **dict.fromkeys(zeros)))
        assert torch.equal(a["y"], b["y"]), name
    full = G.run_backward(cfg, R.GELU, g, o["p1"], o["p3"])
    for keep in ((), ("db1",), ("db3",), ("db2",), ("db1", "db2")):
        out = {n: torch.full_like(full[n], 9.0) for n in GRADS}
        wb = G.buf(B.moe_gated_backward_workspace_size(cfg))
        args = {n: out[n] if n in keep else None for n in ("db1", "db3", "db2")}
        B.moe_experts_gated_backward(cfg, R.GELU, g["x"], g["idx"], g["gate"], o["p1"], o["p3"],
                                     g["W1"], g["W3"], g["W2"], g["b2"], g["dy"], out["dx"],
                                     out["dgate"], out["dW1"], args["db1"], out["dW3"],
                                     args["db3"], out["dW2"], args["db2"], wb)
        for n in GRADS:
            want = full[n] if n in keep or not n.startswith("db") else torch.full_like(full[n], 9.0)
            assert torch.equal(out[n], want), (keep, n)


@pytest.mark.parametrize("T", [3, 400])
def test_fp8_arguments_left_out(T):
    s = G.inputs(T, 200, 4, 330, 2, BF16, seed=T)
    cfg, g = G.config(s, 1.25), G.dev(s)
    w8 = [G.quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    (q1, s1), (q3, s3), (q2, s2) = w8
    for name in ("b1", "b3", "b2"):
        zeros = {n: torch.zeros_like(g[n]) for n in ("b1", "b3", "b2") if n != name}
        a = G.run_fp8(cfg, R.SILU, dict(g, **zeros), w8)
        b = dict(g, **dict.fromkeys(zeros))
        y, ws = torch.empty_like(g["x"]), G.buf(B.moe_gated_fp8_workspace_size(cfg))
        B.moe_experts_gated_fp8(cfg, R.SILU, g["x"], g["idx"], g["gate"], q1, s1, b["b1"], q3, s3,
                                b["b3"], q2, s2, b["b2"], y, ws)
        assert torch.equal(a["y"], y), name


def entry_points():
    """Each call with its outputs: (run(stream), outputs, workspace)."""
    ep = {}
    for T, dt, d, F in FORMS:
        s = G.inputs(T, d, 4, F, 2, dt, seed=T)
        cfg, g = G.config(s, 2.0), G.dev(s)
        o = G.run_forward(cfg, R.SILU, g)
        y = torch.empty_like(g["x"])

        def forward(stream, cfg=cfg, g=g, y=y, ws=o["ws"]):
            G.run_forward(cfg, R.SILU, g, keeps=False, y=y, ws=ws, stream=stream)
        ep[f"gated-{T}-{d}-{dt}"] = (forward, [y], o["ws"])
        b = G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
        outs = [torch.empty_like(b[n]) for n in GRADS]

        def backward(stream, cfg=cfg, g=g, o=o, r=outs, ws=b["ws"]):
            B.moe_experts_gated_backward(cfg, R.SILU, g["x"], g["idx"], g["gate"], o["p1"],
                                         o["p3"], g["W1"], g["W3"], g["W2"], g["b2"], g["dy"],
                                         r[0], r[1], r[2], r[5], r[3], r[6], r[4], r[7], ws,
                                         stream=stream)
        ep[f"backward-{T}-{d}-{dt}"] = (backward, outs, b["ws"])
        if dt == BF16:
            w8 = [G.quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
            y8, ws8 = torch.empty_like(g["x"]), G.buf(B.moe_gated_fp8_workspace_size(cfg))

            def fp8(stream, cfg=cfg, g=g, w8=w8, y=y8, ws=ws8):
                G.run_fp8(cfg, R.SILU, g, w8, ws=ws, stream=stream, y=y)
            ep[f"fp8-{T}-{d}"] = (fp8, [y8], ws8)
        E, K, N = g["W1"].shape
        n8, ns = B.moe_weights_fp8_size(E, K, N)
        q, sc, wsq = G.buf(n8), G.buf(ns), G.buf(256, 0)

        def weights(stream, g=g, n=(E, K, N), dt=dt, q=q, sc=sc, ws=wsq):
            B.moe_weights_fp8(*n, B.MOE_BF16 if dt == BF16 else B.MOE_F32, g["W1"], q, sc, ws,
                              stream=stream)
        ep[f"weights-{T}-{d}-{dt}"] = (weights, [q, sc], wsq)
    return ep


def bits(outs):
    return [o.clone().view(torch.uint8) for o in outs]


def test_as_a_threads_first_call():
    stream = torch.cuda.Stream()
    for name, (run, outs, ws) in entry_points().items():
        run(None)
        assert B.moe_last_device_status(ws)[0] == 0, name
        want = bits(outs)
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        on_new_thread(lambda run=run: run(stream))
        assert B.moe_last_device_status(ws)[0] == 0, name
        for a, b in zip(bits(outs), want):
            assert torch.equal(a, b), name


def first_backward_under_capture():
    """In a process of its own: the first backward is a captured one, when no side
    stream can be made; an eager one and a replay have the same bits."""
    for dt, d, F in ((BF16, 128, 256), (F32, 34, 66)):
        s = G.inputs(300, d, 4, F, 2, dt, seed=1)
        cfg, g = G.config(s, 2.0), G.dev(s)
        o = G.run_forward(cfg, R.SILU, g)
        ws = G.buf(B.moe_gated_backward_workspace_size(cfg))
        torch.cuda.synchronize()
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=st):
            b = G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"], ws=ws)
        graph.replay()
        torch.cuda.synchronize()
        c = G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
        for n in GRADS:
            assert torch.equal(b[n], c[n]), n
    print("same bits")


def test_a_process_first_backward_under_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([root, os.path.join(root, "tests")]))
    r = subprocess.run([sys.executable, "-c", "import test_gpu_gated_calls as t; "
                        "t.first_backward_under_capture()"], env=env, cwd=root,
                       capture_output=True, text=True)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("T,d,E,F,k,cf,min_cap,dt", [
    (130, 128, 24, 192, 16, 2.0, 1, BF16), (130, 66, 24, 70, 16, 2.0, 1, F32),
    (300, 64, 5, 128, 2, 1.0, 1000, BF16), (300, 30, 5, 50, 2, 1.0, 1000, F32),
    (400, 64, 40, 128, 3, 1e-6, 1, BF16), (400, 31, 40, 33, 3, 1e-6, 1, BF16),
    (400, 64, 3, 128, 3, 1e6, 1, BF16)])
def test_borders_of_k_and_capacity(T, d, E, F, k, cf, min_cap, dt):
    """Sixteen choices; more slots than rows; a single slot an expert."""
    s = G.inputs(T, d, E, F, k, dt, seed=T + k)
    s["idx"][1] = s["idx"][1, 0]
    cfg, g = G.config(s, cf), G.dev(s)
    cfg.min_capacity = min_cap
    o = G.run_forward(cfg, R.SILU, g)
    G.check_forward(cfg, R.SILU, s, o, G.reference(cfg, R.SILU, s))
    G.check_backward(cfg, R.SILU, s, o["p1"], o["p3"],
                     G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"]))
    if dt == BF16:
        w8 = [G.quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
        G.check_forward(cfg, R.SILU, s, G.run_fp8(cfg, R.SILU, g, w8),
                        G.reference8(cfg, R.SILU, s, w8))


@pytest.mark.parametrize("T,d,F,dt", [
    (2, 64, 524288, BF16), (2, 524288, 64, BF16), (2, 3, 524288, F32), (2, 524287, 2, F32),
    (70, 64, 65536, BF16), (70, 65536, 64, BF16), (70, 3, 524288, F32), (70, 524287, 2, F32)])
def test_the_widest(T, d, F, dt):
    s = G.inputs(T, d, 2, F, 1, dt, seed=T, biases=False)
    cfg, g = G.config(s, 2.0), G.dev(s)
    o = G.run_forward(cfg, R.SILU, g)
    G.check_forward(cfg, R.SILU, s, o, G.reference(cfg, R.SILU, s))
    G.check_backward(cfg, R.SILU, s, o["p1"], o["p3"],
                     G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"]))
    if dt == BF16:
        w8 = [G.quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
        G.check_forward(cfg, R.SILU, s, G.run_fp8(cfg, R.SILU, g, w8),
                        G.reference8(cfg, R.SILU, s, w8))

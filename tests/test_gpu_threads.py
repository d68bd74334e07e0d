"""Calls from other host threads than the first: what a call does not depend
on the thread that makes it."""
import ctypes
import subprocess
import threading

import pytest
import torch

from gpu_harness import hier_to_device, to_device
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import workloads as wl
from test_gpu_few import _w, call, outputs, workspace

pytestmark = pytest.mark.gpu


def on_new_thread(fn):
    """fn on a thread that has made no CUDA call."""
    errors = []

    def run():
        try:
            fn()
        except Exception as e:  # noqa: BLE001 (reported by the caller's thread)
            errors.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_as_a_threads_first_call(dtype):
    w = _w(5, 64, 4, 64, 2, dtype=dtype)
    cfg = B.config_for(w)
    d = to_device(w, wl.generate(w, seed=1))
    want, got, ws = outputs(w, cfg), outputs(w, cfg), workspace(cfg)
    call(cfg, d, want, ws)
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    on_new_thread(lambda: call(cfg, d, got, ws, stream))
    assert B.moe_last_device_status(ws)[0] == 0
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_expert_ffn_as_a_threads_first_call():
    w = _w(64, 64, 4, 128, 1)
    cfg = B.config_for(w)
    d = to_device(w, wl.generate(w, seed=2))
    z = dict(device="cuda")
    offset = torch.arange(0, 65, 16, dtype=torch.int32, **z)
    gate = torch.ones(64, **z)
    ws = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, **z)
    outs = [(torch.zeros((64, 128), dtype=torch.bfloat16, **z), torch.zeros((64, 64), **z))
            for _ in range(2)]

    def run(o, stream=None):
        B.moe_expert_ffn(cfg, d["x"], offset, gate, d["W1"], None, d["W2"], None, *o, ws,
                         stream=stream)
    run(outs[0])
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    on_new_thread(lambda: run(outs[1], stream))
    assert B.moe_last_device_status(ws)[0] == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def entry_points():
    """Every other entry point that enqueues work, as (call, outputs, workspace):
    the call takes a stream."""
    z = dict(device="cuda")
    w = wl.Workload("t", T=96, d=64, E=6, d_ff=128, k=2, cf=1.0, mode=wl.TOPK, dtype="bf16",
                    noisy=True)
    cfg, d = B.config_for(w), to_device(w, wl.generate(w, seed=3, biases=True))
    A = w.T * w.k

    def new(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, **z)

    def space(n):
        return new(n, dtype=torch.uint8)
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    router = (d["x"], d["Wg"], d["Wn"], d["noise"], None)
    experts = (d["W1"], d["b1"], d["W2"], d["b2"])
    # A forward's state, which some of them start from.
    base, bws = space(B.moe_workspace_size(cfg)), space(B.moe_backward_workspace_size(cfg))
    y0, out0 = new(w.T, w.d, dtype=bf), new(3)
    idx, gate = new(w.T, w.k, dtype=i32), new(w.T, w.k)
    B.moe_forward(cfg, *router, *experts, y0, out0, base, idx, gate)
    _, n8, ns = B.moe_checkpoint_size(cfg)
    h8, hs = space(n8), space(ns)
    B.moe_checkpoint_save(cfg, None, None, h8, hs, base)
    dy = torch.ones_like(y0)
    ep = {}

    def add(name, make, outs, ws):
        ep[name] = (make, outs, ws)

    o, ws = [new(w.T, w.k, dtype=i32), new(w.T, w.k), new(w.T, 2)], base.clone()
    add("moe_gate", lambda s, o=o, ws=ws: B.moe_gate(cfg, *router, *o, ws, stream=s), o, ws)
    o, ws = [new(w.T, w.d, dtype=bf), new(3)], base.clone()
    add("moe_forward", lambda s, o=o, ws=ws: B.moe_forward(cfg, *router, *experts, *o, ws,
                                                           stream=s), o, ws)
    o = [new(w.T, w.k, dtype=i32), new(w.T, w.k, dtype=u8), new(w.E, dtype=i32),
         new(w.E + 1, dtype=i32), new(A, w.d, dtype=bf), new(A, dtype=i32), new(A)]
    ws = base.clone()
    add("moe_dispatch", lambda s, o=o, ws=ws: B.moe_dispatch(cfg, idx, gate, d["x"], *o, ws,
                                                             stream=s), o, ws)
    o = [torch.zeros_like(v) for v in o]
    add("moe_dispatch_noalloc", lambda s, o=o: B.moe_dispatch_noalloc(cfg, idx, gate, d["x"], *o,
                                                                      stream=s), o, ws)

    def grads(dtype):
        return [new(w.T, w.d, dtype=bf), new(w.d, w.E), new(w.d, w.E), new(w.E),
                new(w.E, w.d, w.d_ff, dtype=dtype), new(w.E, w.d_ff, dtype=dtype),
                new(w.E, w.d_ff, w.d, dtype=dtype), new(w.E, w.d, dtype=dtype), new(w.T, w.k)]
    o, ws = grads(torch.float32), base.clone()
    add("moe_backward", lambda s, o=o, ws=ws: B.moe_backward(
        cfg, *router[:4], d["W1"], d["W2"], d["b2"], idx, gate, None, None, dy, 0.1, 0.2, 0.3, *o,
        ws, bws, stream=s), o, ws)
    o, ws = grads(bf), base.clone()
    add("moe_backward_checkpoint", lambda s, o=o, ws=ws: B.moe_backward_checkpoint(
        cfg, *router, d["W1"], d["W2"], d["b2"], idx, gate, h8, hs, dy, 0.1, 0.2, 0.3, *o, ws,
        bws, stream=s), o, ws)
    o, ws = [space(n8), space(ns)], base.clone()
    add("moe_checkpoint_save", lambda s, o=o, ws=ws: B.moe_checkpoint_save(
        cfg, None, None, *o, ws, stream=s), o, ws)
    ws = base.clone()
    add("moe_checkpoint_load", lambda s, ws=ws: B.moe_checkpoint_load(
        cfg, h8, hs, None, None, ws, stream=s), [ws], ws)
    thr, thr2 = (torch.full((w.E,), v, **z) for v in (0.2, 0.4))
    o, ws = [new(w.T, w.d, dtype=bf)], space(B.moe_threshold_workspace_size(cfg))
    add("moe_forward_threshold", lambda s, o=o, ws=ws: B.moe_forward_threshold(
        cfg, d["x"], d["Wg"], None, thr2, *experts, *o, ws, stream=s), o, ws)
    few = B.config(32, w.d, w.E, w.d_ff, w.E, 1.0)
    o, ws = [new(32, w.d, dtype=bf)], space(B.moe_few_workspace_size(few))
    add("moe_forward_threshold_few", lambda s, o=o, ws=ws: B.moe_forward_threshold_few(
        few, d["x"], d["Wg"], None, thr, *experts, *o, ws, stream=s), o, ws)
    o, ws = [new(w.T, w.d, dtype=bf), new(1)], space(B.moe_balanced_workspace_size(cfg))
    add("moe_forward_balanced", lambda s, o=o, ws=ws: B.moe_forward_balanced(
        cfg, d["x"], d["Wg"], None, thr, *experts, *o, None, ws, stream=s), o, ws)
    h = wl.HierWorkload("t", T=64, d=64, a=4, b=8, kp=2, ks=2, d_ff=64, cf=4.0, dtype="bf16",
                        noisy=False)
    hd = hier_to_device(h, wl.generate_hier(h, seed=4))
    o = [torch.zeros_like(hd["x"]), new(2)]
    ws = space(B.moe_hier_workspace_size(B.hier_config_for(h)))
    add("moe_forward_hier", lambda s, o=o, ws=ws: B.moe_forward_hier(
        B.hier_config_for(h), hd["x"], hd["Wp"], None, None, hd["Ws"], None, None, hd["W1"], None,
        hd["W2"], None, *o, ws, stream=s), o, ws)
    return ep


def test_every_entry_point_as_a_threads_first_call():
    stream = torch.cuda.Stream().cuda_stream
    for name, (run, outs, ws) in entry_points().items():
        run(None)
        assert B.moe_last_device_status(ws)[0] == 0, name
        want = [o.clone() for o in outs]
        for o in outs:
            if o is not ws:
                o.zero_()
        torch.cuda.synchronize()
        on_new_thread(lambda run=run: run(stream))
        assert B.moe_last_device_status(ws)[0] == 0, name
        for a, b in zip(outs, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


# ----------------------------------------------------------------------------- at once
# What launches of a kernel may take of shared memory is one setting for all
# threads, and the two sizes of each test ask for different amounts: no call may
# lower it under another. The calls come from loops in C, a few microseconds
# apart, so that they do meet.
HAMMER = """
typedef const void *P;
typedef int (*F17)(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P);
typedef int (*F18)(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P);
typedef int (*F20)(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P);
typedef int (*FB)(P, P, P, P, P, P, P, P, P, P, P, P, P, float, float, float, P, P, P, P, P, P, P,
                  P, P, P, P, P);
#define A10 a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9]
/* The first status that is not 0, of n calls. */
int hammer(P f, int kind, const P *a, int n) {
  for (int i = 0; i < n; ++i) {
    int r;
    if (kind == 17)
      r = ((F17)f)(A10, a[10], a[11], a[12], a[13], a[14], a[15], a[16]);
    else if (kind == 18)
      r = ((F18)f)(A10, a[10], a[11], a[12], a[13], a[14], a[15], a[16], a[17]);
    else if (kind == 20)
      r = ((F20)f)(A10, a[10], a[11], a[12], a[13], a[14], a[15], a[16], a[17], a[18], a[19]);
    else
      r = ((FB)f)(A10, a[10], a[11], a[12], 0.f, 0.f, 0.f, a[13], a[14], a[15], a[16], a[17],
                  a[18], a[19], a[20], a[21], a[22], a[23], a[24]);
    if (r) return r;
  }
  return 0;
}
"""
BACKWARD = 25


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    at = tmp_path_factory.mktemp("hammer")
    (at / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", at / "hammer.so", at / "hammer.c"],
                   check=True)
    fn = ctypes.CDLL(str(at / "hammer.so")).hammer
    fn.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int]

    def run(name, cfg, args, stream, rounds=30, calls=200):
        """`calls` calls in a row, then a wait, `rounds` times."""
        a = [ctypes.addressof(cfg)] + [B._p(v) for v in args] + [stream.cuda_stream]
        f = ctypes.cast(getattr(B.lib(), name), ctypes.c_void_p)
        kind = BACKWARD if name == "moe_backward" else len(a)
        for _ in range(rounds):
            st = fn(f, kind, (ctypes.c_void_p * len(a))(*a), calls)
            stream.synchronize()
            assert st == 0, (name, B.STATUS_NAMES[st])
    return run


def at_once(hammer, lanes):
    """Each lane, (calls, outputs, workspace), runs its calls once alone and
    then, on a thread and a stream of its own, many times beside the others."""
    want = []
    for calls, outs, ws in lanes:
        for name, cfg, args in calls:
            hammer(name, cfg, args, torch.cuda.current_stream(), 1, 1)
        assert B.moe_last_device_status(ws)[0] == 0
        want.append([o.clone() for o in outs])
        for o in outs:
            o.fill_(0)
    torch.cuda.synchronize()
    gate, errors = threading.Barrier(len(lanes)), []

    def loop(calls):
        s = torch.cuda.Stream()
        try:
            for name, cfg, args in calls:
                gate.wait()
                hammer(name, cfg, args, s)
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)
            gate.abort()
    threads = [threading.Thread(target=loop, args=(lane[0],)) for lane in lanes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (_, outs, ws), kept in zip(lanes, want):
        assert B.moe_last_device_status(ws)[0] == 0
        for o, k in zip(outs, kept):
            assert torch.equal(o, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_of_two_sizes(hammer, dtype):
    lanes = []
    for w in (_w(1, 64, 4, 64, 1, dtype=dtype), _w(64, 64, 1024, 64, 16, cf=64.0, dtype=dtype)):
        cfg = B.config_for(w)
        d = to_device(w, wl.generate(w, seed=w.E))
        o, ws = outputs(w, cfg), workspace(cfg)
        args = [d["x"], d["Wg"], None, None, None, d["W1"], None, d["W2"], None, o["y"], o["idx"],
                o["gate"], o["pos"], o["keep"], ws]
        lanes.append(([("moe_forward_few", cfg, args)], list(o.values()), ws))
    at_once(hammer, lanes)


def test_forward_and_backward_of_two_expert_counts(hammer):
    """The whole layer, whose kernels take more with more experts."""
    lanes = []
    for E in (4, 1024):
        w = _w(128, 64, E, 64, 2, cf=4.0)
        cfg = B.config_for(w)
        d = to_device(w, wl.generate(w, seed=E))
        dy = torch.ones_like(d["x"])
        y, dx = torch.zeros_like(dy), torch.zeros_like(dy)
        dWg, dW1, dW2 = (torch.zeros(s, device="cuda")
                         for s in ((64, E), (E, 64, 64), (E, 64, 64)))
        ws = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        bws = torch.zeros(B.moe_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        forward = [d["x"], d["Wg"], None, None, None, d["W1"], None, d["W2"], None, y, None, None,
                   None, None, None, ws]
        backward = [d["x"], d["Wg"], None, None, d["W1"], d["W2"], None, None, None, None, None,
                    dy, dx, dWg, None, None, dW1, None, dW2, None, None, ws, bws]
        lanes.append(([("moe_forward", cfg, forward), ("moe_backward", cfg, backward)],
                      [y, dx, dWg, dW1, dW2], ws))
    at_once(hammer, lanes)


def test_hierarchical_layers_of_two_sizes(hammer):
    lanes = []
    for a, kp in ((4, 2), (32, 8)):
        w = wl.HierWorkload("t", T=128, d=64, a=a, b=32, kp=kp, ks=2, d_ff=64, cf=4.0,
                            dtype="bf16", noisy=False)
        cfg = B.hier_config_for(w)
        d = hier_to_device(w, wl.generate_hier(w, seed=a))
        y, out2 = torch.zeros_like(d["x"]), torch.zeros(2, device="cuda")
        ws = torch.zeros(B.moe_hier_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        args = [d["x"], d["Wp"], None, None, d["Ws"], None, None, d["W1"], None, d["W2"], None, y,
                out2, None, None, None, None, ws]
        lanes.append(([("moe_forward_hier", cfg, args)], [y, out2], ws))
    at_once(hammer, lanes)

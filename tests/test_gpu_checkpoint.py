"""The 8-bit checkpoint and the backward from it on the GPU: the format value
for value, the gradients against plain fp64 and, bit for bit, against
moe_backward on the loaded rows; a stack of layers on one workspace, graphs,
refusals and errors."""
import numpy as np
import pytest
import torch

import checkpoint_reference as ref
import few_reference as few
from gpu_harness import act_to_f64, dev_act, to_device
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

W = wl.Workload
WEIGHTS = (0.4, 0.6, 0.3)


def scratch(n, fill=0xFF):
    """Scratch memory that holds anything."""
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


def checkpoint(cfg):
    rows, n8, ns = B.moe_checkpoint_size(cfg)
    return scratch(n8, 0xAB), scratch(ns, 0xCD), rows


# ----------------------------------------------------------------------------- the format
def _rows(R, F, dtype, seed):
    rng = np.random.default_rng(seed)
    h = np.maximum(rng.standard_normal((R, F)), 0) * np.exp2(rng.integers(-8, 8, (R, 1)))
    if R > 6:
        h[1] = 0.0
        h[2, : F // 2] = 0.0
        h[3] *= 2.0 ** -125          # scales at their smallest exponent
        h[4, ::7] *= 2.0 ** -30      # far below the block's largest
        h[5] *= 2.0 ** 118 / max(1e-3, h[5].max())
        h[6, :: max(1, F // 5)] = 3.3895313892515355e38  # bf16's largest
    h = h.astype(np.float32)
    return wl.f32_to_bf16_bits(h) if dtype == "bf16" else h


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("F", [1, 8, 31, 32, 33, 40, 256, 1000, 1024, 1032, 2050, 2056])
def test_format_against_fp64(dtype, F):
    R, E = 11, 3
    cfg = B.config(R, 8, E, F, 1, 3.0,
                   act_dtype=B.MOE_BF16 if dtype == "bf16" else B.MOE_F32)
    bits = _rows(R, F, dtype, F)
    h = dev_act(bits, dtype)
    n = 9  # two rows past the last expert's: neither read nor written
    off = torch.tensor([0, 4, 4, n], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h8, hs, rows = checkpoint(cfg)
    assert rows == R
    B.moe_checkpoint_save(cfg, h, off, h8, hs, ws)
    out = torch.full_like(h, -5)
    B.moe_checkpoint_load(cfg, h8, hs, off, out, ws)
    assert B.moe_last_device_status(ws) == (0, 0)
    q, s, v = ref.quantise(few.f64(bits[:n], dtype))
    nb = s.shape[1]
    assert np.array_equal(h8.cpu().numpy().reshape(R, F)[:n], q)
    assert np.array_equal(hs.cpu().numpy().reshape(R, nb)[:n], s)
    assert np.all(h8.cpu().numpy().reshape(R, F)[n:] == 0xAB)
    assert np.all(hs.cpu().numpy().reshape(R, nb)[n:] == 0xCD)
    assert np.array_equal(act_to_f64(out[:n]), v)
    assert bool((out[n:] == -5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("F", [64, 50])
def test_values_below_zero_are_stored_as_zero(dtype, F):
    cfg = B.config(4, 8, 1, F, 1, 1.0, act_dtype=B.MOE_BF16 if dtype == "bf16" else B.MOE_F32)
    h = np.random.default_rng(2).standard_normal((4, F)).astype(np.float32)
    h[1] = -np.abs(h[1])
    h[2, 3], h[2, 40], h[3, 0] = -np.inf, -0.0, -1e-38
    bits = wl.f32_to_bf16_bits(h) if dtype == "bf16" else h
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h8, hs, _ = checkpoint(cfg)
    B.moe_checkpoint_save(cfg, dev_act(bits, dtype), off, h8, hs, ws)
    q, s, _ = ref.quantise(few.f64(bits, dtype))
    assert B.moe_last_device_status(ws)[0] == 0
    assert np.array_equal(h8.cpu().numpy().reshape(4, F), q)
    assert np.array_equal(hs.cpu().numpy().reshape(4, -1), s)


@pytest.mark.parametrize("F", [64, 50])
def test_nonfinite_rows_are_recorded_and_load_as_nan(F):
    cfg = B.config(4, 8, 1, F, 1, 1.0)
    bits = _rows(4, F, "bf16", 1)
    bits[2, 35], bits[3, 1] = 0x7F80, 0x7FC0
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h8, hs, _ = checkpoint(cfg)
    B.moe_checkpoint_save(cfg, dev_act(bits, "bf16"), off, h8, hs, ws)
    st, det = B.moe_last_device_status(ws)
    assert st == 4 and det // F in (2, 3)
    out = torch.zeros((4, F), dtype=torch.bfloat16, device="cuda")
    B.moe_checkpoint_load(cfg, h8, hs, off, out, ws)
    _, _, v = ref.quantise(few.f64(bits, "bf16"))
    assert np.array_equal(np.isnan(act_to_f64(out)), np.isnan(v))
    assert np.isnan(v).sum() == min(F, 64) - 32 + 32


def test_no_rows():
    cfg = B.config(4, 8, 2, 64, 1, 1.0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h8, hs, _ = checkpoint(cfg)
    h = torch.full((4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    B.moe_checkpoint_save(cfg, h, off, h8, hs, ws)
    out = torch.zeros_like(h)
    B.moe_checkpoint_load(cfg, h8, hs, off, out, ws)
    assert B.moe_last_device_status(ws)[0] == 0
    assert bool((h8 == 0xAB).all()) and bool((hs == 0xCD).all()) and bool((out == 0).all())


# ----------------------------------------------------------------------------- the backward
CASES = {
    "tc_top2": W("c", 96, 64, 5, 128, 2, 1.0, wl.TOPK, "bf16", True),
    "tc_clean": W("c", 70, 128, 4, 64, 2, 2.0, wl.TOPK, "bf16", False),
    "tc_switch": W("c", 130, 64, 6, 192, 1, 1.0, wl.SWITCH, "bf16", True),
    "tc_all_experts": W("c", 40, 64, 4, 64, 4, 1.0, wl.TOPK, "bf16", True),
    "tc_capacity_one": W("c", 33, 64, 40, 64, 2, 0.2, wl.TOPK, "bf16", True),
    "odd_bf16": W("c", 61, 44, 5, 70, 3, 1.0, wl.TOPK, "bf16", True),
    "one_token": W("c", 1, 64, 3, 64, 2, 1.0, wl.TOPK, "bf16", False),
    "one_token_f32": W("c", 1, 5, 3, 7, 1, 1.0, wl.SWITCH, "f32", False),
    "f32": W("c", 75, 48, 6, 96, 2, 0.8, wl.TOPK, "f32", True),
    "f32_odd": W("c", 53, 21, 5, 37, 3, 1.2, wl.TOPK, "f32", True),
}


def forward(w, d, inp):
    """moe_forward on its own workspace, its choices and its checkpoint."""
    cfg = B.config_for(w)
    act = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    z = dict(device="cuda")
    o = dict(y=torch.empty((w.T, w.d), dtype=act, **z), out3=torch.zeros(3, **z),
             idx=torch.empty((w.T, w.k), dtype=torch.int32, **z),
             gate=torch.empty((w.T, w.k), **z),
             pos=torch.empty((w.T, w.k), dtype=torch.int32, **z),
             keep=torch.empty((w.T, w.k), dtype=torch.uint8, **z),
             ws=torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, **z))
    B.moe_forward(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], d["bias"], d["W1"], d["b1"], d["W2"],
                  d["b2"], o["y"], o["out3"], o["ws"], o["idx"], o["gate"], o["pos"], o["keep"])
    o["h8"], o["hs"], _ = checkpoint(cfg)
    B.moe_checkpoint_save(cfg, None, None, o["h8"], o["hs"], o["ws"])
    assert B.moe_last_device_status(o["ws"])[0] == 0
    return o


def grads(w, small=None):
    act = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    small = small or act

    def n(*s, dtype=torch.float32):
        return torch.full(s, float("nan"), dtype=dtype, device="cuda")
    T, d, E, F = w.T, w.d, w.E, w.d_ff
    return dict(dx=n(T, d, dtype=act), dWg=n(d, E), dWn=n(d, E) if w.noisy else None, dbias=n(E),
                dW1=n(E, d, F, dtype=small), db1=n(E, F, dtype=small),
                dW2=n(E, F, d, dtype=small), db2=n(E, d, dtype=small), dgate=n(T, w.k))


def backward(w, d, f, dy, weights=WEIGHTS, ws=None, bws=None, stream=None, g=None):
    cfg = B.config_for(w)
    ws = scratch(B.moe_workspace_size(cfg)) if ws is None else ws
    bws = scratch(B.moe_backward_workspace_size(cfg)) if bws is None else bws
    g = grads(w) if g is None else g
    B.moe_backward_checkpoint(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], d["bias"], d["W1"],
                              d["W2"], d["b2"], f["idx"], f["gate"], f["h8"], f["hs"], dy,
                              *weights, g["dx"], g["dWg"], g["dWn"], g["dbias"], g["dW1"],
                              g["db1"], g["dW2"], g["db2"], g["dgate"], ws, bws, stream=stream)
    return g, ws


def setup(name, seed=3):
    w = CASES[name] if isinstance(name, str) else name
    inp = wl.generate(w, seed=seed, biases=True)
    inp["bias"] = (np.random.default_rng(seed).standard_normal(w.E) * 0.2).astype(np.float32)
    d = to_device(w, inp)
    dyb = wl.generate_dy(w, seed)
    return w, inp, d, dyb, dev_act(dyb, w.dtype)


@pytest.mark.parametrize("name", sorted(CASES))
def test_backward_against_fp64(name):
    w, inp, d, dyb, dy = setup(name)
    f = forward(w, d, inp)
    g, ws = backward(w, d, f, dy)
    assert B.moe_last_device_status(ws)[0] == 0
    # The hidden values as stored, per choice.
    n8 = f["h8"].cpu().numpy().reshape(-1, w.d_ff)
    hs = f["hs"].cpu().numpy().reshape(n8.shape[0], -1)
    idx, keep, pos = (f[n].cpu().numpy() for n in ("idx", "keep", "pos"))
    off = np.zeros(w.E + 1, int)
    np.add.at(off[1:], idx[keep.astype(bool)], 1)
    off = np.cumsum(off)
    h = np.zeros((w.T, w.k, w.d_ff))
    for t, j in np.argwhere(keep):
        r = off[idx[t, j]] + pos[t, j]
        s = np.repeat(2.0 ** (hs[r].astype(float) - 127), ref.BLOCK)[: w.d_ff]
        h[t, j] = ref.VALUES[n8[r]] * s
    want, err, _ = ref.backward(inp, w.dtype, w.mode, idx, f["gate"].cpu().numpy(), keep, h,
                                few.f64(dyb, w.dtype), WEIGHTS)
    for n, v in want.items():
        if v is None:
            continue
        off_by = np.abs(act_to_f64(g[n]) - v)
        assert np.all(off_by <= err[n]), (n, off_by.max(), (off_by / err[n]).max())


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("weights", [WEIGHTS, (0.0, 0.0, 0.0)])
def test_backward_is_moe_backward_on_the_loaded_rows(name, weights):
    w, inp, d, _, dy = setup(name)
    f = forward(w, d, inp)
    cfg = B.config_for(w)

    def plain():
        o = grads(w, torch.float32)
        B.moe_backward(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], d["W1"], d["W2"], d["b2"],
                       f["idx"], f["gate"], f["pos"], f["keep"], dy, *weights, o["dx"], o["dWg"],
                       o["dWn"], o["dbias"], o["dW1"], o["db1"], o["dW2"], o["db2"], o["dgate"],
                       f["ws"], scratch(B.moe_backward_workspace_size(cfg)))
        assert B.moe_last_device_status(f["ws"])[0] == 0
        return o
    exact_rows = plain()
    B.moe_checkpoint_load(cfg, f["h8"], f["hs"], None, None, f["ws"])
    loaded_rows = plain()
    g, ws = backward(w, d, f, dy, weights)
    assert B.moe_last_device_status(ws)[0] == 0
    for n, v in g.items():
        if v is not None:
            assert torch.equal(v, loaded_rows[n].to(v.dtype)), n
    # What uses only the rows' ReLU pattern does not see the rounding at all.
    for n in ("dW1", "db1", "db2"):
        assert torch.equal(g[n], exact_rows[n].to(g[n].dtype)), n


@pytest.mark.parametrize("variant", ["single", "pair"])
def test_bf16_weight_gradients_of_both_kernels(monkeypatch, variant):
    """Whole and partial tiles of the weight gradient in bf16, in the one-CTA
    and the CTA-pair kernel: moe_backward's fp32 ones, rounded."""
    monkeypatch.setenv("MOE_BWD_TC_VARIANT", variant)
    for w in (W("c", 700, 320, 3, 448, 2, 2.0, wl.TOPK, "bf16", False),
              W("c", 64, 64, 70, 64, 2, 1.0, wl.TOPK, "bf16", False)):
        test_backward_is_moe_backward_on_the_loaded_rows(w, WEIGHTS)


def test_a_stack_of_layers_on_one_workspace():
    """Three layers forward and backward through one workspace, each layer
    keeping x, its choices and a checkpoint: every gradient is what the layer
    gives alone, with a workspace of its own."""
    w = W("c", 150, 64, 6, 128, 2, 1.25, wl.TOPK, "bf16", True)
    cfg = B.config_for(w)
    layers = []
    x = None
    ws = scratch(B.moe_workspace_size(cfg))
    bws = scratch(B.moe_backward_workspace_size(cfg))
    for i in range(3):
        inp = wl.generate(w, seed=40 + i, biases=True)
        inp["bias"] = None
        d = to_device(w, inp)
        if x is not None:
            d["x"] = x
        f = dict(y=torch.empty_like(d["x"]), idx=torch.empty((w.T, w.k), dtype=torch.int32, device="cuda"),
                 gate=torch.empty((w.T, w.k), device="cuda"))
        B.moe_forward(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], None, d["W1"], d["b1"], d["W2"],
                      d["b2"], f["y"], None, ws, f["idx"], f["gate"])
        f["h8"], f["hs"], _ = checkpoint(cfg)
        B.moe_checkpoint_save(cfg, None, None, f["h8"], f["hs"], ws)
        layers.append((d, f))
        x = f["y"]
    dy = dev_act(wl.generate_dy(w, 1), "bf16")
    got = []
    up = dy
    for d, f in reversed(layers):
        g, _ = backward(w, d, f, up, ws=ws, bws=bws)
        got.append(g)
        up = g["dx"]
    assert B.moe_last_device_status(ws)[0] == 0
    up = dy
    for (d, f), g in zip(reversed(layers), got):
        alone = forward(w, d, None)
        want, ws1 = backward(w, d, alone, up)
        assert B.moe_last_device_status(ws1)[0] == 0
        for n, v in want.items():
            assert torch.equal(v, g[n]), n
        up = g["dx"]


def test_backward_in_a_graph():
    """Forward, save and backward captured into one graph on a side stream;
    replays reproduce the eager bits."""
    w, inp, d, _, dy = setup("tc_top2")
    cfg = B.config_for(w)
    f = forward(w, d, inp)
    want, _ = backward(w, d, f, dy)
    ws = scratch(B.moe_workspace_size(cfg))
    bws = scratch(B.moe_backward_workspace_size(cfg))
    g = grads(w)
    o = dict(f, h8=torch.zeros_like(f["h8"]), hs=torch.zeros_like(f["hs"]))

    def step(s):
        B.moe_forward(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], d["bias"], d["W1"], d["b1"],
                      d["W2"], d["b2"], o["y"], None, ws, o["idx"], o["gate"], stream=s)
        B.moe_checkpoint_save(cfg, None, None, o["h8"], o["hs"], ws, stream=s)
        backward(w, d, o, dy, ws=ws, bws=bws, stream=s, g=g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(torch.cuda.current_stream())
    for v in g.values():
        if v is not None:
            v.fill_(float("nan"))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert B.moe_last_device_status(ws)[0] == 0
    for n, v in want.items():
        if v is not None:
            assert torch.equal(v, g[n]), n


def test_backward_on_more_streams_than_side_streams():
    """The library pairs eight caller streams with side streams; further ones
    run everything on their own, with the same bits."""
    w, inp, d, _, dy = setup("tc_top2")
    f = forward(w, d, inp)
    want, _ = backward(w, d, f, dy)
    torch.cuda.synchronize()
    cfg = B.config_for(w)
    lanes = [(torch.cuda.Stream(), scratch(B.moe_workspace_size(cfg)),
              scratch(B.moe_backward_workspace_size(cfg)), grads(w)) for _ in range(10)]
    torch.cuda.synchronize()
    for s, ws, bws, g in lanes:
        backward(w, d, f, dy, ws=ws, bws=bws, stream=s, g=g)
    torch.cuda.synchronize()
    for s, ws, _, g in lanes:
        assert B.moe_last_device_status(ws, s)[0] == 0
        for n, v in want.items():
            if v is not None:
                assert torch.equal(v, g[n]), n


def test_optional_outputs():
    w, inp, d, _, dy = setup("tc_clean")
    f = forward(w, d, inp)
    want, _ = backward(w, d, f, dy)
    g = grads(w)
    for n in ("dbias", "db1", "db2", "dgate"):
        g[n] = None
    g, ws = backward(w, d, f, dy, g=g)
    assert B.moe_last_device_status(ws)[0] == 0
    for n, v in g.items():
        if v is not None:
            assert torch.equal(v, want[n]), n


@pytest.mark.parametrize("name", ["tc_top2", "f32"])
def test_an_expert_out_of_range_is_recorded(name):
    w, inp, d, _, dy = setup(name)
    f = forward(w, d, inp)
    for bad in (-1, w.E, 1 << 30):
        idx = f["idx"].clone()
        idx[5, 1] = bad
        _, ws = backward(w, d, dict(f, idx=idx), dy)
        st, det = B.moe_last_device_status(ws)
        assert st == 6 and det == 5 * w.k + 1
    g, ws = backward(w, d, f, dy)
    assert B.moe_last_device_status(ws)[0] == 0

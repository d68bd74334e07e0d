"""Non-finite values that only an expert's weights bring in (the router's
logits are finite): they reach y, are recorded as MOE_ERR_NONFINITE, and stay
with the tokens that use the expert."""
import numpy as np
import pytest
import torch

from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import workloads as wl
from test_gpu_few import _w, run_few, run_threshold
from gpu_harness import to_device

pytestmark = pytest.mark.gpu

NONFINITE = 4
BITS = {"nan": (0x7FC0, np.nan), "inf": (0x7F80, np.inf), "-inf": (0xFF80, -np.inf)}

# One chunk of K (whole tiles of layer 1), sixteen (tiles shared by several
# blocks, joined), and the CUDA cores' types and widths.
SHAPES = {
    "whole_tiles": (64, 512, "bf16"),
    "joined_tiles": (1024, 256, "bf16"),
    "odd_bf16": (66, 130, "bf16"),
    "f32": (64, 128, "f32"),
}
PLACES = [("W1", "nan"), ("b1", "nan"), ("W2", "nan"), ("b2", "nan"), ("b1", "inf"),
          ("b2", "-inf")]


def planted(w, inp, name, value, expert):
    """inp with one value of the expert's array `name` replaced."""
    a = inp[name].copy()
    at = (expert,) + tuple(n // 2 for n in a.shape[1:])
    a[at] = BITS[value][0 if w.dtype == "bf16" else 1]
    return dict(inp, **{name: a})


def check(w, good, res, expert, name):
    """The tokens that kept the expert are not finite and one of them is
    reported; the others' rows are what they were."""
    uses = (good["idx"] == expert).any(dim=1)
    assert uses.any()
    assert res["status"] == NONFINITE
    assert torch.equal(res["idx"], good["idx"])
    assert torch.equal(res["y"][~uses], good["y"][~uses])
    bad = ~torch.isfinite(res["y"][uses].float())
    # A hidden value reaches every column, one of layer 2 its own.
    assert bool((bad.all() if name in ("W1", "b1") else bad.any(dim=1).all()))
    return set(torch.nonzero(uses).flatten().tolist())


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("name,value", PLACES)
def test_few_reports_what_the_experts_bring_in(shape, T, name, value):
    d, d_ff, dtype = SHAPES[shape]
    w = _w(T, d, 6, d_ff, 2, cf=6.0, dtype=dtype)
    inp = wl.generate(w, seed=17, biases=True)
    good = run_few(w, to_device(w, inp))
    assert good["status"] == 0
    e = int(good["idx"][0, 0])
    res = run_few(w, to_device(w, planted(w, inp, name, value, e)))
    assert res["detail"] in check(w, good, res, e, name)  # the combine's: the token


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_few_relu_of_minus_infinity_is_zero(shape, T):
    """A hidden value of -Inf is cut like any other below zero."""
    d, d_ff, dtype = SHAPES[shape]
    w = _w(T, d, 6, d_ff, 2, cf=6.0, dtype=dtype)
    inp = wl.generate(w, seed=17, biases=True)
    e = int(run_few(w, to_device(w, inp))["idx"][0, 0])
    low = inp["b1"].copy()
    low[e, d_ff // 2] = wl.f32_to_bf16_bits(np.float32([-1e30]))[0] if dtype == "bf16" else -1e30
    want = run_few(w, to_device(w, dict(inp, b1=low)))
    res = run_few(w, to_device(w, planted(w, inp, "b1", "-inf", e)))
    assert want["status"] == res["status"] == 0
    assert torch.equal(res["y"], want["y"])


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_threshold_few_reports_what_the_experts_bring_in(shape, T):
    d, d_ff, dtype = SHAPES[shape]
    w = _w(T, d, 6, d_ff, 1, dtype=dtype)
    inp = wl.generate(w, seed=18, biases=True)
    thr = np.full(6, 0.2, np.float32)
    good = run_threshold(w, inp, thr, 6)
    assert good["status"] == 0
    e = int(good["idx"].min())
    for name in ("W1", "b1"):
        res = run_threshold(w, planted(w, inp, name, "nan", e), thr, 6)
        assert res["detail"] in check(w, good, res, e, name)


def test_few_logit_errors_name_their_token_and_expert():
    """A non-finite x makes the token's logits non-finite: the first record is
    of one of them, or of the token's row in the combine."""
    w = _w(6, 64, 8, 128, 2, cf=8.0)
    inp = wl.generate(w, seed=3)
    for bad in (0x7FC0, 0x7F80):
        x = inp["x"].copy()
        x[4, 7] = bad
        res = run_few(w, to_device(w, dict(inp, x=x)))
        assert res["status"] == NONFINITE
        # The logits are recorded behind a grid barrier before the combine.
        assert 4 * w.E <= res["detail"] < 5 * w.E


# ----------------------------------------------------------------------------- the whole layer
LAYERS = {
    "single": (96, 128, 192, "bf16"),
    "pair": (96, 128, 192, "bf16"),
    "odd_bf16": (40, 66, 130, "bf16"),
    "f32": (40, 64, 128, "f32"),
}


def run_layer(w, d):
    cfg = B.config_for(w)
    act = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    y = torch.empty((w.T, w.d), dtype=act, device="cuda")
    idx = torch.empty((w.T, w.k), dtype=torch.int32, device="cuda")
    gate = torch.empty((w.T, w.k), device="cuda")
    ws = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    B.moe_forward(cfg, d["x"], d["Wg"], None, None, None, d["W1"], d["b1"], d["W2"], d["b2"], y,
                  None, ws, idx, gate)
    st, det = B.moe_last_device_status(ws)
    return dict(y=y, idx=idx, gate=gate, ws=ws, status=st, detail=det)


@pytest.mark.parametrize("name,value", PLACES)
@pytest.mark.parametrize("layer", sorted(LAYERS))
def test_layer_reports_what_the_experts_bring_in(monkeypatch, layer, name, value):
    if layer in ("single", "pair"):
        monkeypatch.setenv("MOE_FFN_TC_VARIANT", layer)
    T, d, d_ff, dtype = LAYERS[layer]
    w = _w(T, d, 6, d_ff, 2, cf=6.0, dtype=dtype)
    inp = wl.generate(w, seed=19, biases=True)
    good = run_layer(w, to_device(w, inp))
    assert good["status"] == 0
    e = int(good["idx"][0, 0])
    check(w, good, run_layer(w, to_device(w, planted(w, inp, name, value, e))), e, name)


@pytest.mark.parametrize("layer", sorted(LAYERS))
def test_a_checkpoint_and_its_backward_report_a_nan_of_layer_1(monkeypatch, layer):
    """The NaN that moe_forward's layer 1 makes reaches the checkpoint, whose
    save reports it, and the gradients."""
    if layer in ("single", "pair"):
        monkeypatch.setenv("MOE_FFN_TC_VARIANT", layer)
    T, d, d_ff, dtype = LAYERS[layer]
    w = _w(T, d, 6, d_ff, 2, cf=6.0, dtype=dtype)
    inp = wl.generate(w, seed=20, biases=True)
    cfg = B.config_for(w)
    e = int(run_layer(w, to_device(w, inp))["idx"][0, 0])
    dev = to_device(w, planted(w, inp, "b1", "nan", e))
    f = run_layer(w, dev)
    _, n8, ns = B.moe_checkpoint_size(cfg)
    h8 = torch.empty(n8, dtype=torch.uint8, device="cuda")
    hs = torch.empty(ns, dtype=torch.uint8, device="cuda")
    B.moe_checkpoint_save(cfg, None, None, h8, hs, f["ws"])
    status, detail = B.moe_last_device_status(f["ws"])
    assert status == NONFINITE and (detail % d_ff) // 32 == d_ff // 2 // 32
    # One block of 32 in each of the expert's rows.
    rows = torch.bincount(f["idx"].flatten(), minlength=w.E).cpu()
    marks = (hs.reshape(-1, (d_ff + 31) // 32) == 255).cpu()
    first = int(rows[:e].sum())
    assert int(marks.sum()) == int(rows[e])
    assert bool(marks[first:first + int(rows[e]), d_ff // 2 // 32].all())
    act = f["y"].dtype

    def n(*s, dtype=act):
        return torch.zeros(s, dtype=dtype, device="cuda")
    dW2 = n(w.E, d_ff, d)
    bws = n(B.moe_backward_workspace_size(cfg), dtype=torch.uint8)
    B.moe_backward_checkpoint(cfg, dev["x"], dev["Wg"], None, None, None, dev["W1"], dev["W2"],
                              dev["b2"], f["idx"], f["gate"], h8, hs, torch.ones_like(f["y"]),
                              0.0, 0.0, 0.0, n(T, d), n(d, w.E, dtype=torch.float32), None, None,
                              n(w.E, d, d_ff), None, dW2, None, None, f["ws"], bws)
    assert B.moe_last_device_status(f["ws"])[0] == NONFINITE
    assert not bool(torch.isfinite(dW2[e].float()).all())

"""Gated experts with gate values of both signs, zeros and magnitudes over 1, as
a router other than a softmax gives them."""
import pytest
import torch

import gated_reference as R
import test_gpu_gated as G

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def signed(s, seed):
    """The inputs with gates ~ N(0, 9), some of them +0 and -0."""
    gen = torch.Generator().manual_seed(seed)
    gate = 3 * torch.randn(s["gate"].shape, generator=gen)
    flat = gate.view(-1)
    flat[::5] = 0.0
    flat[3::10] = -0.0
    flat[1] = -7.5
    return dict(s, gate=gate)


def magnitudes(s):
    return dict(s, gate=s["gate"].abs())


def widened(name, value, err):
    """The reference's bounds hold for gates >= 0: every term but the last
    rounding's is linear in the gates' magnitudes, so the bound for them, with
    half a step of the value that the signs give, holds here."""
    step = R.STEP[BF16] if name == "bf16" else R.STEP[F32]
    return err + step * value.abs()


def check_forward(s, o, ref, ref_abs):
    t = "bf16" if s["x"].dtype == BF16 else "f32"
    assert G.B.moe_last_device_status(o["ws"])[0] == 0
    G.close("y", o["y"], ref["y"], widened(t, ref["y"], ref_abs["y_err"]))


FORMS = [(3, BF16, 128, 256, 4, 2, ""), (40, BF16, 512, 768, 8, 2, ""),
         (400, BF16, 128, 256, 4, 3, ""), (700, BF16, 256, 576, 2, 2, "pair"),
         (300, BF16, 128, 320, 9, 6, ""), (3, F32, 34, 66, 4, 2, ""),
         (517, F32, 130, 234, 6, 3, ""), (2300, F32, 72, 100, 4, 2, ""),
         (30, BF16, 36, 50, 4, 2, ""), (400, BF16, 36, 50, 4, 2, "")]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_gates_of_any_sign(form, monkeypatch):
    """Values and gradients; dgate does not carry the gate, so it has the bits
    that the gates' magnitudes, or ones, give."""
    T, dt, d, F, E, k, variant = form
    if variant:
        monkeypatch.setenv("MOE_FFN_TC_VARIANT", variant)
        monkeypatch.setenv("MOE_BWD_TC_VARIANT", variant)
    s = signed(G.inputs(T, d, E, F, k, dt, seed=T), T)
    a = magnitudes(s)
    cfg, g = G.config(s, 2.0), G.dev(s)
    t = "bf16" if dt == BF16 else "f32"
    for kind in (R.SILU, R.GELU, R.RELU):
        ref, ref_abs = (G.reference(cfg, kind, v) for v in (s, a))
        o = G.run_forward(cfg, kind, g)
        check_forward(s, o, ref, ref_abs)
        b = G.run_backward(cfg, kind, g, o["p1"], o["p3"])
        assert G.B.moe_last_device_status(b["ws"])[0] == 0
        p = (o["p1"], o["p3"])
        want, _ = R.backward(kind, s["x"], s["idx"], s["gate"], *p, s["W1"], s["W3"], s["W2"],
                             s["b2"], s["dy"], G.cap(cfg))
        _, err = R.backward(kind, a["x"], a["idx"], a["gate"], *p, a["W1"], a["W3"], a["W2"],
                            a["b2"], a["dy"], G.cap(cfg))
        for n in ("dx", "dW1", "dW3", "dW2", "db1", "db3", "db2"):
            G.close(n, b[n], want[n], widened(t, want[n], err[n]))
        G.close("dgate", b["dgate"], want["dgate"], err["dgate"])
        ones = dict(g, gate=torch.ones_like(g["gate"]))
        c = G.run_backward(cfg, kind, ones, *p)
        assert torch.equal(c["dgate"], b["dgate"])


@pytest.mark.parametrize("T,d,F,k", [(3, 128, 256, 2), (40, 200, 330, 3), (400, 128, 256, 2),
                                     (300, 130, 234, 6)])
def test_gates_of_any_sign_in_8_bits(T, d, F, k):
    s = signed(G.inputs(T, d, 7, F, k, BF16, seed=T), T)
    cfg, g = G.config(s, 2.0), G.dev(s)
    w8 = [G.quantise(g, n, BF16) for n in ("W1", "W3", "W2")]
    ref, ref_abs = (G.reference8(cfg, R.SILU, v, w8) for v in (s, magnitudes(s)))
    check_forward(s, G.run_fp8(cfg, R.SILU, g, w8), ref, ref_abs)


def test_zero_gates_alone():
    """Every gate zero: y is x, dx is dy, no weight or bias has a gradient, and
    dgate still is what a first step away from zero would follow."""
    for T, dt, d, F in ((3, BF16, 128, 256), (400, BF16, 128, 256), (3, F32, 34, 66),
                        (400, F32, 34, 66)):
        s = G.inputs(T, d, 4, F, 2, dt, seed=T)
        s["gate"].zero_()
        cfg, g = G.config(s, 4.0), G.dev(s)
        o = G.run_forward(cfg, R.SILU, g)
        assert torch.equal(o["y"].cpu(), s["x"])
        b = G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
        assert torch.equal(b["dx"].cpu(), s["dy"])
        for n in ("dW1", "dW3", "dW2", "db1", "db3", "db2"):
            assert not bool(b[n].any()), n
        want, err = R.backward(R.SILU, s["x"], s["idx"], s["gate"], o["p1"], o["p3"], s["W1"],
                               s["W3"], s["W2"], s["b2"], s["dy"], G.cap(cfg))
        G.close("dgate", b["dgate"], want["dgate"], err["dgate"])
        assert bool((b["dgate"] != 0).any())

"""CPU checks: the reference of the checkpointed backward against differences
of its loss, the format's properties, and the host-side refusals."""
import ctypes

import numpy as np
import pytest

import checkpoint_reference as ref
import few_reference as few
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import build as moe_build
from sparsely_gated_mixture_gb300 import workloads as wl


@pytest.mark.parametrize("mode,k,noisy", [(wl.TOPK, 2, True), (wl.TOPK, 4, True),
                                          (wl.TOPK, 3, False), (wl.SWITCH, 1, True),
                                          (wl.SWITCH, 1, False)])
def test_router_gradients_against_differences(mode, k, noisy):
    """Central differences (step 1e-6: truncation ~1e-12, rounding of L at
    2^-53 |L| / 1e-6 ~ 1e-9) of L in W_g, W_noise, the bias and x."""
    w = wl.Workload("fd", T=9, d=5, E=4, d_ff=6, k=k, cf=1.0, mode=mode, dtype="f32", noisy=noisy)
    inp = wl.generate(w, seed=k, biases=True)
    inp["bias"] = np.linspace(-0.3, 0.4, 4).astype(np.float32)
    for n in ("x", "Wg", "Wn", "noise", "bias", "W2", "b2", "W1"):
        inp[n] = None if inp[n] is None else inp[n].astype(np.float64)
    _, _, _, H = ref.gate_state(inp, "f32")
    idx = few.topk(H, k)
    gate = few.gates(H, idx, mode)
    _, keep = few.slots(idx, 4, few.capacity(9, 4, k, 1.0))
    rng = np.random.default_rng(1)
    dy = rng.standard_normal((9, 5))
    h = np.maximum(rng.standard_normal((9, k, 6)), 0)
    weights = (0.3, 0.4, 0.5)
    g, _, order = ref.backward(inp, "f32", mode, idx, gate, keep, h, dy, weights)

    def L():
        return ref.loss(inp, "f32", mode, idx, keep, h, dy, weights, order)
    # x reaches L through the experts' rows too: h is held here, so the
    # experts' share and the residual leave dx before the comparison.
    dx = g["dx"] - dy
    for t in range(9):
        for j in range(k):
            if keep[t, j]:
                e = idx[t, j]
                dx[t] -= inp["W1"][e] @ (gate[t, j] * (inp["W2"][e] @ dy[t]) * (h[t, j] > 0))
    for name, grad in (("Wg", g["dWg"]), ("Wn", g["dWn"]), ("bias", g["dbias"]), ("x", dx)):
        if inp[name] is None:
            continue
        for at in np.ndindex(inp[name].shape):
            v = inp[name][at]
            inp[name][at] = v + 1e-6
            up = L()
            inp[name][at] = v - 1e-6
            down = L()
            inp[name][at] = v
            assert abs((up - down) / 2e-6 - grad[at]) <= 1e-7 * (1 + abs(grad[at])), (name, at)


def test_format_properties():
    rng = np.random.default_rng(0)
    h = np.maximum(rng.standard_normal((40, 70)), 0) * np.exp2(rng.integers(-100, 100, (40, 1)))
    h[0] = 0
    h[1, 3] = 2.0 ** -133
    q, s, v = ref.quantise(h)
    assert np.array_equal(v > 0, h > 0)
    top = np.concatenate([h, np.zeros((40, 26))], 1).reshape(40, 3, 32).max(axis=2)
    lim = np.repeat(2.0 ** (s.astype(float) - 127), 32, 1)[:, :70]
    assert np.all(np.abs(v - h) <= np.maximum(2.0 ** -4 * h, 2.0 ** -9 * lim))
    assert np.all(448 * 2.0 ** (s.astype(float) - 127) >= top)
    bf = few.f64(wl.f32_to_bf16_bits(v.astype(np.float32)), "bf16")
    assert np.array_equal(bf, v)  # loading into bf16 rounds nothing


F = 1 << 20  # a pointer that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.lib()


def test_sizes(lib):
    cfg = B.config(64, 64, 8, 100, 2, 1.0)
    assert B.moe_checkpoint_size(cfg) == (128, 12800, 128 * 4)
    assert B.moe_checkpoint_size(B.config(64, 64, 8, 96, 2, 0.5)) == (64, 64 * 96, 64 * 3)
    assert lib.moe_checkpoint_size(ctypes.byref(cfg), None, None, None) == 1
    with pytest.raises(B.MoEError):
        B.moe_checkpoint_size(B.config(64, 64, 8, 0, 2, 0.5))


def test_sizes_past_the_kernels_counts_refused(lib):
    n = ctypes.c_int64()
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    rows = 1 << 26  # of 64 blocks of 32
    for cfg, status in ((B.config(1, 8, 1, (1 << 30) + 8, 1, 1.0), 2),
                        (B.config(rows, 8, 1, 2048, 1, 1.0), 2),
                        (B.config(rows - 2, 8, 1, 2048, 1, 1.0), 0),
                        (B.config(rows, 8, 1, 2016, 1, 1.0), 0)):
        assert lib.moe_checkpoint_size(ctypes.byref(cfg), ctypes.byref(n), ctypes.byref(a),
                                       ctypes.byref(b)) == status
    cfg = B.config(rows, 8, 1, 2048, 1, 1.0)
    assert lib.moe_checkpoint_save(ctypes.byref(cfg), F, F, F, F, F, None) == 2
    assert lib.moe_checkpoint_load(ctypes.byref(cfg), F, F, F, F, F, None) == 2


@pytest.mark.parametrize("bad", [{0: None}, {1: None}, {2: None}, {3: None}, {4: None},
                                 {4: F + 16}, {0: F + 4}, {2: F + 1}])
def test_save_pointers_rejected(lib, bad):
    args = [F, F, F, F, F, None]  # hbuf, expert_offset, h8, hscale, ws, stream
    for i, v in bad.items():
        args[i] = v
    cfg = B.config(64, 64, 8, 100, 2, 1.0)
    assert lib.moe_checkpoint_save(ctypes.byref(cfg), *args) == 1


@pytest.mark.parametrize("bad", [{0: None}, {1: None}, {2: None}, {3: None}, {4: None},
                                 {4: F + 16}, {3: F + 4}])
def test_load_pointers_rejected(lib, bad):
    args = [F, F, F, F, F, None]  # h8, hscale, expert_offset, hbuf, ws, stream
    for i, v in bad.items():
        args[i] = v
    cfg = B.config(64, 64, 8, 100, 2, 1.0)
    assert lib.moe_checkpoint_load(ctypes.byref(cfg), *args) == 1


@pytest.mark.parametrize("bad", [
    {0: None}, {1: None}, {2: F}, {5: None}, {6: None}, {8: None}, {9: None}, {10: None},
    {11: None}, {12: None}, {13: float("nan")}, {15: float("inf")}, {16: None}, {17: None},
    {18: F}, {20: None}, {22: None}, {25: None}, {26: None}, {26: F + 64}, {21: F + 4}])
def test_backward_pointers_rejected(lib, bad):
    #       x  Wg Wn    noise bias W1 W2 b2    idx gate h8 hs dy
    args = [F, F, None, None, None, F, F, None, F, F, F, F, F, 0.0, 0.0, 0.0,
            # dx dWg dWn dbias dW1 db1  dW2 db2  dgate ws bws stream
            F, F, None, None, F, None, F, None, None, F, F, None]
    for i, v in bad.items():
        args[i] = v
    cfg = B.config(64, 64, 8, 100, 2, 1.0)
    assert lib.moe_backward_checkpoint(ctypes.byref(cfg), *args) == 1


def test_wrappers_raise(lib):
    cfg = B.config(64, 64, 8, 100, 2, 1.0)
    for call in (lambda: B.moe_checkpoint_save(cfg, F, None, F, F, F, stream=0),
                 lambda: B.moe_checkpoint_load(cfg, F, F, None, F, F, stream=0),
                 lambda: B.moe_backward_checkpoint(
                     cfg, F, F, None, None, None, F, F, None, None, F, F, F, F, 0, 0, 0, F, F,
                     None, None, F, None, F, None, None, F, F, stream=0)):
        with pytest.raises(B.MoEError):
            call()

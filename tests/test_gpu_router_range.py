"""Router weights that are finite in fp32 but round to Inf in bf16 (from
3.3962e38 on): the routers that write a weight as three bf16 numbers keep it
finite."""
import numpy as np
import pytest
import torch

from gpu_harness import to_device
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import workloads as wl
from test_gpu_few import _w, run_few

pytestmark = pytest.mark.gpu

ROUNDS_UP = 3.3961775292304601e38  # halfway from the largest bf16 number to the next


def inputs(w):
    """One column of x is 2^-118, the others zero; the weights that it meets
    are the largest floats, in steps of 2^116, negative for odd experts. So
    each logit is one product, exact in fp32, some multiple of 1/4."""
    inp = wl.generate(w, seed=1)
    x = np.zeros((w.T, w.d), np.float32)
    x[:, 5] = 2.0 ** -118
    inp["x"] = wl.f32_to_bf16_bits(x)
    e = np.arange(w.E)
    big = (np.float64(np.finfo(np.float32).max) - (e % 6) * 2.0 ** 116).astype(np.float32)
    assert big.min() > ROUNDS_UP
    inp["Wg"] = inp["Wg"].copy()
    inp["Wg"][5] = np.where(e % 2 == 0, big, -big)
    H = inp["Wg"][5].astype(np.float64) * 2.0 ** -118
    order = np.argsort(-H, kind="stable")[: w.k]
    g = np.exp(H[order] - H[order[0]])
    return inp, order, g / g.sum()


def check(w, idx, gate, order, want):
    assert np.array_equal(idx, np.tile(order.astype(np.int32), (w.T, 1)))
    # Logits of 1024 in fp32 sums of d terms, k exponentials and their sum.
    rel = 2 * (w.d + 2) * 2.0 ** -24 * 1024 + (w.k + 16) * 2.0 ** -24
    assert np.all(np.abs(gate - want) <= rel * want)


@pytest.mark.parametrize("T", [1, 40])
def test_few(T):
    w = _w(T, 64, 12, 64, 4, cf=12.0)
    inp, order, want = inputs(w)
    res = run_few(w, to_device(w, inp))
    assert res["status"] == 0
    check(w, res["idx"].cpu().numpy(), res["gate"].double().cpu().numpy(), order, want)


@pytest.mark.parametrize("E", [8, 12, 200])
def test_gate(E):
    w = wl.Workload("r", T=300, d=64, E=E, d_ff=64, k=4, cf=1.0, mode=wl.TOPK, dtype="bf16",
                    noisy=False)
    inp, order, want = inputs(w)
    d = to_device(w, inp)
    cfg = B.config_for(w)
    idx = torch.empty((w.T, w.k), dtype=torch.int32, device="cuda")
    gate = torch.empty((w.T, w.k), device="cuda")
    thr = torch.empty((w.T, 2), device="cuda")
    ws = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    B.moe_gate(cfg, d["x"], d["Wg"], None, None, None, idx, gate, thr, ws)
    assert B.moe_last_device_status(ws)[0] == 0
    check(w, idx.cpu().numpy(), gate.double().cpu().numpy(), order, want)

"""Infinite pre-activations in the gated experts: an Inf stays what the formulas
make of it, whichever kernels a size, a type or a width takes."""
import pytest
import torch

import gated_reference as R
import test_gpu_gated as G
from sparsely_gated_mixture_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# A few rows and more, on the tensor cores and on the CUDA cores in either type;
# 600 rows of 576 also through a pair of CTAs.
FORMS = [(3, BF16, 128, 256, "single"), (400, BF16, 128, 256, "single"),
         (600, BF16, 256, 576, "pair"), (3, F32, 34, 66, "single"), (400, F32, 34, 66, "single"),
         (3, BF16, 36, 50, "single"), (400, BF16, 36, 50, "single")]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kind", [R.SILU, R.GELU, R.RELU])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_an_infinite_pre_activation(form, kind, sign, monkeypatch):
    """p1 = +-Inf in one column of one expert, with p3 finite and positive there:
    act(+Inf) is Inf for all three, so y is an Inf of W2's sign; act(-Inf) is 0
    for ReLU and by the formulas 0 * Inf, a NaN, for the others. Tokens without
    that expert keep their bits."""
    T, dt, d, F, variant = form
    monkeypatch.setenv("MOE_FFN_TC_VARIANT", variant)
    s = G.inputs(T, d, 4, F, 2, dt, seed=T + kind)
    s["idx"][0] = torch.tensor([1, 2], dtype=torch.int32)
    s["idx"][1] = torch.tensor([0, 3], dtype=torch.int32)
    s["b3"][1, 5] = 50.0
    W2 = s["W2"][1, 5]
    W2[W2 == 0] = 0.5
    cfg = G.config(s, 4.0)
    plain = G.run_forward(cfg, kind, G.dev(s))
    s["b1"][1, 5] = sign * float("inf")
    o = G.run_forward(cfg, kind, G.dev(s))
    want = G.reference(cfg, kind, s)["y"]
    got = o["y"].cpu().double()
    hit = (s["idx"] == 1).any(1)
    assert torch.equal(o["y"].cpu()[~hit], plain["y"].cpu()[~hit])
    if sign > 0:
        assert bool(torch.isinf(want[hit]).all())
    elif kind != R.RELU:
        assert bool(torch.isnan(want[hit]).all())
    for what in (torch.isposinf, torch.isneginf, torch.isnan):
        assert torch.equal(what(got), what(want)), what.__name__
    finite = sign < 0 and kind == R.RELU
    assert B.moe_last_device_status(o["ws"])[0] == (0 if finite else 4)
    # The pre-activations themselves are kept as they are.
    pre = o["p1"].float().cpu()
    assert int(torch.isinf(pre).sum()) == int((s["idx"] == 1).sum())
    assert not bool(torch.isnan(pre).any())

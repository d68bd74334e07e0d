"""Host-side checks of the gated experts' entry points: sizes and refusals, with
pointers that are never dereferenced (the checks fail first)."""
import ctypes

import pytest
import torch

import gated_reference as R
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import build as moe_build

F = 1 << 20  # a well-aligned address


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.lib()


def size(lib, name, cfg):
    n = ctypes.c_size_t()
    return getattr(lib, name)(ctypes.byref(cfg), ctypes.byref(n)), n.value


SIZES = ["moe_gated_workspace_size", "moe_gated_backward_workspace_size",
         "moe_gated_fp8_workspace_size"]


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("field,value,status", [
    ("k", 0, 1), ("k", 17, 1), ("E", 0, 1), ("T", 0, 1), ("capacity_factor", 0.0, 1),
    ("act_dtype", 5, 1), ("min_capacity", 0, 1), ("E", 2048, 2), ("d", 524289, 2),
    ("d_ff", 524289, 2), ("d", 0, 1), ("d_ff", -1, 1)])
def test_bad_config(lib, name, field, value, status):
    cfg = B.config(64, 32, 16, 64, 2, 1.0)
    setattr(cfg, field, value)
    assert size(lib, name, cfg)[0] == status


def test_sizes(lib):
    for name in SIZES:
        small, large = (size(lib, name, B.config(T, 64, 8, 128, 2, 1.0)) for T in (600, 4096))
        assert small[0] == large[0] == 0 and 0 < small[1] < large[1]
        assert getattr(lib, name)(ctypes.byref(B.config(16, 64, 8, 128, 2, 1.0)), None) == 1
    # Too many warps of 128 columns.
    wide = B.config(1 << 20, 64, 2, 524288, 2, 2.0)
    assert size(lib, SIZES[0], wide)[0] == 2
    f32 = B.config(16, 64, 8, 128, 2, 1.0, act_dtype=B.MOE_F32)
    assert size(lib, "moe_gated_fp8_workspace_size", f32)[0] == 2
    # Rows beyond the capacity take no room.
    kept = B.config(4096, 64, 8, 128, 2, 0.25)
    assert size(lib, SIZES[0], kept)[1] < large[1]


def forward_args():
    return [B.MOE_ACT_SILU, F, F, F, F, None, F, None, F, None, F, None, None, None, None, F, None]


def backward_args():
    return [B.MOE_ACT_SILU] + [F] * 8 + [F] * 10 + [F, None]


def fp8_args():
    return [B.MOE_ACT_SILU, F, F, F, F, F, None, F, F, None, F, F, None, F, None, None, F, None]


REQUIRED = {
    "moe_experts_gated": (forward_args, [1, 2, 3, 4, 6, 8, 10, 15], [5, 7, 9, 13, 14]),
    "moe_experts_gated_backward": (backward_args, [1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 12, 13, 15, 17,
                                                   19], [9, 14, 16, 18]),
    "moe_experts_gated_fp8": (fp8_args, [1, 2, 3, 4, 5, 7, 8, 10, 11, 13, 16], [6, 9, 12, 14, 15]),
}


@pytest.mark.parametrize("name", sorted(REQUIRED))
def test_pointers(lib, name):
    make, required, optional = REQUIRED[name]
    cfg = B.config(64, 32, 16, 64, 2, 1.0)
    call = getattr(lib, name)
    for i in required:
        for bad in (None, F + 8):
            args = make()
            args[i] = bad
            assert call(ctypes.byref(cfg), *args) == 1, (i, bad)
    for i in optional:
        args = make()
        args[i] = F + 8
        assert call(ctypes.byref(cfg), *args) == 1, i
    for activation in (-1, 3):
        args = make()
        args[0] = activation
        assert call(ctypes.byref(cfg), *args) == 1
    assert call(None, *make()) == 1


def test_pre_activations_come_in_pairs(lib):
    cfg = B.config(64, 32, 16, 64, 2, 1.0)
    for i in (11, 12):
        args = forward_args()
        args[i] = F
        assert lib.moe_experts_gated(ctypes.byref(cfg), *args) == 1


def test_fp8_layer_is_bf16(lib):
    cfg = B.config(64, 32, 16, 64, 2, 1.0, act_dtype=B.MOE_F32)
    assert lib.moe_experts_gated_fp8(ctypes.byref(cfg), *fp8_args()) == 2


@pytest.mark.parametrize("E,K,N,status", [
    (0, 8, 8, 1), (1, 0, 8, 1), (1, 8, -3, 1), (1025, 8, 8, 2), (1, 524289, 8, 2),
    (1, 8, 524289, 2), (3, 130, 257, 0)])
def test_weights_fp8_size(lib, E, K, N, status):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_weights_fp8_size(E, K, N, ctypes.byref(a), ctypes.byref(b)) == status
    if status == 0:
        assert (a.value, b.value) == (3 * 257 * 256, 3 * 3 * 2)
        assert B.moe_weights_fp8_size(E, K, N) == (a.value, b.value)
        assert lib.moe_weights_fp8_size(E, K, N, None, ctypes.byref(b)) == 1
    assert lib.moe_weights_fp8(E, K, N, 7, F, F, F, F, None) == (status or 1)
    for i in range(4):
        for bad in (None, F + 8):
            args = [F, F, F, F, None]
            args[i] = bad
            assert lib.moe_weights_fp8(E, K, N, 1, *args) == (status or 1)


# ----------------------------------------------------------------------------- the reference itself
def test_reference_gradients_are_differences():
    """The formulas of the backward against central differences of the forward."""
    g = torch.Generator().manual_seed(1)
    T, d, E, Fh, k, C = 5, 6, 3, 7, 2, 4

    def normal(*s):
        return torch.randn(s, generator=g, dtype=torch.float32)
    x, W1, W3, W2 = normal(T, d), normal(E, d, Fh), normal(E, d, Fh), normal(E, Fh, d)
    b1, b3, b2, dy = normal(E, Fh), normal(E, Fh), normal(E, d), normal(T, d)
    idx = torch.tensor([[0, 1], [1, 1], [2, 0], [1, 0], [1, 2]], dtype=torch.int32)
    gate = torch.rand((T, k), generator=g)
    for kind in (R.SILU, R.GELU, R.RELU):
        def loss(**kw):
            a = dict(x=x, gate=gate, W1=W1, b1=b1, W3=W3, b3=b3, W2=W2, b2=b2)
            a.update(kw)
            y = R.forward(kind, a["x"], idx, a["gate"], a["W1"], a["b1"], a["W3"], a["b3"],
                          a["W2"], a["b2"], C)["y"]
            return float((y * dy).sum())
        # In 64 bits throughout: a tensor of the reference's own type.
        R.STEP[torch.float64] = 0.0
        x, W1, W3, W2, b1, b3, b2, gate = (v.double() for v in (x, W1, W3, W2, b1, b3, b2, gate))
        f = R.forward(kind, x, idx, gate, W1, b1, W3, b3, W2, b2, C)
        out, _ = R.backward(kind, x, idx, gate, f["pre"][0], f["pre"][1], W1, W3, W2, b2, dy, C)
        eps = 1e-5
        for name, v in dict(x=x, gate=gate, W1=W1, b1=b1, W3=W3, b3=b3, W2=W2, b2=b2).items():
            for i in range(0, v.numel(), max(1, v.numel() // 7)):
                hi, lo = v.clone(), v.clone()
                hi.view(-1)[i] += eps
                lo.view(-1)[i] -= eps
                diff = (loss(**{name: hi}) - loss(**{name: lo})) / (2 * eps)
                got = float(out["d" + name].reshape(-1)[i])
                # Differences: O(eps^2) curvature and 1e-16 * |loss| / eps of rounding.
                assert abs(diff - got) < 1e-6 * (1 + abs(got)), (kind, name, i)


def test_reference_8_bits():
    table = R.e4m3_table()
    assert table[0] == 0 and table[1] == 2.0 ** -9 and table[126] == 448 and len(table) == 127
    q, sc = R.weights8(torch.tensor([[[448.0, -3.0], [0.0, 17.0]]]))
    assert sc.tolist() == [[[127]]]
    assert R.values8(q[0], sc[0], 2).tolist() == [[448.0, -3.0], [0.0, 16.0]]  # 17: a tie, to even
    q, sc = R.weights8(torch.tensor([[[449.0]]]))
    assert sc.tolist() == [[[128]]] and R.values8(q[0], sc[0], 1).tolist() == [[448.0]]

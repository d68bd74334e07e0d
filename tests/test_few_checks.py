"""Host-side checks of the few-token entry points (no GPU work is enqueued)."""
import ctypes

import pytest

from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import build as moe_build


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.lib()


F = 1 << 20  # a pointer that is never dereferenced: the checks fail first


def test_workspace_sizes(lib):
    small = B.moe_few_workspace_size(B.config(1, 64, 8, 128, 2, 1.0))
    assert 0 < small < B.moe_few_workspace_size(B.config(64, 64, 8, 128, 2, 1.0))
    n = ctypes.c_size_t()
    for cfg, status in ((B.config(65, 64, 8, 128, 2, 1.0), 2), (B.config(0, 64, 8, 128, 2, 1.0), 1),
                        (B.config(4, 64, 8, 128, 9, 1.0), 1),
                        (B.config(4, 64, 32, 128, 17, 1.0), 2),
                        (B.config(4, 64, 8, 524288 + 8, 2, 1.0), 2),
                        (B.config(4, 524288 + 8, 8, 64, 2, 1.0), 2)):
        assert lib.moe_few_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == status
    assert lib.moe_few_workspace_size(ctypes.byref(B.config(1, 64, 8, 128, 2, 1.0)), None) == 1


def test_workspace_holds_the_cuda_cores_partial_sums(lib):
    """Up to 8 slices of K of both products, whatever share of the rows the
    experts get (widths that the tensor cores do not take)."""
    for act, d, d_ff in ((B.MOE_BF16, 4098, 2050), (B.MOE_F32, 8192, 4096)):
        cfg = B.config(64, d, 16, d_ff, 16, 1.0, act_dtype=act)
        assert B.moe_few_workspace_size(cfg) >= 8 * 64 * 16 * (d + d_ff) * 4


def test_workspace_of_the_cuda_cores_holds_no_hidden_rows(lib):
    """They make the hidden rows of layer 1's partial sums where they read them:
    what grows with d_ff are the 8 partial sums of each of its values alone."""
    for act, d, d_ff, step in ((B.MOE_BF16, 66, 130, 4098), (B.MOE_F32, 64, 128, 4096)):
        size = [B.moe_few_workspace_size(B.config(64, d, 16, n, 16, 1.0, act_dtype=act))
                for n in (d_ff, d_ff + step)]
        assert size[1] - size[0] <= 8 * 64 * 16 * step * 4 + 256


@pytest.mark.parametrize("bad", [
    {0: None}, {0: F + 8}, {1: None}, {2: F}, {3: F}, {4: F + 4}, {5: None}, {6: F + 2}, {7: None},
    {9: None}, {10: F + 4}, {11: F + 4}, {12: F + 4}, {13: F + 1}, {14: None}, {14: F + 16}])
def test_few_pointers_rejected(lib, bad):
    cfg = B.config(16, 64, 8, 128, 2, 1.0)
    #       x  Wg Wn    noise bias W1 b1   W2 b2    y  idx   gate  pos   keep  ws stream
    args = [F, F, None, None, None, F, None, F, None, F, None, None, None, None, F, None]
    for i, v in bad.items():
        args[i] = v
    assert lib.moe_forward_few(ctypes.byref(cfg), *args) == 1


def test_few_refuses_larger_batches(lib):
    args = [F, F, None, None, None, F, None, F, None, F, None, None, None, None, F, None]
    assert lib.moe_forward_few(ctypes.byref(B.config(65, 64, 8, 128, 2, 1.0)), *args) == 2
    args = [F, F, None, F, F, None, F, None, F, None, None, None, F, None]
    assert lib.moe_forward_threshold_few(ctypes.byref(B.config(65, 64, 8, 128, 2, 1.0)), *args) == 2


@pytest.mark.parametrize("bad", [{0: None}, {1: None}, {2: F + 4}, {3: None}, {4: None}, {6: None},
                                 {8: None}, {9: F + 4}, {10: F + 4}, {11: F + 4}, {12: F + 128}])
def test_threshold_few_pointers_rejected(lib, bad):
    cfg = B.config(16, 64, 8, 128, 2, 1.0)
    #       x  Wg bias  thr W1 b1   W2 b2    y  idx   gate  mask  ws stream
    args = [F, F, None, F, F, None, F, None, F, None, None, None, F, None]
    for i, v in bad.items():
        args[i] = v
    assert lib.moe_forward_threshold_few(ctypes.byref(cfg), *args) == 1


def test_wrappers_raise(lib):
    cfg = B.config(16, 64, 8, 128, 2, 1.0)
    with pytest.raises(B.MoEError):
        B.moe_forward_few(cfg, None, F, None, None, None, F, None, F, None, F, F, stream=0)
    with pytest.raises(B.MoEError):
        B.moe_forward_threshold_few(cfg, F, F, None, None, F, None, F, None, F, F, stream=0)
    with pytest.raises(B.MoEError):
        B.moe_few_workspace_size(B.config(65, 64, 8, 128, 2, 1.0))

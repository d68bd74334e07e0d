"""The largest batches that the gated experts take (no GPU: sizes and refusals)."""
import ctypes

import pytest

import test_gated_checks as C
from sparsely_gated_mixture_gb300 import binding as B
from test_gated_checks import lib  # noqa: F401  (the fixture)

MOST = 2 ** 31 - 1024
INT_MAX = 2 ** 31 - 1


def config(T, k=1, E=1, cf=2.0, act=B.MOE_F32):
    return B.config(T, 1, E, 1, k, cf, act_dtype=act)


@pytest.mark.parametrize("name", C.SIZES)
@pytest.mark.parametrize("T,k,cf,status", [
    (MOST, 1, 2.0, 0), (MOST + 1, 1, 2.0, 2), (INT_MAX, 1, 2.0, 2),
    (MOST // 8, 8, 8.0, 0), (INT_MAX // 8, 8, 8.0, 2),
    # Rows count, not choices: the capacity leaves half of them.
    (INT_MAX, 1, 0.5, 0)])
def test_rows_of_a_call(lib, name, T, k, cf, status):  # noqa: F811
    act = B.MOE_BF16 if name == "moe_gated_fp8_workspace_size" else B.MOE_F32
    assert C.size(lib, name, config(T, k, E=k, cf=cf, act=act))[0] == status


@pytest.mark.parametrize("name", sorted(C.REQUIRED))
def test_calls_refuse_it_too(lib, name):  # noqa: F811
    act = B.MOE_BF16 if name == "moe_experts_gated_fp8" else B.MOE_F32
    assert getattr(lib, name)(ctypes.byref(config(INT_MAX, act=act)), *C.REQUIRED[name][0]()) == 2


def test_a_slice_of_the_rows_in_32_bits():
    """Why: a weight gradient's slices of an expert's rows and the bias gradients'
    strides over them are counted in 32 bits. Sixteen slices in steps of 16, and
    strides of 64 x 2 rows with eight in flight, stay below 2^31 for MOST rows
    and not for the largest int."""
    def over(rows):
        a_slice = rows + 16 - 1
        column_sum = rows - 1 + 64 * 2 + 7 * 8 * 2
        a_row = rows - 1 + 256
        return max(a_slice, column_sum, a_row) > INT_MAX
    assert not over(MOST) and over(INT_MAX)

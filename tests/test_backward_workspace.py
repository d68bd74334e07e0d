"""The backward's workspace (no GPU): it keeps within the sizes that callers of
moe_backward reserved before its bias gradients went into one launch."""
import pytest

from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import build as moe_build

# bytes: T, d, E, d_ff, k, capacity factor, element type
SIZES = [
    (1186120448, 8192, 4096, 8, 14336, 2, 1.25, B.MOE_BF16),
    (117392128, 4096, 512, 16, 1024, 4, 2.0, B.MOE_BF16),
    (1559781632, 32768, 512, 1024, 1024, 4, 1.5, B.MOE_BF16),
    (271124224, 16384, 768, 64, 2048, 1, 1.25, B.MOE_BF16),
    (129280, 1, 64, 3, 64, 2, 1.0, B.MOE_BF16),
    (5215744, 517, 130, 6, 234, 3, 2.0, B.MOE_F32),
    (44220672, 64, 64, 1024, 64, 16, 1.0, B.MOE_BF16),
    (38763776, 100, 8192, 4, 64, 1, 4.0, B.MOE_F32),
    (37030656, 2048, 64, 1, 8192, 1, 1.0, B.MOE_BF16),
]


@pytest.mark.parametrize("row", SIZES, ids=lambda r: "x".join(map(str, r[1:6])))
def test_no_larger_than_before(row):
    moe_build.build()
    n, T, d, E, d_ff, k, cf, act = row
    assert B.moe_backward_workspace_size(B.config(T, d, E, d_ff, k, cf, act_dtype=act)) <= n

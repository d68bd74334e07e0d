"""Workspace sizes that do not depend on the process that asks for them: what a
planning process without a GPU is told holds for the one that makes the call."""
import json
import os
import subprocess
import sys

import pytest

from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import build as moe_build

# T, d, E, d_ff, k, capacity factor, element type
CONFIGS = [(4246, 96, 3, 208, 3, 2.0, B.MOE_F32), (517, 130, 6, 234, 3, 1.1, B.MOE_F32),
           (5019, 181, 5, 683, 4, 2.0, B.MOE_F32), (2300, 33, 4, 1, 2, 4.0, B.MOE_BF16),
           (40, 72, 3, 100, 2, 100.0, B.MOE_BF16), (4096, 512, 16, 1024, 4, 2.0, B.MOE_BF16),
           (64, 4096, 8, 14336, 2, 4.0, B.MOE_BF16), (1, 64, 4, 128, 2, 2.0, B.MOE_BF16),
           (8192, 2, 4, 2, 1, 4.0, B.MOE_F32)]
SIZES = ["moe_workspace_size", "moe_gated_workspace_size", "moe_gated_backward_workspace_size",
         "moe_gated_fp8_workspace_size", "moe_few_workspace_size"]


def sizes():
    out = {}
    for c in CONFIGS:
        cfg = B.config(*c[:6], act_dtype=c[6])
        for name in SIZES:
            if name == "moe_gated_fp8_workspace_size" and c[6] != B.MOE_BF16:
                continue
            if name == "moe_few_workspace_size" and c[0] > 64:
                continue
            out[f"{name} {c}"] = getattr(B, name)(cfg)
    return out


def rounded(*parts):
    return sum((p + 255) // 256 * 256 for p in parts)


@pytest.mark.parametrize("T,d,E,F,k,dg,slices", [
    # Of 152 SMs: 72 tiles of 64 x 64, so slices of an expert's rows make four
    # blocks an SM; dgate's partials for every 64 columns.
    (4246, 96, 3, 208, 3, 4, 9),
    # 180 tiles of 128 x 128 in four slices; D's tiles of that size give every SM two.
    (5019, 181, 5, 683, 4, 6, 4)])
def test_sized_for_the_gpu(T, d, E, F, k, dg, slices):
    """The gated backward's rows, dgate's partials and the weight gradients'
    slices, as the launches on 152 SMs use them."""
    moe_build.build()
    cfg = B.config(T, d, E, F, k, 2.0, act_dtype=B.MOE_F32)
    R = T * k
    part = 12 * slices * E * d * F if slices > 1 else 0
    least = rounded(4 * R * d, 4 * R * F, 4 * R * d, 4 * R * F, 4 * R * F, 4 * R * d, 4 * R * dg,
                    part)
    route = rounded(4 * R, R, 4 * R, 4 * R, 8 * E * ((R + 511) // 512))
    got = B.moe_gated_backward_workspace_size(cfg)
    assert least < got < least + route + (1 << 14)


@pytest.mark.gpu
def test_the_same_without_a_gpu():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = "import json, test_workspace_sizes as t; print(json.dumps(t.sizes()))"
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="",
               PYTHONPATH=os.pathsep.join([root, os.path.join(root, "tests")]))
    out = subprocess.run([sys.executable, "-c", code], env=env, cwd=root, capture_output=True,
                         text=True, check=True).stdout
    assert json.loads(out.splitlines()[-1]) == sizes()

"""Calls from other host threads than the first: what a call does not depend
on the thread that makes it."""
import threading

import pytest
import torch

from gpu_harness import to_device
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import workloads as wl
from test_gpu_few import _w, call, outputs, workspace

pytestmark = pytest.mark.gpu


def on_new_thread(fn):
    """fn on a thread that has made no CUDA call."""
    errors = []

    def run():
        try:
            fn()
        except Exception as e:  # noqa: BLE001 (reported by the caller's thread)
            errors.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_as_a_threads_first_call(dtype):
    w = _w(5, 64, 4, 64, 2, dtype=dtype)
    cfg = B.config_for(w)
    d = to_device(w, wl.generate(w, seed=1))
    want, got, ws = outputs(w, cfg), outputs(w, cfg), workspace(cfg)
    call(cfg, d, want, ws)
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    on_new_thread(lambda: call(cfg, d, got, ws, stream))
    assert B.moe_last_device_status(ws)[0] == 0
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_expert_ffn_as_a_threads_first_call():
    w = _w(64, 64, 4, 128, 1)
    cfg = B.config_for(w)
    d = to_device(w, wl.generate(w, seed=2))
    z = dict(device="cuda")
    offset = torch.arange(0, 65, 16, dtype=torch.int32, **z)
    gate = torch.ones(64, **z)
    ws = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, **z)
    outs = [(torch.zeros((64, 128), dtype=torch.bfloat16, **z), torch.zeros((64, 64), **z))
            for _ in range(2)]

    def run(o, stream=None):
        B.moe_expert_ffn(cfg, d["x"], offset, gate, d["W1"], None, d["W2"], None, *o, ws,
                         stream=stream)
    run(outs[0])
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    on_new_thread(lambda: run(outs[1], stream))
    assert B.moe_last_device_status(ws)[0] == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)



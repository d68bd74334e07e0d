"""GPU parity of the few-token layer (moe_forward_few and
moe_forward_threshold_few) against plain fp64, and what a decoding program
does with it: graphs, streams, workspaces that hold anything, refusals and a
bounded wait that runs out."""
import numpy as np
import pytest
import torch

import few_reference as ref
from gpu_harness import act_bits, act_to_f64, dev_act, dev_f32, to_device
from sparsely_gated_mixture_gb300 import binding as B
from sparsely_gated_mixture_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def _w(T, d, E, d_ff, k, cf=2.0, mode=wl.TOPK, dtype="bf16", noisy=False):
    return wl.Workload("few", T=T, d=d, E=E, d_ff=d_ff, k=k, cf=cf, mode=mode, dtype=dtype,
                       noisy=noisy)


def workspace(cfg, fill=0xFF):
    """Scratch memory that holds anything."""
    return torch.full((B.moe_few_workspace_size(cfg),), fill, dtype=torch.uint8, device="cuda")


def outputs(w, cfg):
    act = torch.bfloat16 if w.dtype == "bf16" else torch.float32
    z = dict(device="cuda")
    return dict(y=torch.full((w.T, w.d), -7, dtype=act, **z),
                idx=torch.full((w.T, w.k), -7, dtype=torch.int32, **z),
                gate=torch.full((w.T, w.k), -7.0, dtype=torch.float32, **z),
                pos=torch.full((w.T, w.k), -7, dtype=torch.int32, **z),
                keep=torch.full((w.T, w.k), 7, dtype=torch.uint8, **z))


def call(cfg, d, o, ws, stream=None):
    B.moe_forward_few(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], d["bias"], d["W1"], d["b1"],
                      d["W2"], d["b2"], o["y"], ws, o["idx"], o["gate"], o["pos"], o["keep"],
                      stream=stream)


def run_few(w, d, ws=None):
    cfg = B.config_for(w)
    ws = workspace(cfg) if ws is None else ws
    o = outputs(w, cfg)
    call(cfg, d, o, ws)
    st, det = B.moe_last_device_status(ws)
    return dict(o, status=st, detail=det)


def check_few(w, inp, res):
    assert res["status"] == 0, (B.STATUS_NAMES[res["status"]], res["detail"])
    H, H_err = ref.logits(inp, w.dtype)
    idx = res["idx"].cpu().numpy()
    # The choices: fp64's own, or swaps that the logits' error explains.
    own = ref.topk(H, w.k)
    for t in np.nonzero((own != idx).any(axis=1))[0]:
        g = idx[t]
        assert len(set(g.tolist())) == w.k and g.min() >= 0 and g.max() < w.E
        tol = 2 * H_err[t].max()
        assert np.all(np.diff(H[t, g]) <= tol), t
        rest = np.setdiff1d(np.arange(w.E), g)
        assert rest.size == 0 or H[t, rest].max() <= H[t, g].min() + tol, t
    gate = ref.gates(H, idx, w.mode)
    rel = 2 * H_err.max() + (w.k + 16) * ref.U + (w.E * ref.U if w.mode == wl.SWITCH else 0)
    got = res["gate"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - gate) <= rel * gate), np.abs(got / gate - 1).max()
    pos, keep = ref.slots(idx, w.E, ref.capacity(w.T, w.E, w.k, w.cf))
    assert np.array_equal(res["pos"].cpu().numpy(), pos)
    assert np.array_equal(res["keep"].cpu().numpy(), keep)
    y, err, _ = ref.output(inp, w.dtype, idx, gate, keep, rel)
    off = np.abs(act_to_f64(res["y"]) - y)
    assert np.all(off <= err), (off.max(), (off / err).max(), np.argwhere(off > err)[:4])
    drop = np.nonzero(~keep.astype(bool).any(axis=1))[0]
    if drop.size:
        xb = inp["x"][drop].view(np.int16 if w.dtype == "bf16" else np.int32)
        assert np.array_equal(act_bits(res["y"][torch.as_tensor(drop).cuda()]), xb)
    return drop.size


CASES = {
    "toy_switch_f32": _w(8, 4, 3, 8, 1, 1.0, wl.SWITCH, "f32"),
    "one_token": _w(1, 64, 16, 128, 4),
    "one_token_f32": _w(1, 64, 16, 128, 4, dtype="f32"),
    "one_expert": _w(17, 64, 1, 128, 1),
    "all_experts_all_tokens": _w(64, 64, 16, 64, 16, cf=4.0),
    "full_batch_noisy": _w(64, 256, 8, 512, 2, cf=4.0, noisy=True),
    "tight_capacity": _w(61, 128, 8, 256, 2, cf=0.6, noisy=True),
    "capacity_one": _w(64, 64, 32, 64, 2, cf=0.05),
    "wide_tiles": _w(5, 1024, 3, 1032, 2),
    "long_k": _w(3, 8, 4, 4104, 2),
    "long_k_back": _w(9, 4104, 4, 8, 2),
    "width_not_64": _w(40, 72, 6, 200, 3),
    "width_even": _w(33, 66, 5, 130, 2),
    "width_odd": _w(33, 65, 5, 33, 2),
    "width_one": _w(3, 1, 2, 1, 1),
    "f32_aligned": _w(64, 128, 6, 516, 3, dtype="f32", noisy=True),
    "f32_odd": _w(19, 35, 7, 51, 3, cf=0.8, dtype="f32", noisy=True),
    "f32_switch_rows": _w(64, 36, 2, 140, 1, cf=2.0, mode=wl.SWITCH, dtype="f32"),
    "many_experts": _w(64, 64, 1024, 64, 8, cf=128.0),
    "many_experts_odd": _w(50, 40, 999, 24, 16, cf=64.0, noisy=True),
    "switch_noisy": _w(31, 128, 12, 96, 1, cf=1.0, mode=wl.SWITCH, noisy=True),
    "k16": _w(64, 128, 40, 64, 16, cf=1.0),
    "largest": _w(64, 72, 1024, 24, 16, cf=1024.0, noisy=True),
    "largest_odd": _w(64, 67, 1024, 23, 16, cf=1024.0, noisy=True),
    "widest": _w(2, 8, 2, 524288, 1),
    "widest_back": _w(2, 524288, 2, 8, 1),
    "widest_f32": _w(2, 5, 2, 524287, 1, dtype="f32"),
    "largest_f32": _w(64, 68, 1024, 24, 16, cf=1024.0, dtype="f32"),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_few_against_fp64(name):
    w = CASES[name]
    inp = wl.generate(w, seed=11, biases=True)
    inp["bias"] = (np.random.default_rng(5).standard_normal(w.E) * 0.3).astype(np.float32)
    check_few(w, inp, run_few(w, to_device(w, inp)))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_batch_sizes(T, dtype):
    """Every expert's rows around the tile heights, without biases or noise."""
    w = _w(T, 192, 3, 320, 2, cf=3.0, dtype=dtype)
    inp = wl.generate(w, seed=T)
    check_few(w, inp, run_few(w, to_device(w, inp)))


def test_few_ties_take_the_lowest_index():
    """A zero router: every logit is equal, so every token takes experts
    0..k-1 with gates exactly 1/k and the capacity keeps the first tokens."""
    w = _w(40, 64, 8, 64, 4, cf=1.0)
    inp = wl.generate(w, seed=2)
    inp["Wg"] = np.zeros_like(inp["Wg"])
    res = run_few(w, to_device(w, inp))
    assert np.array_equal(res["idx"].cpu().numpy(), np.tile([0, 1, 2, 3], (40, 1)))
    assert np.all(res["gate"].cpu().numpy() == 0.25)
    assert check_few(w, inp, res) == 20  # C = 20 of 40 tokens, the others dropped


def test_few_nonfinite_logit_is_reported_and_stays_with_its_token():
    w = _w(6, 64, 8, 128, 2, cf=8.0)
    inp = wl.generate(w, seed=3)
    good = run_few(w, to_device(w, inp))
    assert good["status"] == 0
    for bad in (np.uint16(0x7FC0), np.uint16(0x7F80)):  # NaN, +inf
        x = inp["x"].copy()
        x[4, 7] = bad
        res = run_few(w, to_device(w, dict(inp, x=x)))
        assert res["status"] == 4 and res["detail"] // w.E in (4, 0)
        idx = res["idx"].cpu().numpy()
        assert idx.min() >= 0 and idx.max() < w.E
        rows = [0, 1, 2, 3, 5]
        assert torch.equal(res["y"][rows], good["y"][rows])
        assert not torch.isfinite(res["y"][4].float()).all()


def test_few_optional_outputs_and_same_bits_twice():
    w = _w(23, 128, 16, 256, 4, cf=1.0, noisy=True)
    inp = wl.generate(w, seed=8, biases=True)
    d = to_device(w, inp)
    a = run_few(w, d)
    b = run_few(w, d)
    for n in ("y", "idx", "gate", "pos", "keep"):
        assert torch.equal(a[n], b[n]), n
    cfg = B.config_for(w)
    y = torch.empty_like(a["y"])
    ws = workspace(cfg, 0)
    B.moe_forward_few(cfg, d["x"], d["Wg"], d["Wn"], d["noise"], None, d["W1"], d["b1"], d["W2"],
                      d["b2"], y, ws)
    assert B.moe_last_device_status(ws)[0] == 0
    assert torch.equal(y, a["y"])


@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_in_place(T, dtype):
    """y may be x: the same bits as into another buffer."""
    w = _w(T, 264, 6, 520, 2, cf=2.0, dtype=dtype)
    d = to_device(w, wl.generate(w, seed=31))
    apart = run_few(w, d)
    cfg = B.config_for(w)
    o = outputs(w, cfg)
    o["y"] = d["x"] = d["x"].clone()
    ws = workspace(cfg)
    call(cfg, d, o, ws)
    assert B.moe_last_device_status(ws)[0] == 0
    for name, v in o.items():
        assert torch.equal(apart[name], v), name


def test_few_agrees_with_the_whole_layer():
    """A prompt through moe_forward, then its tokens again a few at a time, as
    decoding follows a prompt: the rows agree to the rounding of both."""
    w = _w(48, 256, 8, 512, 2, cf=8.0)
    inp = wl.generate(w, seed=13, biases=True)
    d = to_device(w, inp)
    cfg = B.config_for(w)
    y = torch.empty((w.T, w.d), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((w.T, w.k), dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    B.moe_forward(cfg, d["x"], d["Wg"], None, None, None, d["W1"], d["b1"], d["W2"], d["b2"], y,
                  None, ws, expert_idx=idx)
    lo = 0
    for n in (1, 2, 13, 32):
        part = w.with_(T=n)
        res = run_few(part, dict(d, x=d["x"][lo:lo + n].contiguous()))
        assert res["status"] == 0
        assert torch.equal(res["idx"], idx[lo:lo + n])
        # Each side is within its own bound of fp64: the few-token form within
        # err, moe_forward, which also rounds each expert term to bf16, within
        # err + 2^-8 * terms (1 + 2^-8 for the rounding of y after it). The
        # terms themselves, not |y - x|, carry that rounding: they may cancel.
        rows = dict(inp, x=inp["x"][lo:lo + n])
        H, H_err = ref.logits(rows, w.dtype)
        i = res["idx"].cpu().numpy()
        _, err, terms = ref.output(rows, w.dtype, i, ref.gates(H, i, w.mode),
                                   np.ones_like(i, np.uint8), 2 * H_err.max() + 32 * ref.U)
        off = np.abs(act_to_f64(res["y"]) - act_to_f64(y[lo:lo + n]))
        assert np.all(off <= 2 * err + 2.0 ** -8 * (1 + 2.0 ** -8) * terms)
        lo += n


def _captured(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fn(torch.cuda.current_stream())
    return g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_graphs_share_a_workspace(dtype):
    """Two captured steps of different shapes on one workspace, replayed in
    turn with an eager call between them: each reproduces its eager bits."""
    ws_n = 0
    steps = []
    for w in (_w(5, 128, 8, 256, 2, cf=4.0, dtype=dtype), _w(33, 64, 12, 72, 3, dtype=dtype)):
        inp = wl.generate(w, seed=w.T)
        cfg = B.config_for(w)
        ws_n = max(ws_n, B.moe_few_workspace_size(cfg))
        steps.append((w, cfg, to_device(w, inp)))
    ws = torch.full((ws_n,), 0xFF, dtype=torch.uint8, device="cuda")
    runs = []
    for w, cfg, d in steps:
        want = run_few(w, d)
        o = outputs(w, cfg)
        g = _captured(lambda s, cfg=cfg, d=d, o=o: call(cfg, d, o, ws, s))
        runs.append((g, o, want))
    for _ in range(3):
        for g, o, _ in runs:
            o["y"].fill_(-7)
            g.replay()
        call(steps[0][1], steps[0][2], outputs(steps[0][0], steps[0][1]), ws)
    torch.cuda.synchronize()
    for (g, o, want) in runs:
        for n in ("y", "idx", "gate", "pos", "keep"):
            assert torch.equal(o[n], want[n]), n
    assert B.moe_last_device_status(ws)[0] == 0


def test_few_on_two_streams():
    """Calls in flight on two streams, each with its own workspace."""
    w = _w(16, 256, 8, 512, 2, cf=4.0)
    d = to_device(w, wl.generate(w, seed=4))
    cfg = B.config_for(w)
    want = run_few(w, d)
    torch.cuda.synchronize()
    lanes = [(torch.cuda.Stream(), workspace(cfg), outputs(w, cfg)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, o in lanes:
            call(cfg, d, o, ws, s)
    torch.cuda.synchronize()
    for s, ws, o in lanes:
        assert B.moe_last_device_status(ws, s)[0] == 0
        assert torch.equal(o["y"], want["y"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_wait_limit_reported_and_next_call_runs(monkeypatch, dtype):
    w = _w(8, 512, 8, 1024, 2, cf=4.0, dtype=dtype)
    d = to_device(w, wl.generate(w, seed=6))
    want = run_few(w, d)
    cfg = B.config_for(w)
    ws = workspace(cfg)
    monkeypatch.setenv("MOE_WAIT_LIMIT_NS", "0")
    assert run_few(w, d, ws)["status"] == 5
    monkeypatch.delenv("MOE_WAIT_LIMIT_NS")
    res = run_few(w, d, ws)
    assert res["status"] == 0 and torch.equal(res["y"], want["y"])


# ----------------------------------------------------------------------------- threshold mask
def run_threshold(w, inp, thr, kmax):
    cfg = B.config(w.T, w.d, w.E, w.d_ff, kmax, 1.0,
                   act_dtype=B.MOE_BF16 if w.dtype == "bf16" else B.MOE_F32)
    d = to_device(w, inp)
    o = outputs(w.with_(k=kmax), cfg)
    words = torch.full((w.T, (w.E + 31) // 32), -1, dtype=torch.int32, device="cuda")
    ws = workspace(cfg)
    B.moe_forward_threshold_few(cfg, d["x"], d["Wg"], d["bias"], dev_f32(thr), d["W1"], d["b1"],
                                d["W2"], d["b2"], o["y"], ws, o["idx"], o["gate"], words)
    st, det = B.moe_last_device_status(ws)
    bits = (words.cpu().numpy().view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1
    return dict(o, status=st, detail=det, mask=bits.reshape(w.T, -1).astype(bool))


def check_threshold(w, inp, thr, kmax):
    res = run_threshold(w, inp, thr, kmax)
    assert res["status"] == 0, (B.STATUS_NAMES[res["status"]], res["detail"])
    H, H_err = ref.logits(inp, w.dtype)
    P = ref.softmax(H)
    rel = 2 * H_err.max() + (w.E + 16) * ref.U
    th = thr.astype(np.float64)
    mask = res["mask"]
    assert not mask[:, w.E:].any()
    mask = mask[:, :w.E]
    differ = mask != (P > th)
    assert np.all(np.abs(P - th)[differ] <= (rel * P)[differ] + ref.U * np.broadcast_to(th, P.shape)[differ])
    n = mask.sum(axis=1)
    idx = np.full((w.T, kmax), w.E, np.int32)
    gate = np.zeros((w.T, kmax))
    for t in range(w.T):
        e = np.nonzero(mask[t])[0]
        idx[t, :e.size] = e
        gate[t, :e.size] = P[t, e] / P[t, e].sum() if e.size else 0
    assert np.array_equal(res["idx"].cpu().numpy(), idx)
    got = res["gate"].cpu().numpy()
    assert np.all(np.abs(got - gate) <= 2 * rel * gate)
    y, err, _ = ref.output(inp, w.dtype, idx, gate, (idx < w.E).astype(np.uint8), 2 * rel)
    off = np.abs(act_to_f64(res["y"]) - y)
    assert np.all(off <= err), (off.max(), (off / err).max())
    none = np.nonzero(n == 0)[0]
    if none.size:
        xb = inp["x"][none].view(np.int16 if w.dtype == "bf16" else np.int32)
        assert np.array_equal(act_bits(res["y"][torch.as_tensor(none).cuda()]), xb)
    return n, none.size


THR = {
    "one_token": (_w(1, 64, 8, 64, 1), (0.5, 1.5), 8),
    "e16": (_w(64, 64, 16, 128, 1), (3.3, 4.5), 4),
    "e64": (_w(48, 128, 64, 64, 1), (4.1, 6.4), 16),
    "f32_odd": (_w(29, 36, 7, 50, 1, dtype="f32"), (0.6, 1.4), 7),
    "odd": (_w(20, 73, 5, 31, 1), (0.7, 1.3), 5),
    "e1000": (_w(37, 64, 1000, 40, 1), (64.0, 90.0), 16),
    "all_pass": (_w(64, 64, 16, 64, 1), (0.0, 1e-6), 16),
}


@pytest.mark.parametrize("name", sorted(THR))
def test_threshold_few_against_fp64(name):
    w, (lo, hi), kmax = THR[name]
    inp = wl.generate(w, seed=21, biases=True)
    inp["bias"] = (np.random.default_rng(3).standard_normal(w.E) * 0.3).astype(np.float32)
    if name == "e1000":
        inp["Wg"] = inp["Wg"] * np.float32(3.0)
    thr = (np.random.default_rng(4).uniform(lo, hi, w.E) / w.E).astype(np.float32)
    n, _ = check_threshold(w, inp, thr, kmax)
    assert n.max() > 0


def test_threshold_few_ties_and_tokens_without_a_pick():
    """Every P exactly 1/8; thresholds equal to it are not passed."""
    w = _w(30, 64, 8, 64, 1)
    inp = wl.generate(w, seed=9, biases=True)
    inp["Wg"] = np.zeros_like(inp["Wg"])
    thr = np.where(np.arange(8) % 2 == 0, 0.125, np.nextafter(np.float32(0.125), 0)).astype(
        np.float32)
    n, _ = check_threshold(w, inp, thr, 8)
    assert np.all(n == 4)
    _, none = check_threshold(w, inp, np.full(8, 0.125, np.float32), 8)
    assert none == w.T


def test_threshold_few_over_the_bound_is_reported():
    w = _w(10, 64, 8, 64, 1)
    inp = wl.generate(w, seed=9)
    res = run_threshold(w, inp, np.full(8, 1e-6, np.float32), 2)
    assert res["status"] == 6 and 0 <= res["detail"] < w.T
    assert np.array_equal(res["idx"].cpu().numpy(), np.tile([0, 1], (w.T, 1)))
    assert res["mask"][:, :8].all()

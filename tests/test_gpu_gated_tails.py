"""The gated experts' backward for row counts that are not a multiple of eight:
the zero rows behind the last packed one end there (warps that the grid's last
block has to spare must not go on, into the rows of dy)."""
import pytest
import torch

import gated_reference as R
import test_gpu_gated as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", list(range(65, 73)) + [1, 7, 130, 1001])
@pytest.mark.parametrize("d,F", [(64, 4096), (192, 2048), (64, 64)])
def test_any_number_of_rows(T, d, F):
    """One expert's rows and two; wide hidden rows, whose zeros take longest."""
    for E in (1, 2):
        s = G.inputs(T, d, E, F, 1, torch.bfloat16, seed=T)
        cfg, g = G.config(s, float(E)), G.dev(s)
        o = G.run_forward(cfg, R.SILU, g)
        b = G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
        G.check_backward(cfg, R.SILU, s, o["p1"], o["p3"], b)
        # The rows are those of dy: with dy = 0 nothing has a gradient.
        z = G.run_backward(cfg, R.SILU, dict(g, dy=torch.zeros_like(g["dy"])), o["p1"], o["p3"])
        for n in ("dx", "dgate", "dW1", "dW3", "dW2", "db1", "db3", "db2"):
            assert not bool(z[n].any()), n


def test_wide_hidden_rows():
    """Against a product in 32 bits on the GPU: 70 rows of 16384 hidden values."""
    T, d, F, E = 70, 64, 16384, 2
    s = G.inputs(T, d, E, F, 1, torch.bfloat16, seed=T, biases=False)
    cfg, g = G.config(s, 2.0), G.dev(s)
    o = G.run_forward(cfg, R.SILU, g)
    b = G.run_backward(cfg, R.SILU, g, o["p1"], o["p3"])
    order = torch.argsort(g["idx"][:, 0].long(), stable=True)
    x, dy, gate = (g[n][order].double() for n in ("x", "dy", "gate"))
    expert = g["idx"][order, 0].long()
    for e in range(E):
        at = expert == e
        p1, p3 = (o[n][at].double() for n in ("p1", "p3"))
        D = dy[at] @ g["W2"][e].double().t()
        t = torch.sigmoid(p1)
        want = dict(dW1=x[at].t() @ (gate[at] * D * p3 * t * (1 + p1 * (1 - t))),
                    dW3=x[at].t() @ (gate[at] * D * p1 * t),
                    dW2=(gate[at] * p1 * t * p3).t() @ dy[at])
        for n, w in want.items():
            # A rounded operand and a rounded result: 2^-8 of a sum's terms and of itself.
            # Their root mean square is under both, and a row of 35 left out changes
            # it by a sixth.
            rel = float((b[n][e].double() - w).norm() / w.norm())
            assert rel < 2 * 2.0 ** -8, (n, e, rel)

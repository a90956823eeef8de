"""Infinities among the operands of the experts' products with few rows, where h and the gradients of gate
and up are kept in two parts: a result is infinite, NaN or finite as the formula has it, whatever the second part
holds (0, or a value of the other sign)."""

import numpy as np
import pytest
import torch

from oracle import layer as L
from tests import test_gpu_ffn as F
from tests.test_gpu_norm_inf import same_class

pytestmark = pytest.mark.gpu

INF = float("inf")
# streamed (below 8 rows per expert, without a checkpoint), and in tiles of rows and their rests
SHAPES = [([[3, 2]], 72, 40), ([[2, 1], [5, 0]], 136, 264), ([[33, 0, 5]], 136, 264), ([[1]], 264, 72), ([[32, 30]], 264, 320)]


def _dot(a, b):
    """a @ b from its products, in 64 bits (a library product may pad with zeros, and 0 * inf is NaN)."""
    with np.errstate(invalid="ignore"):
        return np.stack([(r[:, None] * b).sum(0) for r in a])


def _blocks(st):
    return [(d, e, at, n) for d, e, at, n in L.blocks(st["splits"], st["rows"]) if n]


def _w(st, k, d, e):
    return F._f64(st[k][d][e])


@pytest.mark.parametrize("counts,H,I", SHAPES)
@pytest.mark.parametrize("saved_t", [None, "bf16"])
def test_infinite_weights_of_the_down_product(counts, H, I, saved_t):
    rng = np.random.default_rng(H)
    st = F.make(rng, counts, H, I, spare=0)
    _, clean, _ = F.run_forward(st, "bf16", saved_t)
    for d in range(st["N"]):
        st["w_down"][d][:, 5, 3] = INF
        st["w_down"][d][:, H - 1, I - 1] = -INF
        st["w_down"][d][:, 8, 1] = INF
        st["w_down"][d][:, 8, 2] = INF                    # of both signs in some rows: NaN
    xv, y, _ = F.run_forward(st, "bf16", saved_t)
    for d, e, at, n in _blocks(st):
        _, _, h, _ = L.ffn(xv[d][at:at + n], *(_w(st, k, d, e) for k in ("w_gate", "w_up", "w_down")))
        got, want = F._f64(y[d][at:at + n]), _dot(h, _w(st, "w_down", d, e).T)
        assert same_class(got, want), f"rank {d} expert {e}"
        fin = np.isfinite(want)
        assert np.array_equal(got[fin], F._f64(clean[d][at:at + n])[fin])


@pytest.mark.parametrize("counts,H,I", SHAPES)
@pytest.mark.parametrize("what", ["w_gate", "w_up", "x", "dy", "up"])
@pytest.mark.parametrize("dw_t", ["bf16", "fp32"])
def test_infinite_operands_of_the_gradients(counts, H, I, what, dw_t):
    rng = np.random.default_rng(H + I)
    st = F.make(rng, counts, H, I, spare=0)
    gate_up = [F._bf16(rng, (r, 2 * I), 1.5) for r in st["rows"]]
    dy = [F._bf16(rng, (r, H)) for r in st["rows"]]
    for d in range(st["N"]):
        r = st["rows"][d] - 1
        if what == "w_gate":
            st["w_gate"][d][:, I - 1, 3] = INF
        elif what == "w_up":
            st["w_up"][d][:, 2, H - 1] = -INF
        elif what == "x":
            st["x"][d][r, 4] = INF
        elif what == "dy":
            dy[d][r, H - 2] = -INF
        else:
            gate_up[d][0, I + 6] = INF
    xv, sv, dx, dw = F.run_backward(st, "bf16", "bf16", dw_t, gate_up, dy)
    for d, e, at, n in _blocks(st):
        x, g, u, y = xv[d][at:at + n], sv[d][at:at + n, :I], sv[d][at:at + n, I:], F._f64(dy[d][at:at + n])
        wg, wu, wd = (_w(st, k, d, e) for k in ("w_gate", "w_up", "w_down"))
        with np.errstate(invalid="ignore"):
            dh = _dot(y, wd)
            dg, du, h = dh * u * L.dsilu(g), dh * L.silu(g), L.silu(g) * u
            want = {"dx": _dot(dg, wg) + _dot(du, wu), "w_gate": _dot(dg.T, x), "w_up": _dot(du.T, x), "w_down": _dot(y.T, h)}
        got = {"dx": F._f64(dx[d][at:at + n]), **{k: F._f64(dw[k][d][e]) for k in dw}}
        for k, v in want.items():
            assert same_class(got[k], v), f"rank {d} expert {e}: {k}"

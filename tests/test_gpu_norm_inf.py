"""Infinities and NaN in any column of a normed row, at lengths whose units fill the lanes and at lengths
that leave lanes past the row's end: what a row becomes goes by the formula, not by the column."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import layer as L
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LENGTHS = [1, 8, 513, 520, 1000, 1024, 2056, 4096, 5120, 7168, 8201, 16392]   # wide and element-wise loads, one and two passes


def _f64(t):
    return t.detach().cpu().double().numpy()


def _normal(rng, shape, dtype):
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(TYPES[dtype]).to(DEV)


def same_class(got, want):
    """NaN where want is, infinities of its sign where it has them, finite elsewhere."""
    inf = np.isinf(want)
    return (np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), inf)
            and np.array_equal(np.sign(got[inf]), np.sign(want[inf])))


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode", ["plain", "residual", "in_place", "mx8"])
def test_an_infinity_in_any_column(H, dtype, mode):
    """rstd = 1 / sqrt(inf) = 0: the infinity itself becomes NaN (inf * 0), every other value 0."""
    at = sorted({0, H // 2, max(0, H - 9), H - 1})
    rng = np.random.default_rng(H)
    x = _normal(rng, (2 * len(at) + 1, H), dtype)
    res = None
    for i, c in enumerate(at):
        x[2 * i, c] = float("inf") if i % 2 else float("-inf")
        x[2 * i + 1, c] = float("nan")
    if mode in ("residual", "in_place"):
        res = torch.zeros_like(x)
        for i, c in enumerate(at):                       # the sum overflows its type
            x[2 * i, c] = 3.2e38
            res[2 * i, c] = 3.2e38
    w = torch.ones(H, dtype=TYPES[dtype], device=DEV)
    T = len(x)
    rstd = torch.empty(T, device=DEV)
    y = torch.empty(T, gc.gc_mx8_row_bytes(H), dtype=torch.uint8, device=DEV) if mode == "mx8" else torch.empty_like(x)
    gc.gc_rms_norm([x], [w], [T], H, [y], residual=None if res is None else [res], rstd=[rstd],
                   sum_out=[x] if mode == "in_place" else None)
    torch.cuda.synchronize()
    got = L.unpack8(y.cpu().numpy(), H) if mode == "mx8" else _f64(y)
    for i, c in enumerate(at):
        row = got[2 * i]
        assert np.isnan(row[c]) and not np.delete(row, c).any(), f"column {c}: {row}"
        assert rstd[2 * i] == 0
        assert np.isnan(got[2 * i + 1]).all() and torch.isnan(rstd[2 * i + 1])
    assert np.isfinite(got[-1]).all()


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("where", ["weight", "dy"])
def test_an_infinity_in_any_column_of_the_backward(H, dtype, where):
    rng = np.random.default_rng(H + 1)
    for c in sorted({0, H // 2, max(0, H - 9), H - 1}):
        s, dy, w = (_normal(rng, sh, dtype) for sh in ((5, H), (5, H), (H,)))
        if where == "weight":
            w[c] = float("inf")
        else:
            dy[3, c] = float("-inf")
        rstd = torch.rsqrt(s.float().square().mean(1))
        dx, dw = torch.empty_like(s), torch.empty(H, device=DEV)
        scratch = torch.empty(gc.gc_rms_norm_backward_scratch_bytes([5], H), dtype=torch.uint8, device=DEV)
        gc.gc_rms_norm_backward([dy], [s], [w], [rstd], [5], H, [dx], [dw], scratch)
        torch.cuda.synchronize()
        with np.errstate(invalid="ignore"):
            want, wdw = L.rms_norm_backward(_f64(dy), _f64(s), _f64(w)[None], _f64(rstd))
        assert same_class(_f64(dx), want), f"column {c}"
        assert same_class(_f64(dw), wdw), f"column {c}"

"""GPU parity of dropout: the mask element for element with the oracle's generator, the
values against bounds counted from the roundings, streams of ranks, steps and offsets,
replayed graphs."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import token as K
from tests.gpu_util import DEV
from tests.test_gpu_embed import HALF, TYPES, U, _f64, _rows, guarded, untouched

pytestmark = pytest.mark.gpu

CASES = [
    # ranks' elements, type, element offset
    ([1], "bf16", 0), ([7], "fp32", 0), ([8, 0, 9], "bf16", 0), ([4096], "bf16", 0), ([4097, 5], "fp32", 0),
    ([100003], "bf16", 0), ([100003, 2048], "bf16", 1), ([70001], "fp32", 1), ([1 + 37 * s for s in range(64)], "bf16", 0),
]


@pytest.mark.parametrize("counts,dtype,offset", CASES)
@pytest.mark.parametrize("mode", ["plain", "residual", "over_x", "over_residual"])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout(counts, dtype, offset, mode, p):
    rng = np.random.default_rng(len(counts) + counts[0])
    x = [_rows(rng, (n,), dtype, 1.0, offset) for n in counts]
    x0 = [_f64(t) for t in x]
    res = None if mode in ("plain", "over_x") else [_rows(rng, (n,), dtype, 2.0, offset) for n in counts]
    r0 = None if res is None else [_f64(t) for t in res]
    outs = [guarded((n,), TYPES[dtype], offset) for n in counts]
    y = {"over_x": x, "over_residual": res}.get(mode, [o[1] for o in outs])
    seed, off, step = 0xFEDCBA9876543210, 3, 1 << 40
    gc.gc_dropout(x, counts, p, seed, y, offset=off, step=torch.tensor([step], device=DEV), residual=res)
    for r, n in enumerate(counts):
        keep = K.keep(n, r, p, seed, off + step)
        want = K.dropout(x0[r], r, p, seed, off + step, None if r0 is None else r0[r])
        part = np.where(keep, np.abs(x0[r]) * 2, 0.0)          # 1 / (1 - p) is at most 2
        # the factor's rounding and the product: 2 u of the part; the sum: u; one rounding to the type
        tol = 3 * U * part + (HALF[dtype] + 2 * U) * np.abs(want) * (1 + 2 ** -8)
        got = _f64(y[r])
        assert (np.abs(got - want) <= tol).all(), r
        if mode == "plain" and n:
            assert ((got != 0) == (keep & (x0[r] != 0))).all()
        assert untouched(outs[r][0], offset, n)


def test_dropout_of_nothing_and_everything():
    x = [torch.tensor([1.5, float("nan"), float("inf"), -2.0], device=DEV)]
    y = [torch.empty(4, device=DEV)]
    gc.gc_dropout(x, [4], 0.0, 5, y)
    assert y[0][0] == 1.5 and y[0][1].isnan() and y[0][2] == float("inf") and y[0][3] == -2.0
    gc.gc_dropout(x, [4], 1.0, 5, y)
    assert (y[0] == 0).all()                                   # a dropped value counts as 0, whatever it is
    gc.gc_dropout(x, [4], 1.0, 5, y, residual=[torch.ones(4, device=DEV)])
    assert (y[0] == 1).all()


def test_gradient_takes_the_same_mask():
    n = [5000, 3001]
    rng = np.random.default_rng(2)
    x, dy = [_rows(rng, (k,), "fp32") for k in n], [_rows(rng, (k,), "fp32") for k in n]
    y, dx = [torch.empty(k, device=DEV) for k in n], [torch.empty(k, device=DEV) for k in n]
    gc.gc_dropout(x, n, 0.3, 77, y, offset=9)
    gc.gc_dropout(dy, n, 0.3, 77, dx, offset=9)
    for r in range(2):
        assert torch.equal(y[r] != 0, dx[r] != 0)
        # linear in x: <dy, y(x)> = <dx, x>
        left, right = (_f64(dy[r]) * _f64(y[r])).sum(), (_f64(dx[r]) * _f64(x[r])).sum()
        assert abs(left - right) <= 8 * U * (np.abs(_f64(dy[r])) * np.abs(_f64(y[r]))).sum()


def test_step_counts_in_a_replayed_graph():
    n = [4099, 64]
    x, y = [torch.ones(k, device=DEV) for k in n], [torch.empty(k, device=DEV) for k in n]
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gc.gc_dropout(x, n, 0.5, 11, y, step=step)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gc.gc_dropout(x, n, 0.5, 11, y, step=step)
        step.add_(1)
    step.zero_()
    for k in range(4):
        g.replay()
        torch.cuda.synchronize()
        for r in range(2):
            assert np.array_equal(_f64(y[r]) != 0, K.keep(n[r], r, 0.5, 11, k)), (k, r)
        x[0].add_(0)                                           # eager work between the replays

"""GPU parity of the combine's gradient with its definition in 64 bits: rows are
exact (one product, one rounding), dots within their additions' roundings."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle.numerics import f32_to_bf16
from tests.gpu_util import DEV, assert_same, from_dev, to_dev
from tests.test_gpu_moe import _expert_rows, _i32, _routing, check_plan, route_on_device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _wide(t):
    return t.detach().cpu().double().numpy()


CASES = [
    # dtype, hidden, N, E, tokens, K, drop
    ("bf16", 4096, 4, 3, [29, 3, 0, 70], 2, 0.0), ("bf16", 8, 1, 2, [1], 1, 0.0), ("bf16", 1000, 2, 4, [5, 40], 2, 0.2),
    ("bf16", 7, 3, 2, [9, 1, 4], 3, 0.1), ("bf16", 4099, 2, 4, [6, 2], 8, 0.1), ("bf16", 264, 64, 1, [s % 4 for s in range(64)], 2, 0.0),
    ("fp32", 999, 4, 3, [29, 3, 0, 70], 2, 0.05), ("fp32", 1024, 2, 4, [17, 5], 5, 0.1), ("fp32", 1, 2, 2, [3, 300], 1, 0.0),
    ("fp32", 4, 2, 2, [70, 1], 4, 0.5), ("bf16", 9000, 1, 4, [3], 2, 0.0),
]


@pytest.mark.parametrize("dtype,H,N,E,T,K,drop", CASES)
def test_combine_backward(dtype, H, N, E, T, K, drop):
    rng = np.random.default_rng(H + N)
    experts = _routing(rng, N, E, T, K, drop)
    ntok, splits, dest = route_on_device(experts, N, E, K)
    rows = [int(r) for r in check_plan(experts, N, E, K, splits, dest).sum(axis=(0, 2))]
    spare = 2                                              # rows no route names keep what they held
    y = [_expert_rows(rng, (r + spare) * H, 1, dtype, False) for r in rows]
    g = [_expert_rows(rng, t * H, 1, dtype, False) for t in T]
    w = [rng.normal(size=(t, K)).astype(np.float32) for t in T]
    y_dev, g_dev = [to_dev(a, dtype) for a in y], [to_dev(a, dtype) for a in g]
    w_dev = [torch.from_numpy(a.reshape(-1)).to(DEV) for a in w]
    dy = [torch.full(((r + spare) * H + 16,), 7.0, dtype=a.dtype, device=DEV) for r, a in zip(rows, y_dev)]
    dw = [torch.full((t * K + 8,), 7.0, device=DEV) for t in T]
    gc.gc_moe_combine_backward(g_dev, y_dev, [r + spare for r in rows], dest, w_dev, ntok, K, H, dtype, dy, dw)
    torch.cuda.synchronize()
    want = [np.full((r + spare, H), 7.0, dtype=np.float32) for r in rows]
    for s in range(N):
        d = dest[s].cpu().numpy()[:2 * T[s] * K].reshape(T[s], K, 2)
        gs, got = _wide(g_dev[s]).reshape(T[s], H), _wide(dw[s])
        assert np.all(got[T[s] * K:] == 7.0)
        for t in range(T[s]):
            for k in range(K):
                r, row = d[t, k]
                if r < 0:
                    assert got[t * K + k] == 0.0
                    continue
                yr = _wide(y_dev[r][row * H:(row + 1) * H])
                terms = np.abs(gs[t] * yr).sum()
                # each lane adds its elements in turn (at least 1 lane per 32 elements, at most 64 lanes), then the lanes
                assert abs(got[t * K + k] - (gs[t] * yr).sum()) <= (max(32, H / 64 + 8) + 8) * U * terms
                want[r][row] = (w[s][t, k] * gs[t].astype(np.float32)).astype(np.float32)
    for r in range(N):
        ref = f32_to_bf16(want[r].reshape(-1)) if dtype == "bf16" else want[r].reshape(-1)
        assert_same(from_dev(dy[r])[:len(ref)], ref, dtype, f"rank {r}")
        assert bool((dy[r][len(ref):] == 7.0).all())


def test_malformed_entries_get_zero_and_write_nothing():
    N, K, H = 2, 2, 64
    dest = [_i32([[0, 0], [5, 0], [1, 1], [1, 99], [-1, 0], [0, -3]]), _i32([[1, 0], [0, 1]])]
    y = [torch.ones(2 * H, device=DEV), torch.full((2 * H,), 2.0, device=DEV)]
    g = [torch.ones(3 * H, device=DEV), torch.full((H,), 3.0, device=DEV)]
    w = [torch.full((6,), 0.5, device=DEV), torch.ones(2, device=DEV)]
    dy = [torch.full((2 * H,), 9.0, device=DEV) for _ in range(2)]
    dw = [torch.full((6,), 9.0, device=DEV), torch.full((2,), 9.0, device=DEV)]
    gc.gc_moe_combine_backward(g, y, [2, 2], dest, w, [3, 1], K, H, "fp32", dy, dw)
    torch.cuda.synchronize()
    assert dw[0].tolist() == [H, 0.0, 2.0 * H, 0.0, 0.0, 0.0] and dw[1].tolist() == [6.0 * H, 3.0 * H]
    assert dy[0].view(2, H)[:, 0].tolist() == [0.5, 3.0] and dy[1].view(2, H)[:, 0].tolist() == [3.0, 0.5]


def test_gradient_is_the_combines_own():
    """<combine(y), g> changes with y and w as the gradients say (both are linear: exact differences)."""
    rng = np.random.default_rng(5)
    N, E, K, H, T = 2, 3, 2, 96, [11, 6]
    experts = _routing(rng, N, E, T, K)
    ntok, splits, dest = route_on_device(experts, N, E, K)
    rows = [int(r) for r in check_plan(experts, N, E, K, splits, dest).sum(axis=(0, 2))]
    f = lambda n: torch.from_numpy(rng.normal(size=n).astype(np.float32)).to(DEV)  # noqa: E731
    y, w, g = [f(r * H) for r in rows], [f(t * K) for t in T], [f(t * H) for t in T]
    dy, dw = [torch.empty_like(a) for a in y], [torch.empty_like(a) for a in w]
    gc.gc_moe_combine_backward(g, y, rows, dest, w, ntok, K, H, "fp32", dy, dw)

    def loss(y_, w_):
        out = [torch.empty_like(a) for a in g]
        gc.gc_moe_combine(y_, rows, dest, w_, ntok, K, H, "fp32", out)
        return sum(float((a.double() * b.double()).sum()) for a, b in zip(out, g))
    for _ in range(3):
        vy, vw = [f(r * H) for r in rows], [f(t * K) for t in T]
        ly = loss([a + b for a, b in zip(y, vy)], w) - loss(y, w)
        lw = loss(y, [a + b for a, b in zip(w, vw)]) - loss(y, w)
        wy = sum(float((a.double() * b.double()).sum()) for a, b in zip(dy, vy))
        ww = sum(float((a.double() * b.double()).sum()) for a, b in zip(dw, vw))
        # 17 * 2 * 96 products, each of a few fp32 roundings of terms up to about 4^3
        scale = sum(T) * K * H * 64 * 8 * U
        assert abs(ly - wy) <= scale and abs(lw - ww) <= scale

"""GPU parity of the experts' gated feed-forward block and its backward pass with
the 64-bit oracle, element by element.

Bounds count roundings: u = 2^-24 per fp32 operation, a sum of K products within
2 K u of the sum of magnitudes whatever its order, half a step (2^-8 of the value)
for each rounding to bf16, 2^-4 (or 2^(e-10)) to an 8-bit code.  An error of h or
of dgate / dup goes through the next product with the weights' magnitudes."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import layer as L
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
FILL = 5.0


def _f64(t):
    return t.detach().cpu().double().numpy()


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).bfloat16()


def make(rng, counts, H, F, spare=1):
    """counts[d][e] rows per block.  Buffers hold `spare` rows behind the last block."""
    N, E = len(counts), len(counts[0])
    splits = np.zeros((N, N, E), dtype=np.int64)
    for d in range(N):
        for e in range(E):
            left = counts[d][e]
            for s in range(N):
                n = left if s == N - 1 else int(rng.integers(0, left + 1))
                splits[s, d, e] = n
                left -= n
    rows = [sum(c) + spare for c in counts]
    st = {"N": N, "E": E, "H": H, "F": F, "rows": rows, "splits": splits,
          "splits_dev": torch.from_numpy(splits.reshape(-1)).to(DEV),
          "x": [_bf16(rng, (r, H)) for r in rows]}
    for k, sh, sc in (("w_gate", (F, H), H), ("w_up", (F, H), H), ("w_down", (H, F), F)):
        st[k] = [_bf16(rng, (E, *sh), sc ** -0.5) for _ in range(N)]
    return st


def dev(ts):
    return [t.to(DEV) for t in ts]


def pack_dev(ts, n):
    """8-bit rows of host rows, by the oracle."""
    return [torch.from_numpy(L.pack8(t.double().numpy()) if len(t) else np.zeros((0, L.row_bytes(n)), np.uint8)).to(DEV)
            for t in ts]


def values(ts, n):
    return [torch.from_numpy(L.unpack8(t.cpu().numpy(), n)) for t in ts]


def scratch_for(st, x_t, backward):
    need = gc.gc_moe_ffn_scratch_bytes(st["rows"], st["E"], st["H"], st["F"], x_dtype=x_t, backward=backward)
    assert need > 0
    full = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    return full, full[:need]


def run_forward(st, x_t, saved_t):
    H, F, rows = st["H"], st["F"], st["rows"]
    x = pack_dev(st["x"], H) if x_t == "mx8" else dev(st["x"])
    xv = [v.numpy() for v in values(x, H)] if x_t == "mx8" else [_f64(t) for t in x]
    y = [torch.full((r, H), FILL, dtype=torch.bfloat16, device=DEV) for r in rows]
    saved = None
    if saved_t == "bf16":
        saved = [torch.full((r, 2 * F), FILL, dtype=torch.bfloat16, device=DEV) for r in rows]
    elif saved_t == "mx8":
        saved = [torch.full((r, gc.gc_mx8_row_bytes(2 * F)), 0x5A, dtype=torch.uint8, device=DEV) for r in rows]
    full, scratch = scratch_for(st, x_t, False)
    gc.gc_moe_ffn(x, rows, st["splits_dev"], st["E"], H, F, dev(st["w_gate"]), dev(st["w_up"]), dev(st["w_down"]), y,
                  scratch, saved=saved)
    torch.cuda.synchronize()
    assert bool((full[len(scratch):] == 0x5A).all())
    return xv, y, saved


def sig_error(g):
    """Relative error of the fp32 sigmoid: argument rounding, exponential, addition, reciprocal."""
    return (np.abs(g) + 8) * 2 * U


def check_forward(st, xv, y, saved, saved_t):
    H, F = st["H"], st["F"]
    for d, e, at, n in L.blocks(st["splits"], st["rows"]):
        if not n:
            continue
        x = xv[d][at:at + n]
        wg, wu, wd = (_f64(st[k][d][e]) for k in ("w_gate", "w_up", "w_down"))
        g, u, h, want = L.ffn(x, wg, wu, wd)
        eg, eu = 2 * H * U * (np.abs(x) @ np.abs(wg).T), 2 * H * U * (np.abs(x) @ np.abs(wu).T)
        # |silu'| <= 1.1; products and the sigmoid; one rounding to bf16
        eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(L.silu(g)) * eu + np.abs(h) * (sig_error(g) + 4 * U)
        eh = eh + HALF * (np.abs(h) + eh) + 1e-38
        ey = eh @ np.abs(wd).T + 2 * F * U * ((np.abs(h) + eh) @ np.abs(wd).T)
        ey = ey + HALF * (np.abs(want) + ey)
        got = _f64(y[d][at:at + n])
        assert np.all(np.abs(got - want) <= ey), f"rank {d} expert {e}: {np.max(np.abs(got - want) / ey)}"
        if saved_t == "bf16":
            sv, es = _f64(saved[d][at:at + n]), np.concatenate([eg, eu], 1)
            ref = np.concatenate([g, u], 1)
            assert np.all(np.abs(sv - ref) <= es + HALF * (np.abs(ref) + es)), f"rank {d} expert {e}: saved"
        elif saved_t == "mx8":
            p, es = saved[d][at:at + n].cpu().numpy(), np.concatenate([eg, eu], 1)
            ref = np.concatenate([g, u], 1)
            ex = np.repeat(p[:, 2 * F:2 * F + F // 16].astype(int) - 127, 32, axis=1)
            step = np.maximum(2.0 ** -4 * (np.abs(ref) + es), 2.0 ** (ex - 10.0))
            assert np.all(np.abs(L.unpack8(p, 2 * F) - ref) <= es + step), f"rank {d} expert {e}: saved"
            amax = np.abs(ref).reshape(n, -1, 32).max(2)
            worst = es.reshape(n, -1, 32).max(2)
            ee = p[:, 2 * F:2 * F + F // 16].astype(int) - 127
            assert np.all(amax - worst <= 448 * 2.0 ** ee) and np.all(amax + worst >= 448 * 2.0 ** (ee - 1.0))
            assert not p[:, 2 * F + F // 16:].any()
    for d in range(st["N"]):                     # rows no expert takes
        end = max((a + n for dd, _, a, n in L.blocks(st["splits"], st["rows"]) if dd == d), default=0)
        assert bool((y[d][end:] == FILL).all())
        if saved is not None:
            assert bool((saved[d][end:] == (0x5A if saved_t == "mx8" else FILL)).all())


SHAPES = [
    # rows per block, hidden, inter
    ([[1]], 8, 8), ([[1, 0]], 64, 32), ([[3, 0, 5], [0, 0, 0]], 72, 40), ([[64, 1]], 128, 96), ([[65, 63]], 200, 160),
    ([[130, 127], [5, 128]], 136, 264), ([[300]], 264, 288), ([[255, 257, 1], [0, 512, 3]], 320, 128),
    ([[17] * 8], 512, 256), ([[2] * 2 for _ in range(9)], 64, 64), ([[s % 5] for s in range(64)], 40, 32),
]


@pytest.mark.parametrize("counts,H,F", SHAPES)
@pytest.mark.parametrize("x_t,saved_t", [("bf16", None), ("bf16", "bf16"), ("bf16", "mx8"), ("mx8", "mx8")])
def test_forward(counts, H, F, x_t, saved_t):
    if saved_t == "mx8" and F % 32:
        F = (F + 31) // 32 * 32
    rng = np.random.default_rng(H * 7 + F + len(counts))
    st = make(rng, counts, H, F)
    xv, y, saved = run_forward(st, x_t, saved_t)
    check_forward(st, xv, y, saved, saved_t)


def run_backward(st, x_t, saved_t, dw_t, gate_up, dy):
    H, F, rows, N, E = (st[k] for k in ("H", "F", "rows", "N", "E"))
    x = pack_dev(st["x"], H) if x_t == "mx8" else dev(st["x"])
    xv = [v.numpy() for v in values(x, H)] if x_t == "mx8" else [_f64(t) for t in x]
    saved = pack_dev(gate_up, 2 * F) if saved_t == "mx8" else dev(gate_up)
    sv = [v.numpy() for v in values(saved, 2 * F)] if saved_t == "mx8" else [_f64(t) for t in saved]
    dx = [torch.full((r, H), FILL, dtype=torch.bfloat16, device=DEV) for r in rows]
    wt = torch.float32 if dw_t == "fp32" else torch.bfloat16
    dw = {k: [torch.full((E, *t.shape[1:]), FILL, dtype=wt, device=DEV) for t in st[k]] for k in ("w_gate", "w_up", "w_down")}
    full, scratch = scratch_for(st, x_t, True)
    gc.gc_moe_ffn_backward(dev(dy), x, saved, rows, st["splits_dev"], E, H, F, dev(st["w_gate"]), dev(st["w_up"]),
                           dev(st["w_down"]), dx, dw["w_gate"], dw["w_up"], dw["w_down"], scratch)
    torch.cuda.synchronize()
    assert bool((full[len(scratch):] == 0x5A).all())
    return xv, sv, dx, dw


def check_backward(st, xv, sv, dy, dx, dw, dw_t):
    H, F = st["H"], st["F"]
    out = HALF if dw_t == "bf16" else U
    for d, e, at, n in L.blocks(st["splits"], st["rows"]):
        if not n:
            for k in dw:
                assert not dw[k][d][e].any(), f"rank {d} expert {e}: {k} of an empty block"
            continue
        x, g, u = xv[d][at:at + n], sv[d][at:at + n, :F], sv[d][at:at + n, F:]
        y = _f64(dy[d][at:at + n])
        wg, wu, wd = (_f64(st[k][d][e]) for k in ("w_gate", "w_up", "w_down"))
        b = L.ffn_backward(y, x, g, u, wg, wu, wd)
        a = np.abs
        edh = 2 * H * U * (a(y) @ a(wd))
        es = sig_error(g)
        # silu' = s (1 + g (1 - s)): s within es, the difference 1 - s within es + u in absolute terms
        ed = a(L.dsilu(g)) * es + (a(g) * (es + 2 * U) + 8 * U)
        edg = edh * a(u * L.dsilu(g)) + a(b["dh"] * u) * ed + 4 * U * a(b["dg"])
        edg = edg + HALF * (a(b["dg"]) + edg) + 1e-38
        edu = edh * a(L.silu(g)) + a(b["du"]) * (es + 4 * U)
        edu = edu + HALF * (a(b["du"]) + edu) + 1e-38
        eh = a(b["h"]) * (es + 4 * U)
        eh = eh + HALF * (a(b["h"]) + eh) + 1e-38
        dg, du, h = a(b["dg"]) + edg, a(b["du"]) + edu, a(b["h"]) + eh
        exs = {"dx": edg @ a(wg) + edu @ a(wu) + 4 * F * U * (dg @ a(wg) + du @ a(wu)),
               "w_gate": edg.T @ a(x) + 2 * n * U * (dg.T @ a(x)),
               "w_up": edu.T @ a(x) + 2 * n * U * (du.T @ a(x)),
               "w_down": a(y).T @ eh + 2 * n * U * (a(y).T @ h)}
        got = {"dx": _f64(dx[d][at:at + n]), **{k: _f64(dw[k][d][e]) for k in dw}}
        for k, ref in (("dx", b["dx"]), ("w_gate", b["dwg"]), ("w_up", b["dwu"]), ("w_down", b["dwd"])):
            err = exs[k] + (HALF if k == "dx" else out) * (a(ref) + exs[k]) + 1e-38
            assert np.all(a(got[k] - ref) <= err), f"rank {d} expert {e}: {k} {np.max(a(got[k] - ref) / err)}"
    for d in range(st["N"]):
        end = max((p + n for dd, _, p, n in L.blocks(st["splits"], st["rows"]) if dd == d), default=0)
        assert bool((dx[d][end:] == FILL).all())


@pytest.mark.parametrize("counts,H,F", SHAPES)
@pytest.mark.parametrize("x_t,saved_t,dw_t", [("bf16", "bf16", "bf16"), ("bf16", "bf16", "fp32"), ("mx8", "mx8", "bf16"),
                                              ("bf16", "mx8", "fp32")])
def test_backward(counts, H, F, x_t, saved_t, dw_t):
    if saved_t == "mx8" and F % 32:
        F = (F + 31) // 32 * 32
    rng = np.random.default_rng(H * 5 + F + len(counts))
    st = make(rng, counts, H, F)
    gate_up = [_bf16(rng, (r, 2 * F), 1.5) for r in st["rows"]]
    dy = [_bf16(rng, (r, H)) for r in st["rows"]]
    xv, sv, dx, dw = run_backward(st, x_t, saved_t, dw_t, gate_up, dy)
    check_backward(st, xv, sv, dy, dx, dw, dw_t)


def test_no_rows_at_all():
    """Every block empty: the forward writes nothing, the weight gradients are zeros."""
    rng = np.random.default_rng(0)
    st = make(rng, [[0, 0], [0, 0]], 64, 32, spare=0)
    xv, y, _ = run_forward(st, "bf16", None)
    gate_up = [_bf16(rng, (0, 64)) for _ in range(2)]
    xv, sv, dx, dw = run_backward(st, "bf16", "bf16", "bf16", gate_up, [_bf16(rng, (0, 64))] * 2)
    check_backward(st, xv, sv, [_bf16(rng, (0, 64))] * 2, dx, dw, "bf16")


def test_malformed_split_table_stays_inside_the_buffers():
    """Negative and oversized entries: blocks end at the buffers' rows."""
    rng = np.random.default_rng(9)
    st = make(rng, [[5, 9, 4], [3, 0, 2]], 64, 64, spare=0)
    st["splits"][0, 0] = [2, -7, 1 << 40]
    st["splits"][1, 1] = [1 << 62, 5, 5]
    st["splits_dev"] = torch.from_numpy(st["splits"].reshape(-1)).to(DEV)
    xv, y, saved = run_forward(st, "bf16", "bf16")
    check_forward(st, xv, y, saved, "bf16")


def test_non_finite_rows_stay_in_their_row():
    rng = np.random.default_rng(4)
    st = make(rng, [[40, 30]], 96, 64)
    st["x"][0][7, 3] = float("inf")
    st["x"][0][45, 0] = float("nan")
    _, y, saved = run_forward(st, "bf16", "mx8")
    got = _f64(y[0][:70])
    bad = ~np.isfinite(got).all(1)
    assert bad[[7, 45]].all() and bad.sum() == 2
    v = L.unpack8(saved[0].cpu().numpy()[:70], 128)
    assert (~np.isfinite(v)).any(1).sum() == 2
